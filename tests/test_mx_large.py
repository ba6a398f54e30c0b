"""Sizes at which the microscaled and routing calls change their ways: plans of many
slots, down products in runs of columns, experts whose rows end around a block of rows,
many slots a token, tensors whose offsets pass 32 bits; and the example that runs the
operators together. Tolerances are those of tests/test_mx.py and tests/test_experts.py.
"""
import importlib.util
import os

import numpy as np
import pytest

import tests.mx_reference as ref

HALF_STEP = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8}


@pytest.fixture(scope="module")
def mq():
    import torch
    assert torch.cuda.is_available()
    import dense_sparse_bit_amd
    return dense_sparse_bit_amd


def _np(t):
    return t.detach().double().cpu().numpy()


def _plan(ids, E):
    """ref.plan without its loops over slots."""
    T, k = ids.shape
    flat = ids.reshape(-1).astype(np.int64)
    live = np.flatnonzero((flat >= 0) & (flat < E))
    order = live[np.argsort(flat[live], kind="stable")]
    count = np.bincount(flat[live], minlength=E)
    offsets = np.concatenate(([0], np.cumsum(-(-count // 16) * 16)))
    first = np.concatenate(([0], np.cumsum(count)))
    e = flat[order]
    row = offsets[e] + np.arange(len(order)) - first[e]
    row_of = np.full(T * k, -1, dtype=np.int64)
    row_token = np.full((T * k + 15 * min(T * k, E)) // 16 * 16, -1, dtype=np.int64)
    row_of[order], row_token[row] = row, order // k
    return offsets, row_token, row_of.reshape(T, k)


def test_plan_statement_agrees_with_the_loops():
    ids = np.random.default_rng(1).integers(-2, 9, (50, 3)).astype(np.int32)
    for got, want in zip(_plan(ids, 7), ref.plan(ids, 7)):
        np.testing.assert_array_equal(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E", [(32768, 8, 64), (32769, 8, 60), (300001, 1, 1024), (70000, 6, 1), (263000, 4, 1000)])
def test_plans_of_many_slots(mq, T, k, E):
    """Up to and beyond 2^18 slots (one launch, then chunks of slots); the last chunk is of
    another length than the others."""
    import torch
    print(f"[plan] {T} {k} {E}", flush=True)
    rng = np.random.default_rng(T)
    ids = (rng.random((T, k)) ** 3 * E).astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    ids[rng.random((T, k)) < 0.05] = E + 3
    p = mq.expert_plan(torch.from_numpy(ids).cuda(), E)
    for name, got, want in zip(("offsets", "row_token", "row_of"), p, _plan(ids, E)):
        np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=name)


def _layer(mq, ids, E, D, I, x_dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(D + I)
    T, k = ids.shape
    x = torch.randn(T, D, generator=g, device="cuda").to(x_dtype)
    w = [mq.mx_quantize(torch.randn(E, *s, generator=g, device="cuda") / s[1] ** 0.5) for s in ((I, D), (I, D), (D, I))]
    weights = torch.rand(T, k, generator=g, device="cuda")
    return x, w, mq.expert_plan(torch.from_numpy(ids).cuda(), E), weights


def _check_layer(mq, ids, E, D, I, x_dtype, y_type, tokens):
    """Both products, at the given tokens."""
    import torch
    y_dtype = {"fp32": torch.float32, "bf16": torch.bfloat16}[y_type]
    x, (wg, wu, wd), plan, weights = _layer(mq, ids, E, D, I, x_dtype)
    k = ids.shape[1]
    h = mq.mx_experts_up(x, wg, wu, plan, out_dtype=y_dtype)
    assert (h[plan.row_token < 0] == 0).all()
    row_of = plan.row_of.cpu().numpy()
    xv = _np(mq.mx_dequantize(mq.mx_quantize(x[torch.as_tensor(tokens, device="cuda")])))
    hv_all = mq.mx_dequantize(mq.mx_quantize(h))
    y = mq.mx_experts_down(h, wd, plan, weights, out_dtype=y_dtype)
    assert torch.equal(y, mq.mx_experts_down(h, wd, plan, weights, out_dtype=y_dtype))
    got_y, wn = _np(y[torch.as_tensor(tokens, device="cuda")]), _np(weights)
    read = {}

    def matrices(e):
        if e not in read:
            read[e] = [_np(mq.mx_dequantize(mq.MX(w.codes[e], w.scales[e], w.rows, w.cols))) for w in (wg, wu, wd)]
        return read[e]

    up_unit, down_unit = (4 * -(-D // 128) + 16) * 2.0 ** -23, (4 * -(-I // 128) + 16) * 2.0 ** -23
    for n, t in enumerate(tokens):
        want_y, tol_y = np.zeros(D), np.zeros(D)
        for j in range(k):
            p, e = row_of[t, j], ids[t, j]
            assert (p >= 0) == (0 <= e < E)
            if p < 0:
                continue
            g, u, d = matrices(e)
            gate, up = g @ xv[n], u @ xv[n]
            dg, du = up_unit * (np.abs(g) @ np.abs(xv[n])), up_unit * (np.abs(u) @ np.abs(xv[n]))
            act = gate / (1 + np.exp(-gate))
            want = act * up
            tol = 1.1 * dg * (np.abs(up) + du) + np.abs(act) * du + 2.0 ** -19 * np.abs(want) + 1e-12 * np.abs(up)
            tol += HALF_STEP[y_type] * (np.abs(want) + tol)
            assert (np.abs(_np(h[p]) - want) <= tol).all(), (t, j)
            hv = _np(hv_all[p])
            want_y += wn[t, j] * (d @ hv)
            tol_y += wn[t, j] * (down_unit + (k + 1) * 2.0 ** -23) * (np.abs(d) @ np.abs(hv))
        tol_y += HALF_STEP[y_type] * (np.abs(want_y) + tol_y)
        assert (np.abs(got_y[n] - want_y) <= tol_y).all(), (t, float((np.abs(got_y[n] - want_y) / np.maximum(tol_y, 1e-300)).max()))


@pytest.mark.gpu
@pytest.mark.parametrize("counts", [[127, 128, 129, 0, 1], [16, 17, 257, 383, 500], [0, 0, 1000], [33] * 12])
def test_experts_whose_rows_end_around_a_block(mq, counts):
    import torch
    print(f"[experts] {counts}", flush=True)
    ids = np.repeat(np.arange(len(counts)), counts).astype(np.int32)
    ids = np.random.default_rng(3).permutation(ids)[:, None]
    edges = [int(np.flatnonzero(ids[:, 0] == e)[i]) for e, c in enumerate(counts) if c for i in sorted({0, c // 2, c - 1})]
    _check_layer(mq, np.ascontiguousarray(ids), len(counts), 520, 200, torch.bfloat16, "fp32", edges)


@pytest.mark.gpu
@pytest.mark.parametrize("T,k,E", [(1, 33, 40), (5, 40, 64), (8, 32, 33), (40, 50, 64)])
def test_experts_of_many_slots(mq, T, k, E):
    import torch
    print(f"[experts] {T} {k} {E}", flush=True)
    rng = np.random.default_rng(T)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[rng.random((T, k)) < 0.1] = -1
    if T > 1:
        ids[1] = -1
    _check_layer(mq, ids, E, 260, 72, torch.float32, "bf16", list(range(min(T, 8))))


@pytest.mark.gpu
@pytest.mark.parametrize("D,I,y_type", [(2304, 64, "fp32"), (2301, 40, "bf16")])
def test_down_products_in_runs_of_columns(mq, D, I, y_type):
    """The rows' fp32 sums take more than a run may: two runs, the second a shorter one,
    with columns that are no multiple of four."""
    import torch
    T, k, E = 3000, 8, 8
    rng = np.random.default_rng(D)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    ids[rng.random((T, k)) < 0.02] = -1
    rows = mq.plan_rows(T, k, E)
    assert rows * D * 4 > 200 << 20 and rows * 256 * 4 < 200 << 20
    _check_layer(mq, ids, E, D, I, torch.bfloat16, y_type, [0, 1, 1499, 2998, 2999])


@pytest.mark.gpu
def test_offsets_beyond_32_bits(mq):
    """More than 2^31 elements in, out and on the way; the last rows are right."""
    import torch
    R, K = 70016, 32768
    x = torch.randn(64, K, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(torch.bfloat16)
    big = x.repeat(R // 64, 1)
    big[-1] *= 3
    a = mq.mx_quantize(big)
    back = mq.mx_dequantize(a, dtype=torch.bfloat16)
    one = mq.mx_dequantize(mq.mx_quantize(big[-64:]), dtype=torch.bfloat16)
    assert torch.equal(back[-64:], one) and torch.equal(back[35008:35072], back[:64])
    del back
    w = mq.mx_quantize(big[:K, 200:296])
    # the last rows: against 64 bits' values, as in tests/test_mx.py (one group of inputs)
    xv, wv = mq.mx_dequantize(mq.mx_quantize(big[-64:, :96])).double(), mq.mx_dequantize(w).double()
    want, size = xv @ wv.t().contiguous(), xv.abs() @ wv.abs().t().contiguous()
    tol = 20 * 2.0 ** -23 * size + 2.0 ** -8 * want.abs() * (1 + 2.0 ** -10)
    for operand in (mq.mx_quantize(big[:, :96]), big[:, :96]):
        y = mq.mx_linear(operand, w)
        assert y.numel() > 2 ** 31
        assert ((y[-64:].double() - want).abs() <= tol).all()
        del y


@pytest.mark.gpu
def test_quantizing_on_the_way_or_apart(mq):
    """Both sides of the rule give the bits of quantization and product."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(2)
    lib = mq.lib()
    for M, N, K in ((16, 4096, 4096), (16, 4096, 8208), (16, 40000, 4096), (17, 256, 512)):
        x = torch.randn(M, K, generator=g, device="cuda")
        w = mq.mx_quantize(torch.randn(N, K, generator=g, device="cuda"))
        apart = lib.mq_mx_linear_workspace_bytes(M, N, K) > 0
        assert apart == (M > 16 or M * K > 1 << 17 or M * K * N > 1 << 31)
        assert torch.equal(mq.mx_linear(x, w), mq.mx_linear(mq.mx_quantize(x), w)), (M, N, K)


def test_rows_beyond_32_bit_offsets_are_refused():
    import dense_sparse_bit_amd as mq
    lib = mq.lib()
    big, T, D = 0x10000, 1 << 22, 4096
    args = lambda t: (big, 1, D, t, 1, 64, D, 16, big, big, big, big, big, big, big, big, 1, None, 0, None)
    assert lib.mq_mx_experts_up_workspace_bytes(T, 1, 64, D, 16) == 0
    assert lib.mq_mx_experts_up(*args(T)) == -2
    assert lib.mq_mx_experts_up(*args(T // 4)) == -1                    # without a workspace


@pytest.mark.gpu
def test_refusals_on_the_device(mq):
    """Every refusal has its own error, an operand's included, and launches nothing."""
    import torch
    x = torch.randn(4, 64, device="cuda")
    w = mq.mx_quantize(torch.randn(20, 64, device="cuda"))
    ids, _ = mq.route(x, 2)
    plan = mq.expert_plan(ids, 64)
    with pytest.raises(RuntimeError, match="ambiguous"):
        mq.route(x, 2, renormalize=torch.zeros(2))
    for error, call in (
            (ValueError, lambda: mq.route(x, 65)), (ValueError, lambda: mq.route(x, 2, score="sum")),
            (ValueError, lambda: mq.route(x, 2, bias=torch.zeros(63, device="cuda"))),
            (TypeError, lambda: mq.route(x.double(), 2)), (ValueError, lambda: mq.route(x.t(), 2)),
            (mq.MQError, lambda: mq.route(x, 40)), (ValueError, lambda: mq.expert_plan(ids.long(), 64)),
            (ValueError, lambda: mq.expert_plan(ids, 0)), (ValueError, lambda: mq.expert_plan(ids.t(), 64)),
            (TypeError, lambda: mq.mx_quantize(x.double())), (ValueError, lambda: mq.mx_quantize(x.t())),
            (ValueError, lambda: mq.mx_quantize(x[:, :0])), (ValueError, lambda: mq.mx_linear(x[:, :63], w)),
            (ValueError, lambda: mq.mx_linear(x.cpu(), w)), (TypeError, lambda: mq.mx_linear(x, w, out_dtype=torch.int8)),
            (ValueError, lambda: mq.mx_linear(x, w, y=torch.empty(4, 19, device="cuda"))),
            (ValueError, lambda: mq.mx_linear(x, w._replace(rows=40))), (TypeError, lambda: mq.mx_dequantize(x)),
            (TypeError, lambda: mq.mx_experts_up(x, w, w, ids)), (ValueError, lambda: mq.mx_experts_up(x, w, w, plan))):
        with pytest.raises(error):
            call()
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_example():
    """The layer against plain fp32 over the same quantized values: bf16 rounds h before its
    second quantization, where a change of half a step can move a code by one; the result is
    rounded to bf16 (2^-9 on average below that)."""
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "examples", "mixture_layer.py")
    spec = importlib.util.spec_from_file_location("mixture_layer", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    assert all(e < 2.0 ** -6 for e in module.main(D=512, I=256, E=8, k=2))
