"""Routing, expert plans and the experts' products against the 64-bit statements of
tests/mx_reference.py.

Ids and plans must be equal. Routing weights are computed in 64 bits and rounded once to
fp32: half a step, 2^-24, with room for the 64-bit sums' own roundings (a part in 2^40).
Products: as in tests/test_mx.py. Gate and up each have an error of at most
d = (4 ceil(D/128) + 16) 2^-23 S. silu changes by at most 1.1 times a change of its input
(its slope's largest value is below 1.1); its exponential, sum and quotient are off by less
than 2^-19 of it together, or of |g| 2^-19 where exp is evaluated at 2^-24 relative error of
its argument (|g| 2^-24 <= 2^-19 for |g| <= 32, and beyond that silu is g or below 1e-12).
"""
import numpy as np
import pytest

import tests.mx_reference as ref

pytestmark = pytest.mark.gpu

HALF_STEP = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}


@pytest.fixture(scope="module")
def mq():
    import torch
    assert torch.cuda.is_available()
    import dense_sparse_bit_amd
    return dense_sparse_bit_amd


def _dtype(name):
    import torch
    return {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[name]


def _np(t):
    return t.detach().double().cpu().numpy()


def _check_route(mq, logits, k, score="softmax", bias=None, groups=1, top_groups=None, group_score="max",
                 renormalize=True, scale=1.0):
    top_groups = groups if top_groups is None else top_groups
    ids, weights = mq.route(logits, k, score=score, bias=bias, groups=groups, top_groups=top_groups,
                            group_score=group_score, renormalize=renormalize, scale=scale)
    want_ids, want = ref.route(_np(logits), k, score, None if bias is None else _np(bias), groups, top_groups, group_score,
                               renormalize, scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), want_ids)
    got = _np(weights)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(want))
    ok = ~np.isnan(want)
    assert (np.abs(got - want)[ok] <= (2.0 ** -24 + 2.0 ** -40) * np.abs(want)[ok] + 2.0 ** -149).all()
    return ids, weights


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("T,E,k", [(1, 8, 2), (1, 128, 8), (3, 1, 1), (5, 60, 6), (7, 64, 8), (33, 65, 4), (9, 256, 8),
                                   (4, 257, 16), (3, 512, 32), (2, 1000, 10), (2, 1024, 32), (200, 130, 1)])
def test_route(mq, dtype, T, E, k):
    import torch
    print(f"[route] {T} {E} {k} {dtype}", flush=True)
    g = torch.Generator().manual_seed(T * E + k)
    logits = (3 * torch.randn(T, E, generator=g)).to(_dtype(dtype)).cuda()
    bias = (0.2 * torch.randn(E, generator=g)).cuda()
    for score in ("softmax", "sigmoid"):
        for b in (None, bias):
            _check_route(mq, logits, k, score=score, bias=b)
            _check_route(mq, logits, k, score=score, bias=b, renormalize=False, scale=2.5)


@pytest.mark.parametrize("E,groups,top_groups,k", [(16, 4, 2, 3), (256, 8, 4, 8), (64, 64, 5, 5), (160, 8, 3, 6), (96, 2, 1, 8),
                                                   (1024, 32, 4, 16), (12, 12, 4, 4)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_route_groups(mq, E, groups, top_groups, k, group_score):
    import torch
    g = torch.Generator().manual_seed(E + groups)
    logits = (2 * torch.randn(21, E, generator=g)).cuda()
    logits[3, : E // 2] = -float("inf")
    logits[4] = -float("inf")
    logits[5] = 0.25                                                  # every group and expert level
    logits[6, 1:] = -float("inf")
    for score in ("softmax", "sigmoid"):
        for bias in (None, (0.1 * torch.randn(E, generator=g)).cuda()):
            _check_route(mq, logits, k, score=score, bias=bias, groups=groups, top_groups=top_groups,
                         group_score=group_score)


def test_route_masks_ties_and_faults(mq):
    import torch
    inf, nan = float("inf"), float("nan")
    x = torch.zeros(12, 96)
    x[0] = -inf                                                       # nothing left
    x[1] = -inf
    x[1, 70] = 2.0                                                    # one expert for four slots
    x[2] = torch.arange(96) % 5                                       # ties everywhere
    x[3, 50] = nan
    x[4, 60] = inf
    x[5] = 3.4e38                                                     # the type's largest values
    x[6] = -3.4e38
    x[7] = torch.linspace(-2000, 2000, 96)                            # scores that underflow
    x[8] = torch.linspace(40, 700, 96)                                # sigmoids of one
    x[9, :90] = -inf
    x[10] = torch.linspace(-1, 1, 96)
    x[10, 95] = -3.4028234663852886e38
    bias = torch.zeros(96)
    bias[3], bias[95] = -inf, 0.5
    for b in (None, bias.cuda()):
        for score in ("softmax", "sigmoid"):
            for groups, top in ((1, 1), (8, 2)):
                for gs in ("max", "top2"):
                    _check_route(mq, x.cuda(), 4, score=score, bias=b, groups=groups, top_groups=top, group_score=gs)
    bad = bias.clone()
    bad[11] = nan
    _check_route(mq, x.cuda(), 4, bias=bad.cuda())
    # rows of a wider matrix, and no tokens
    wide = torch.randn(9, 200, generator=torch.Generator().manual_seed(2)).cuda()
    _check_route(mq, wide[:, 10:106], 4)
    _check_route(mq, wide[::2, 3:67].bfloat16(), 4)
    ids, weights = mq.route(wide[:0], 4)
    assert ids.shape == (0, 4) and weights.shape == (0, 4)


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 64), (3, 2, 5), (16, 4, 8), (100, 8, 128), (1000, 3, 7), (5, 32, 1024),
                                   (2500, 4, 33), (0, 4, 8), (700, 16, 600)])
def test_expert_plan(mq, T, k, E):
    import torch
    print(f"[plan] {T} {k} {E}", flush=True)
    g = torch.Generator().manual_seed(T + E)
    uneven = (torch.rand(T, k, generator=g) ** 3 * E).long().clamp(max=E - 1)
    for ids in (uneven, torch.full((T, k), E - 1), torch.full((T, k), -1),
                torch.where(torch.rand(T, k, generator=g) < 0.3, torch.tensor(E + 5), uneven),
                torch.where(torch.rand(T, k, generator=g) < 0.3, torch.tensor(-2 ** 31), uneven)):
        ids = ids.to(torch.int32)
        p = mq.expert_plan(ids.cuda(), E)
        for name, got, want in zip(("offsets", "row_token", "row_of"), p, ref.plan(ids.numpy(), E)):
            np.testing.assert_array_equal(got.cpu().numpy(), want, err_msg=name)


def _mixture(mq, T, k, E, D, I, x_type, seed, empty=0.1):
    import torch
    g = torch.Generator().manual_seed(seed)
    x = (torch.randn(T, D, generator=g) * torch.exp(0.5 * torch.randn(D, generator=g))).to(_dtype(x_type)).cuda()
    wg, wu = (torch.randn(2, E, I, D, generator=g) / D ** 0.5).cuda()
    wd = (torch.randn(E, D, I, generator=g) / I ** 0.5).cuda()
    ids = (torch.rand(T, k, generator=g) ** 2 * E).long().clamp(max=E - 1)
    ids = torch.where(torch.rand(T, k, generator=g) < empty, -1, ids).to(torch.int32).cuda()
    weights = torch.rand(T, k, generator=g).cuda()
    return x, [mq.mx_quantize(w) for w in (wg, wu, wd)], ids, weights


MIXTURES = [(1, 1, 1, 32, 16), (1, 8, 16, 256, 64), (2, 2, 4, 130, 40), (7, 3, 5, 520, 100), (16, 4, 8, 256, 128),
            (17, 2, 3, 128, 33), (40, 4, 6, 384, 96), (150, 2, 3, 200, 72), (300, 4, 4, 512, 256), (64, 8, 64, 128, 48),
            (600, 1, 2, 96, 520)]


@pytest.mark.parametrize("x_type,y_type", [("bf16", "fp32"), ("fp32", "bf16"), ("fp16", "fp16")])
@pytest.mark.parametrize("T,k,E,D,I", MIXTURES)
def test_experts(mq, T, k, E, D, I, x_type, y_type):
    import torch
    print(f"[experts] {T} {k} {E} {D} {I} {x_type}", flush=True)
    x, (wg, wu, wd), ids, weights = _mixture(mq, T, k, E, D, I, x_type, T + D)
    plan = mq.expert_plan(ids, E)
    h = mq.mx_experts_up(x, wg, wu, plan, out_dtype=_dtype(y_type))
    rows = plan.row_token.numel()
    assert h.shape == (rows, I)
    row_token, row_of = plan.row_token.cpu().numpy(), plan.row_of.cpu().numpy()
    expert = np.searchsorted(plan.offsets.cpu().numpy(), np.arange(rows), side="right") - 1
    xv = _np(mq.mx_dequantize(mq.mx_quantize(x)))
    gv, uv, dv = (_np(mq.mx_dequantize(w)) for w in (wg, wu, wd))
    got = _np(h)
    unit = (4 * -(-D // 128) + 16) * 2.0 ** -23
    for p in range(rows):
        t = row_token[p]
        if t < 0:
            assert (got[p] == 0).all(), p
            continue
        e = expert[p]
        gate, up = gv[e] @ xv[t], uv[e] @ xv[t]
        dg, du = unit * (np.abs(gv[e]) @ np.abs(xv[t])), unit * (np.abs(uv[e]) @ np.abs(xv[t]))
        act = gate / (1 + np.exp(-gate))
        want = act * up
        tol = 1.1 * dg * (np.abs(up) + du) + np.abs(act) * du + 2.0 ** -19 * np.abs(act * up) + 1e-12 * np.abs(up)
        tol += HALF_STEP[y_type] * (np.abs(want) + tol) + (2.0 ** -25 if y_type == "fp16" else 0)
        assert (np.abs(got[p] - want) <= tol).all(), (p, float((np.abs(got[p] - want) / tol).max()))
    # down: from the rows as they are, whatever the rows of no token hold
    h = h.clone()
    h[plan.row_token < 0] = float("nan")
    y = mq.mx_experts_down(h, wd, plan, weights, out_dtype=_dtype(y_type))
    hv = _np(mq.mx_dequantize(mq.mx_quantize(h)))
    w = _np(weights)
    unit = (4 * -(-I // 128) + 16) * 2.0 ** -23
    want, tol = np.zeros((T, D)), np.zeros((T, D))
    for t in range(T):
        for j in range(k):
            p = row_of[t, j]
            if p >= 0:
                want[t] += w[t, j] * (dv[expert[p]] @ hv[p])
                # k weighted terms are added in fp32: at most k + 1 roundings of the terms' size
                tol[t] += w[t, j] * (unit + (k + 1) * 2.0 ** -23) * (np.abs(dv[expert[p]]) @ np.abs(hv[p]))
    tol += HALF_STEP[y_type] * (np.abs(want) + tol) + (2.0 ** -25 if y_type == "fp16" else 0)
    err = np.abs(_np(y) - want)
    assert (err <= tol).all(), float((err / np.maximum(tol, 1e-300)).max())
    # repeated calls give the same bits
    assert torch.equal(y, mq.mx_experts_down(h, wd, plan, weights, out_dtype=_dtype(y_type)))


def test_experts_nan_weights_and_empty_batches(mq):
    import torch
    x, (wg, wu, wd), ids, weights = _mixture(mq, 6, 2, 4, 96, 64, "bf16", 1, empty=0.0)
    ids[2] = -1
    ids[4] = -1
    weights[4] = float("nan")
    plan = mq.expert_plan(ids, 4)
    y = mq.mx_experts(x, wg, wu, wd, plan, weights, out_dtype=torch.float32)
    assert (y[2] == 0).all() and torch.isnan(y[4]).all()
    assert torch.isfinite(y[[0, 1, 3, 5]]).all()
    none = mq.expert_plan(ids[:0], 4)
    assert mq.mx_experts(x[:0], wg, wu, wd, none, weights[:0]).shape == (0, 96)
    # all slots without an expert
    away = mq.expert_plan(torch.full_like(ids, 9), 4)
    assert (mq.mx_experts(x, wg, wu, wd, away, torch.ones_like(weights)) == 0).all()


def test_experts_take_a_malformed_plan_without_harm(mq):
    """Entries out of range mean "no row": wrong numbers in, no access outside the buffers."""
    import torch
    x, (wg, wu, wd), ids, weights = _mixture(mq, 40, 2, 4, 128, 64, "bf16", 2, empty=0.0)
    plan = mq.expert_plan(ids, 4)
    far = torch.tensor([2 ** 31 - 1, -2 ** 31, 10 ** 6, -7], dtype=torch.int32, device="cuda")
    for field, t in zip(("offsets", "row_token", "row_of"), plan):
        bad = t.clone().flatten()
        bad[1:5] = far
        p = plan._replace(**{field: bad.view_as(t)})
        h = mq.mx_experts_up(x, wg, wu, p)
        mq.mx_experts_down(h, wd, p, weights)
        torch.cuda.synchronize()


@pytest.mark.parametrize("T", [1, 5, 30, 400])
def test_mixture_in_a_graph(mq, T):
    """Routing, plan and experts captured once: replays follow new inputs."""
    import torch
    E, k, D, I = 8, 2, 256, 128
    x, (wg, wu, wd), _, _ = _mixture(mq, T, k, E, D, I, "bf16", 3)
    g = torch.Generator(device="cuda").manual_seed(4)
    router = torch.randn(D, E, generator=g, device="cuda", dtype=torch.bfloat16)
    logits = (x @ router).contiguous()

    def layer():
        ids, weights = mq.route(logits, k)
        return mq.mx_experts(x, wg, wu, wd, mq.expert_plan(ids, E), weights)

    eager = layer()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = layer()
    for i in range(4):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, eager), i
        x.copy_(torch.randn(T, D, generator=g, device="cuda"))
        logits.copy_(x @ router)
        eager = layer()
