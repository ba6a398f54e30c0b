"""Group-scaled 4-bit weights and their products against the 64-bit statements of
tests/w4_reference.py.

Codes, scales and zero points are compared bit for bit. Products have two kinds of inputs:
- whole numbers and scales of one power of two: a sum of |x| (15 + z) below 2^24 units is
  exact in fp32 in any order, so outputs must be equal;
- free values: with A = the group's sum of |x|, the sums of x c and x z are made of at most
  3 * group additions (an fp32 value is three), each off by at most 2^-23 (truncation) of the
  magnitudes added, 15 A and z A; then one product, one addition a group, and one for each of
  up to 16 parts of K. So |y - exact| <= (3 group + groups + 24) 2^-23 S, S = the sum over
  groups of |s| (15 + |z|) A, plus half a step of the output's type.
"""
import numpy as np
import pytest

import tests.w4_reference as ref

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


def _dev(a, dtype="fp32"):
    import torch
    return torch.from_numpy(np.ascontiguousarray(a)).cuda().to(_dtype(dtype))


def _check_quantized(mq, x, group, kind, zeros):
    """x: device [R, K]; the library's codes, scales, zero points and values against the reference."""
    R, K = x.shape
    a = mq.w4_quantize(x, group=group, zeros=zeros, scale_dtype=_dtype(kind))
    codes, s, z = ref.quantize(_np(x), group, kind, zeros)
    np.testing.assert_array_equal(_np(a.scales), ref.pack_scales(s, R, K, group))
    if zeros:
        np.testing.assert_array_equal(_np(a.zeros), ref.pack_scales(z, R, K, group))
    else:
        assert a.zeros is None
    np.testing.assert_array_equal(a.codes.cpu().numpy(), ref.pack(codes))
    np.testing.assert_array_equal(_np(mq.w4_dequantize(a)), ref.values(codes, s, z, group).astype(np.float32))
    return a


SIZES = [(1, 1), (1, 32), (2, 31), (3, 33), (16, 128), (17, 129), (15, 512), (33, 520), (7, 1000), (70, 2056)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("dtype,kind", [("fp32", "fp16"), ("bf16", "bf16"), ("fp16", "fp16"), ("fp32", "bf16")])
def test_quantize_matches_the_reference(mq, dtype, kind, group, zeros):
    import torch
    for R, K in SIZES:
        g = torch.Generator(device="cuda").manual_seed(R * 1000 + K)
        x = (torch.randn(R, K, generator=g, device="cuda") * torch.exp(2 * torch.randn(R, 1, generator=g, device="cuda")))
        _check_quantized(mq, x.to(_dtype(dtype)), group, kind, zeros)


@pytest.mark.parametrize("zeros", [False, True])
def test_quantize_at_ties_extremes_and_not_finite(mq, zeros):
    """Quotients on half steps and next to them, groups of zeros, of one sign, of subnormals, of
    the largest values, and with NaN and infinities."""
    rng = np.random.default_rng(1)
    rows = []
    for s in (1.0, 0.75, 2.0 ** -24, 2.0 ** -20 * 1.0009765625, 1000.0):
        half = (np.arange(-15, 16) / 2 * s).astype(np.float32)
        half[0], half[1] = 7 * s, -7 * s
        for step in (0, 1, -1):
            v = half.copy()
            for _ in range(abs(step)):
                v = np.nextafter(v, np.float32(np.inf if step > 0 else -np.inf))
            rows.append(np.append(v, 0))
    tiny = np.float32(2.0 ** -149)
    rows += [np.zeros(32), np.full(32, -0.0), np.linspace(1, 2, 32), np.linspace(-2, -1, 32), rng.integers(-40, 40, 32) * tiny,
             rng.integers(0, 3, 32) * tiny, rng.standard_normal(32) * 2.0 ** -126, rng.standard_normal(32) * 1e-38,
             np.linspace(-3.4e38, 3.4e38, 32), np.linspace(-4.6e5, 5e5, 32), np.full(32, 65504 * 7.0), rng.standard_normal(32) * 1e30]
    for bad in (np.nan, np.inf, -np.inf):
        v = rng.standard_normal(32)
        v[rng.integers(32)] = bad
        rows.append(v)
    x = np.array(rows, dtype=np.float32)
    for kind in ("fp16", "bf16"):
        _check_quantized(mq, _dev(x), 32, kind, zeros)
        _check_quantized(mq, _dev(np.concatenate((x, x[::-1]), 1)), 64, kind, zeros)
        _check_quantized(mq, _dev(x[:, :17]), 128, kind, zeros)


def test_quantize_batches_strides_and_outputs(mq):
    import torch
    g = torch.Generator(device="cuda").manual_seed(0)
    for dtype in ("fp32", "bf16"):
        wide = torch.randn(5, 40, 700, generator=g, device="cuda").to(_dtype(dtype))
        x = wide[:, 1::2, 3:333]
        a = mq.w4_quantize(x, group=64, zeros=True)
        back = mq.w4_dequantize(a)
        for b in range(5):
            one = _check_quantized(mq, x[b], 64, "fp16", True)
            assert torch.equal(one.codes, a.codes[b]) and torch.equal(one.scales, a.scales[b]) and torch.equal(one.zeros, a.zeros[b])
            assert torch.equal(mq.w4_dequantize(one), back[b])
        out = mq.w4_quantize(torch.zeros_like(x), group=64, zeros=True)
        again = mq.w4_quantize(x, group=64, zeros=True, out=out)
        assert again is out and torch.equal(out.codes, a.codes) and torch.equal(out.zeros, a.zeros)
        y = torch.empty(5, 20, 330, device="cuda", dtype=_dtype("bf16"))
        assert mq.w4_dequantize(a, out=y) is y
        assert torch.equal(y, back.to(_dtype("bf16")))


def _codes(seed, N, K, group, zeros, power=False, batch=None):
    """Codes, scales and zero points as a checkpoint holds them; power: scales 2^-6."""
    rng = np.random.default_rng(seed)
    lead = (N,) if batch is None else (batch, N)
    codes = rng.integers(0, 16, lead + (K,)).astype(np.uint8)
    per = lead + (-(-K // group),)
    s = np.full(per, 2.0 ** -6) if power else (0.5 + rng.random(per)) / 64
    z = rng.integers(0, 16, per).astype(np.float64) if zeros else None
    return codes, s, z


def _packed(mq, codes, s, z, group, kind="fp16"):
    import torch
    return mq.w4_pack(torch.from_numpy(codes).cuda(), _dev(s, kind), None if z is None else _dev(z, kind), group=group)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
def test_pack_places_codes_and_scales(mq, group, zeros):
    import torch
    for R, K in SIZES:
        codes, s, z = _codes(R + K, R, K, group, zeros)
        w = _packed(mq, codes, s, z, group, "bf16")
        np.testing.assert_array_equal(w.codes.cpu().numpy(), ref.pack(codes))
        np.testing.assert_array_equal(_np(w.scales), ref.pack_scales(_np(_dev(s, "bf16")), R, K, group))
        if zeros:
            np.testing.assert_array_equal(_np(w.zeros), ref.pack_scales(z, R, K, group))
    # a strided batch; the high bits of a byte do not count
    codes, s, z = _codes(3, 40, 70, group, zeros, batch=3)
    wide = torch.full((3, 80, 100), 255, dtype=torch.uint8, device="cuda")
    wide[:, ::2, 5:75] = torch.from_numpy(codes).cuda() | 16 * (torch.arange(70, device="cuda") % 16).to(torch.uint8)
    w = mq.w4_pack(wide[:, ::2, 5:75], _dev(s, "fp16"), None if z is None else _dev(z, "fp16"), group=group)
    for b in range(3):
        np.testing.assert_array_equal(w.codes[b].cpu().numpy(), ref.pack(codes[b]))
    np.testing.assert_array_equal(_np(mq.w4_dequantize(w)), ref.values(codes, _np(_dev(s, "fp16")), z, group).astype(np.float32))


def test_fractional_zero_points(mq):
    codes, s, _ = _codes(5, 20, 300, 64, False)
    z = _np(_dev(np.random.default_rng(6).random(s.shape) * 15, "fp16"))
    w = _packed(mq, codes, s, z, 64)
    s = _np(_dev(s, "fp16"))
    got, want = _np(mq.w4_dequantize(w)), ref.values(codes, s, z, 64)
    # c - z and its product with s, each rounded once: half a step of each
    step = np.repeat(s * (15 + z), 64, axis=1)[:, :300]
    assert (np.abs(got - want) <= 2 * 2.0 ** -24 * step).all()
    x = np.random.default_rng(7).integers(-8, 9, (3, 300)).astype(np.float64)
    _check_linear(mq, x, codes, s, z, 64, w, "fp16", "fp32")


def _bound(x, s, z, group, y_type, want, bias=0.0):
    K = x.shape[1]
    n = s.shape[-1]
    a = np.abs(np.pad(x, ((0, 0), (0, n * group - K)))).reshape(len(x), n, group).sum(2)
    S = a @ (np.abs(s) * (15 + (8 if z is None else np.abs(z)))).T + np.abs(bias)
    sums = (3 * group + n + 24) * 2.0 ** -23 * S
    return sums + HALF_STEP[y_type] * (np.abs(want) + sums) + (2.0 ** -25 if y_type == "fp16" else 0)


def _check_linear(mq, x, codes, s, z, group, w, x_type, y_type, bias=None, exact=False):
    b = None if bias is None else _dev(bias)
    got = _np(mq.w4_linear(_dev(x, x_type), w, bias=b, out_dtype=_dtype(y_type)))
    xv = _np(_dev(x, x_type))
    want = xv @ ref.values(codes, s, z, group).T + (0 if bias is None else bias)
    if exact:
        np.testing.assert_array_equal(got, want)
    else:
        assert (np.abs(got - want) <= _bound(xv, s, z, group, y_type, want, 0.0 if bias is None else bias)).all()


# rows around the tiles' and the ways' borders, columns and inputs that fit no tile
PRODUCTS = [(1, 1, 1), (1, 16, 128), (1, 17, 7), (2, 100, 129), (3, 40, 512), (4, 64, 1000), (5, 33, 520), (8, 48, 2056), (15, 50, 77),
            (16, 16, 4096), (17, 70, 640), (31, 130, 300), (32, 64, 128), (33, 33, 33), (48, 257, 384), (64, 128, 1536), (65, 40, 200),
            (100, 300, 260), (128, 256, 256), (129, 513, 640), (300, 100, 1100)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("x_type", ["bf16", "fp16", "fp32"])
def test_linear_of_whole_numbers_is_exact(mq, x_type, group, zeros):
    """|x| <= 8, K <= 4096: a sum of |x| (15 + 15) is at most 2^20."""
    for M, N, K in PRODUCTS:
        codes, s, z = _codes(M * 7 + N * 3 + K, N, K, group, zeros, power=True)
        w = _packed(mq, codes, s, z, group)
        x = np.random.default_rng(M + N + K).integers(-8, 9, (M, K)).astype(np.float64)
        bias = np.random.default_rng(N).integers(-64, 65, N) / 64.0
        _check_linear(mq, x, codes, s, z, group, w, x_type, "fp32", bias=bias if N % 2 else None, exact=True)


@pytest.mark.parametrize("y_type", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("x_type", ["bf16", "fp16", "fp32"])
def test_linear_of_free_values(mq, x_type, y_type):
    for i, (M, N, K) in enumerate(PRODUCTS):
        group, zeros, kind = (32, 64, 128)[i % 3], i % 2 == 0, ("fp16", "bf16")[i // 2 % 2]
        codes, s, z = _codes(i, N, K, group, zeros)
        w = _packed(mq, codes, s, z, group, kind)
        rng = np.random.default_rng(i)
        x = rng.standard_normal((M, K)) * np.exp(rng.standard_normal((1, K)))
        _check_linear(mq, x, codes, _np(_dev(s, kind)), z, group, w, x_type, y_type, bias=rng.standard_normal(N).astype(np.float32))


def test_fp32_rows_keep_all_their_bits(mq):
    """A row with one value has no sums: x c and x z are each two products at most away from
    exact, and the pieces that x is cut into add up to all of it."""
    rng = np.random.default_rng(3)
    for K, M in ((1, 1), (40, 40), (300, 70)):
        x = np.zeros((M, K))
        x[np.arange(M), np.arange(M) % K] = rng.standard_normal(M).astype(np.float32)
        codes, s, z = _codes(K, 48, K, 32, True)
        w = _packed(mq, codes, s, z, 32)
        s = _np(_dev(s, "fp16"))
        got = _np(mq.w4_linear(_dev(x), w, out_dtype=_dtype("fp32")))
        want = x @ ref.values(codes, s, z, 32).T
        most = np.abs(x) @ np.abs(ref.values(codes * 0 + 15, s, -z, 32)).T
        # three pieces' products into each of two sums, the product by z, the difference, the scale
        assert (np.abs(got - want) <= 9 * 2.0 ** -23 * most).all()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("M", [1, 20, 200])
def test_linear_strides_and_odd_starts(mq, dtype, M):
    import torch
    codes, s, z = _codes(1, 70, 333, 64, True, power=True)
    w = _packed(mq, codes, s, z, 64)
    x = np.random.default_rng(2).integers(-8, 9, (M, 333)).astype(np.float64)
    want = x @ ref.values(codes, s, z, 64).T
    wide = torch.full((2 * M, 700), float("nan"), device="cuda", dtype=_dtype(dtype))
    for start in (0, 1, 5):
        wide.fill_(float("nan"))
        wide[::2, start:start + 333] = _dev(x, dtype)
        np.testing.assert_array_equal(_np(mq.w4_linear(wide[::2, start:start + 333], w, out_dtype=_dtype("fp32"))), want)
    row = _dev(x[:1], dtype).expand(M, 333)
    np.testing.assert_array_equal(_np(mq.w4_linear(row, w, out_dtype=_dtype("fp32"))), np.repeat(want[:1], M, 0))


@pytest.mark.parametrize("M", [1, 40, 300])
def test_rows_that_are_not_finite_stay_among_themselves(mq, M):
    import torch
    codes, s, z = _codes(1, 50, 200, 32, True, power=True)
    w = _packed(mq, codes, s, z, 32)
    x = np.random.default_rng(2).integers(-8, 9, (M, 200)).astype(np.float64)
    want = x @ ref.values(codes, s, z, 32).T
    for dtype in ("bf16", "fp32"):
        for bad in (float("nan"), float("inf")):
            xb = _dev(x, dtype)
            xb[M // 2, 77] = bad
            got = _np(mq.w4_linear(xb, w, out_dtype=_dtype("fp32")))
            assert np.isnan(got[M // 2]).all()
            others = np.arange(M) != M // 2
            np.testing.assert_array_equal(got[others], want[others])
    # a group that is NaN makes its column NaN
    scales = _dev(s, "fp16")
    scales[7, 3] = float("nan")
    w = mq.w4_pack(torch.from_numpy(codes).cuda(), scales, _dev(z, "fp16"), group=32)
    got = _np(mq.w4_linear(_dev(x, "bf16"), w, out_dtype=_dtype("fp32")))
    assert np.isnan(got[:, 7]).all()
    others = np.arange(50) != 7
    np.testing.assert_array_equal(got[:, others], want[:, others])


# ------------------------------------------------------------------------------ experts
def _plan(mq, seed, T, E, k, lost=0.1):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    logits = torch.randn(T, E, generator=g, device="cuda") + 2 * torch.randn(E, generator=g, device="cuda")
    ids = logits.topk(k, dim=1).indices.to(torch.int32)
    if T > 1:
        ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < lost, -1, ids).to(torch.int32).contiguous()
    return ids, mq.expert_plan(ids, E)


def _experts_want(x, codes, s, z, group, plan, by_token):
    offsets, row_token = plan.offsets.cpu().numpy(), plan.row_token.cpu().numpy()
    want = np.zeros((len(row_token), codes.shape[1]))
    for e in range(len(offsets) - 1):
        p = np.arange(offsets[e], offsets[e + 1])
        p = p[row_token[p] >= 0]
        want[p] = x[row_token[p] if by_token else p] @ ref.values(codes[e], s[e], None if z is None else z[e], group).T
    return want


EXPERTS = [(1, 4, 1, 16, 128), (1, 8, 8, 40, 300), (3, 64, 2, 33, 129), (7, 5, 3, 100, 512), (40, 4, 2, 70, 77), (150, 9, 4, 130, 640),
           (700, 3, 2, 260, 256)]


@pytest.mark.parametrize("by_token", [False, True])
@pytest.mark.parametrize("x_type", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (128, False)])
def test_experts_linear_of_whole_numbers_is_exact(mq, x_type, group, zeros, by_token):
    for T, E, k, N, K in EXPERTS:
        codes, s, z = _codes(T + E, N, K, group, zeros, power=True, batch=E)
        w = _packed(mq, codes, s, z, group)
        _, plan = _plan(mq, T, T, E, k)
        rows = plan.row_token.numel()
        x = np.random.default_rng(T).integers(-8, 9, (T if by_token else rows, K)).astype(np.float64)
        want = _experts_want(x, codes, s, z, group, plan, by_token)
        xd = _dev(x, x_type)
        if not by_token:                               # rows of no token do not count
            xd[plan.row_token < 0] = float("nan")
        got = _np(mq.w4_experts_linear(xd, w, plan, by_token=by_token, out_dtype=_dtype("fp32")))
        np.testing.assert_array_equal(got, want)


def test_experts_linear_types_strides_and_no_tokens(mq):
    import torch
    T, E, k, N, K = 60, 6, 2, 72, 200
    codes, s, z = _codes(0, N, K, 64, True, batch=E)
    w = _packed(mq, codes, s, z, 64, "bf16")
    s = _np(_dev(s, "bf16"))
    _, plan = _plan(mq, 1, T, E, k)
    x = np.random.default_rng(0).standard_normal((T, K))
    wide = torch.full((T, 400), float("nan"), device="cuda", dtype=_dtype("bf16"))
    wide[:, 3:3 + K] = _dev(x, "bf16")
    xv = _np(_dev(x, "bf16"))
    want = _experts_want(xv, codes, s, z, 64, plan, True)
    row_token = plan.row_token.cpu().numpy()
    offsets = plan.offsets.cpu().numpy()
    e = np.searchsorted(offsets, np.arange(len(row_token)), side="right") - 1
    for y_type in ("bf16", "fp16", "fp32"):
        y = torch.full((len(row_token), N), float("nan"), device="cuda", dtype=_dtype(y_type))
        got = mq.w4_experts_linear(wide[:, 3:3 + K], w, plan, by_token=True, y=y)
        assert got is y
        for i in range(E):
            p = np.flatnonzero((e == i) & (row_token >= 0))
            err = np.abs(_np(y)[p] - want[p])
            assert (err <= _bound(xv[row_token[p]], s[i], z[i], 64, y_type, want[p])).all()
        assert (y[plan.row_token < 0] == 0).all()
    # no expert for any token, and no tokens
    none = mq.expert_plan(torch.full((5, 2), -1, dtype=torch.int32, device="cuda"), E)
    got = mq.w4_experts_linear(_dev(x[:5], "bf16"), w, none, by_token=True)
    assert got.shape[0] == none.row_token.numel() and (got == 0).all()
    empty = mq.expert_plan(torch.empty((0, 2), dtype=torch.int32, device="cuda"), E)
    assert mq.w4_experts_linear(_dev(x[:0], "bf16"), w, empty).shape == (0, N)
    assert mq.w4_linear(_dev(x[:0], "bf16"), _packed(mq, codes[0], s[0], z[0], 64)).shape == (0, N)


@pytest.mark.parametrize("by_token", [False, True])
def test_experts_linear_with_a_malformed_plan_stays_in_range(mq, by_token):
    """Entries out of range are taken as no row: an offset past the rows, a token past T."""
    import torch
    T, E, k, N, K = 20, 4, 2, 40, 130
    codes, s, z = _codes(0, N, K, 32, False, power=True, batch=E)
    w = _packed(mq, codes, s, z, 32)
    _, plan = _plan(mq, 1, T, E, k, lost=0)
    rows = plan.row_token.numel()
    x = np.random.default_rng(0).integers(-8, 9, (T if by_token else rows, K)).astype(np.float64)
    row_token = plan.row_token.clone()
    live = torch.nonzero(row_token >= 0).flatten()
    row_token[live[0]], row_token[live[5]] = T, -7
    offsets = plan.offsets.clone()
    offsets[E] = 1 << 30
    got = _np(mq.w4_experts_linear(_dev(x, "bf16"), w, mq.ExpertPlan(offsets, row_token, plan.row_of), by_token=by_token,
                                   out_dtype=_dtype("fp32")))
    row_token[live[0]] = -1
    want = _experts_want(x, codes, s, None, 32, mq.ExpertPlan(plan.offsets, row_token, plan.row_of), by_token)
    np.testing.assert_array_equal(got, want)


# ------------------------------------------------------------------------------ streams, graphs
def test_linear_on_other_streams_and_in_a_graph(mq):
    import torch
    codes, s, z = _codes(1, 500, 640, 64, True)
    w = _packed(mq, codes, s, z, 64)
    bits = lambda t: t.view(torch.int16)
    for M in (1, 40, 200):
        x = torch.randn(M, 640, device="cuda").to(_dtype("bf16"))
        want = mq.w4_linear(x, w)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        got = mq.w4_linear(x, w, stream=side)
        side.synchronize()
        assert torch.equal(bits(got), bits(want))
        fixed = x.clone()
        with torch.cuda.stream(side):
            mq.w4_linear(fixed, w)
        side.synchronize()
        graphs, outs = [], []
        for _ in range(2):                             # two graphs, in turn
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                outs.append(mq.w4_linear(fixed, w))
            graphs.append(graph)
        for i in range(4):
            fixed.copy_(torch.randn(M, 640, device="cuda"))
            want = mq.w4_linear(fixed, w)
            torch.cuda.synchronize()
            graphs[i % 2].replay()
            torch.cuda.synchronize()
            assert torch.equal(bits(outs[i % 2]), bits(want))
