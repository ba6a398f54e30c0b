"""The ways of a product with group-scaled 4-bit weights, each at sizes that take it, against
float64 products on the device, whose errors are some 2^29 times below fp32's.

- Whole numbers: |x| <= 4 and |c - z| <= 15 over up to 8190 inputs, below 2^19 in all with scales
  2^-6: exact in fp32 in any order, so outputs must be equal.
- Free values and scales: with A = a group's sum of |x|, n groups and S = the sum over groups of
  |s| (15 + |z|) A, there are at most 3 * group additions a group to the sums of x c and x z (an
  fp32 value is three), each off by at most 2^-23 (truncation) of the magnitudes; a product by s
  or a change of units (2 roundings) and an addition a group; an addition for each of up to 8
  parts, and the bias: |y - exact| <= (3 group + 3 n + 24) 2^-23 S, and half a step of the output.
"""
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


def _weights(mq, g, N, K, group, kind, scales, zeros, batch=()):
    """Packed weights of random codes and their float64 values."""
    import torch
    codes = torch.randint(0, 16, batch + (N, K), generator=g, device="cuda", dtype=torch.uint8)
    s = scales(batch + (N, -(-K // group))).to(_dtype(kind))
    z = torch.randint(0, 16, s.shape, generator=g, device="cuda").to(s.dtype) if zeros else None
    w = mq.w4_pack(codes, s, z, group=group)
    wide = lambda v: v.double().repeat_interleave(group, -1)[..., :K]
    return w, s, z, (codes.double() - (8 if z is None else wide(z))) * wide(s)


def _bound(x, s, z, group, want, y_type):
    import torch
    n = s.shape[-1]
    a = torch.nn.functional.pad(x.double().abs(), (0, n * group - x.shape[1])).view(len(x), n, group).sum(2)
    S = a @ (s.double().abs() * (15 + (8 if z is None else z.double().abs()))).T.contiguous()
    sums = (3 * group + 3 * n + 24) * 2.0 ** -23 * S
    return sums + HALF_STEP[y_type] * (want.abs() + sums) + (2.0 ** -25 if y_type == "fp16" else 0)


@pytest.mark.parametrize("x_type,group,M,N,K,way", ref.WAYS)
def test_every_way_of_whole_numbers_is_exact(mq, x_type, group, M, N, K, way):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    assert mq.lib().mq_w4_linear_way(M, N, K, {"fp32": 0, "bf16": 1, "fp16": 2}[x_type], group) == way
    for zeros in (False, True):
        w, _, _, values = _weights(mq, g, N, K, group, "fp16", lambda shape: torch.full(shape, 2.0 ** -6, device="cuda"), zeros)
        x = torch.randint(-4, 5, (M, K), generator=g, device="cuda").to(_dtype(x_type))
        bias = torch.randint(-64, 65, (N,), generator=g, device="cuda") / 64.0
        want = (x.double() @ values.T.contiguous() + bias).float()
        assert torch.equal(mq.w4_linear(x, w, bias=bias, out_dtype=torch.float32), want)
        # rows further apart and off 16 bytes are taken by other loads, or through a copy
        wide = torch.full((M, K + 9), float("nan"), device="cuda", dtype=x.dtype)
        wide[:, 5:5 + K] = x
        assert torch.equal(mq.w4_linear(wide[:, 5:5 + K], w, bias=bias, out_dtype=torch.float32), want)


@pytest.mark.parametrize("x_type,group,M,N,K,way", ref.WAYS)
def test_every_way_with_scales_far_apart(mq, x_type, group, M, N, K, way):
    """Scales over 2^40 and more, of both signs, zero among them."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(M * 3 + N + K)
    kind = ("fp16", "bf16")[K % 2]

    def scales(shape):
        e = torch.randint(-24, 15, shape, generator=g, device="cuda") if kind == "fp16" else torch.randint(-28, 28, shape, generator=g, device="cuda")
        s = torch.ldexp(1 + torch.rand(shape, generator=g, device="cuda"), e.float())
        s = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.5, s, -s)
        return torch.where(torch.rand(shape, generator=g, device="cuda") < 0.2, torch.zeros_like(s), s)
    w, s, z, values = _weights(mq, g, N, K, group, kind, scales, True)
    x = torch.randn(M, K, generator=g, device="cuda").to(_dtype(x_type))
    want = x.double() @ values.T.contiguous()
    got = mq.w4_linear(x, w, out_dtype=torch.float32).double()
    assert ((got - want).abs() <= _bound(x, s, z, group, want, "fp32")).all()


@pytest.mark.parametrize("M,N,K", [(1, 48, 640), (4, 48, 640), (10, 48, 640), (40, 70, 640), (300, 30, 640), (300, 30, 2500), (700, 4100, 640)])
def test_scales_that_are_not_finite_stay_in_their_rows(mq, M, N, K):
    """A scale that is NaN makes its output NaN, and no other; scales below 2^-126 may count as 0."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + N)
    for group in (32, 64, 128):
        def scales(shape):
            s = (0.5 + torch.rand(shape, generator=g, device="cuda")) / 64
            s[3, 1], s[7, 0], s[N - 1, -1] = float("nan"), float("nan"), float("nan")
            s[5, 0], s[6, 2], s[8, :] = 2.0 ** -130, 2.0 ** -133, 2.0 ** -128
            return s
        w, s, z, values = _weights(mq, g, N, K, group, "bf16", scales, True)
        x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
        got = mq.w4_linear(x, w, out_dtype=torch.float32)
        bad = torch.zeros(N, dtype=torch.bool, device="cuda")
        bad[[3, 7, N - 1]] = True
        assert got[:, bad].isnan().all()
        want = (x.double() @ values.T.contiguous())[:, ~bad]
        near = _bound(x, s[~bad], z[~bad], group, want, "fp32") + 2.0 ** -126 * 30 * K * 8
        assert ((got[:, ~bad].double() - want).abs() <= near).all()


@pytest.mark.parametrize("group", [32, 128])
@pytest.mark.parametrize("M", [4, 300])
def test_a_scale_that_falls_step_by_step(mq, M, group):
    """2^120 down to 2^-120, no step of more than 2^60: what the last groups add is far below the
    first ones' last place, and the sums stay finite in any units."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    K, N = 8 * group, 40
    steps = torch.tensor([100.0, 60, 10, -20, -60, -100, -120, 90], device="cuda")
    w, s, z, values = _weights(mq, g, N, K, group, "bf16", lambda shape: torch.ldexp(torch.ones(shape, device="cuda"), steps), False)
    x = torch.randn(M, K, generator=g, device="cuda").bfloat16()
    want = x.double() @ values.T.contiguous()
    got = mq.w4_linear(x, w, out_dtype=torch.float32).double()
    assert ((got - want).abs() <= _bound(x, s, z, group, want, "fp32") + 2.0 ** -63 * 2.0 ** 100 * 30 * K * 8).all()


@pytest.mark.parametrize("x_type", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,E,k,N,K", [(400, 4, 2, 300, 264), (90, 2, 1, 2100, 130), (2000, 8, 4, 530, 512), (257, 3, 3, 64, 4100),
                                       (60, 4, 2, 300, 264), (70, 8, 4, 4500, 200), (100, 40, 10, 900, 130), (900, 16, 4, 4100, 130)])
def test_experts_tiles_by_token_and_by_row(mq, x_type, group, T, E, k, N, K):
    """Tiles of both sizes, rows from x itself and from a copy; a tenth of the slots without an expert."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T + N)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.int()
    ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.1, -1, ids).int().contiguous()
    plan = mq.expert_plan(ids, E)
    w, _, _, values = _weights(mq, g, N, K, group, "fp16", lambda shape: torch.full(shape, 2.0 ** -6, device="cuda"), True, (E,))
    x = torch.randint(-4, 5, (T, K), generator=g, device="cuda").to(_dtype(x_type))
    token = plan.row_token.long()
    real = token >= 0
    rows = torch.where(real[:, None], x[token.clamp(min=0)], torch.zeros((), dtype=x.dtype, device="cuda"))
    offsets = plan.offsets.tolist()
    want = torch.zeros(len(token), N, dtype=torch.float64, device="cuda")
    for e in range(E):
        at = slice(offsets[e], offsets[e + 1])
        want[at] = rows[at].double() @ values[e].T.contiguous()
    wide = torch.full((T, K + 7), float("nan"), device="cuda", dtype=x.dtype)
    wide[:, 3:3 + K] = x
    for got in (mq.w4_experts_linear(x, w, plan, by_token=True, out_dtype=torch.float32),
                mq.w4_experts_linear(wide[:, 3:3 + K], w, plan, by_token=True, out_dtype=torch.float32),
                mq.w4_experts_linear(torch.where(real[:, None], rows, float("nan")), w, plan, out_dtype=torch.float32)):
        assert torch.equal(got, want.float())


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("T", [1, 5, 64, 400])
def test_a_layer_of_experts_as_it_is_served(mq, T, dtype):
    """Scores to experts, tokens' rows through two products of each expert and back, as one run,
    eagerly and replayed from a graph. Against float64 over the same roundings of what goes
    between the calls; what the calls round differently shows as one step more of each."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    E, k, D, H = 8, 2, 200, 136
    t = _dtype(dtype)
    small = lambda shape: (0.5 + torch.rand(shape, generator=g, device="cuda")) / 256
    w1, s1, z1, v1 = _weights(mq, g, 2 * H, D, 64, "fp16", small, True, (E,))
    w2, s2, z2, v2 = _weights(mq, g, D, H, 32, "fp16", small, False, (E,))
    x = torch.randn(T, D, generator=g, device="cuda").to(t)
    scores = torch.randn(T, E, generator=g, device="cuda")

    def layer():
        ids, weights = mq.route(scores, k)
        plan = mq.expert_plan(ids, E)
        gate, up = mq.w4_experts_linear(x, w1, plan, by_token=True).chunk(2, dim=1)
        out = mq.w4_experts_linear(torch.nn.functional.silu(gate) * up, w2, plan)
        return mq.experts_combine(out, plan, weights), ids, weights

    y, ids, weights = layer()
    eps, tiny = HALF_STEP[dtype], 2.0 ** -25 if dtype == "fp16" else 0.0
    want = torch.zeros(T, D, dtype=torch.float64, device="cuda")
    near = torch.zeros_like(want)
    for j in range(k):
        e = ids[:, j].long()
        h = torch.bmm(v1[e].contiguous(), x.double()[:, :, None].contiguous())[:, :, 0]
        # (scales are at most 1.5 / 256, so |s| (15 + z) is below 30 / 128)
        err = (3 * 64 + 3 * 4 + 24) * 2.0 ** -23 * 30 * x.double().abs().sum(1, keepdim=True) / 128 + eps * h.abs() + tiny
        gate, up = h.chunk(2, 1)
        eg, eu = err.chunk(2, 1)
        a = torch.nn.functional.silu(gate) * up
        # silu' is at most 1.1; silu is rounded, the product too
        ea = 1.1 * eg * (up.abs() + eu) + (gate.abs() + 1.1 * eg) * eu + 2.1 * eps * a.abs() + 2 * tiny * (1 + up.abs())
        out = torch.bmm(v2[e].contiguous(), a[:, :, None].contiguous())[:, :, 0]
        eo = torch.bmm(v2[e].abs().contiguous(), ea[:, :, None].contiguous())[:, :, 0] * 1.01
        eo = eo + (3 * 32 + 3 * 5 + 24) * 2.0 ** -23 * 23 * (a.abs() + ea).sum(1, keepdim=True) / 128 + eps * out.abs() + tiny
        want += weights[:, j:j + 1].double() * out
        near += weights[:, j:j + 1].double() * eo * 1.01
    near = near + 1.01 * eps * (want.abs() + near) + tiny + (k + 1) * 2.0 ** -23 * (want.abs() + near)
    assert ((y.double() - want).abs() <= near).all()

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer()
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        z = layer()[0]
    for i in range(3):
        x.copy_(torch.randn(T, D, generator=g, device="cuda"))
        scores.copy_(torch.randn(T, E, generator=g, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(z, layer()[0])


@pytest.mark.parametrize("M,N,K", [(1, 40, 512), (4, 40, 512), (30, 40, 512), (300, 100, 512), (1000, 4100, 128), (300, 40, 4100)])
@pytest.mark.parametrize("x_type", ["bf16", "fp32"])
def test_rows_that_share_their_memory(mq, x_type, M, N, K):
    """Expanded and overlapping rows: strides of 0, of 8 and of K - 8."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + K)
    w, _, _, values = _weights(mq, g, N, K, 64, "fp16", lambda shape: torch.full(shape, 2.0 ** -6, device="cuda"), True)
    flat = torch.randint(-4, 5, (M * K,), generator=g, device="cuda").to(_dtype(x_type))
    for stride in (0, 8, K - 8):
        x = flat.as_strided((M, K), (stride, 1))
        want = (x.double() @ values.T.contiguous()).float()
        assert torch.equal(mq.w4_linear(x, w, out_dtype=torch.float32), want)


@pytest.mark.parametrize("T", [1, 6, 40, 700])
def test_a_token_with_one_expert_twice(mq, T):
    """Each slot has a row of its own, and the sums go over all of them; gradients too."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(T)
    E, k, D, N = 5, 3, 136, 40
    ids = torch.randint(0, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
    ids[:, 1] = ids[:, 0]
    plan = mq.expert_plan(ids, E)
    x = torch.randint(-4, 5, (T, D), generator=g, device="cuda").float().requires_grad_()
    weights = (torch.randint(1, 5, (T, k), generator=g, device="cuda") / 4.0).requires_grad_()
    rows = mq.experts_gather(x, plan)
    y = mq.experts_combine(rows, plan, weights)
    assert torch.equal(y, x * weights.sum(1, keepdim=True))
    dy = torch.randint(-3, 4, (T, D), generator=g, device="cuda").float()
    dx, dw = torch.autograd.grad(y, (x, weights), dy)
    assert torch.equal(dx, dy * weights.sum(1, keepdim=True))
    assert torch.equal(dw, (dy * x).sum(1, keepdim=True).expand(T, k))
    w, _, _, values = _weights(mq, g, N, D, 64, "fp16", lambda shape: torch.full(shape, 2.0 ** -6, device="cuda"), True, (E,))
    out = mq.experts_combine(mq.w4_experts_linear(x.detach(), w, plan, by_token=True, out_dtype=torch.float32), plan)
    want = sum((values[ids[:, j].long()] * x.detach().double()[:, None, :]).sum(2) for j in range(k))
    assert torch.equal(out, want.float())


def test_rows_past_32_bits(mq):
    """Rows of x spread over 5.2 GB: byte offsets beyond 2^32, for every call that takes strides."""
    import torch
    flat = torch.empty(2_600_000_000, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    K, N, E = 256, 40, 4
    w, _, _, values = _weights(mq, g, N, K, 64, "fp16", lambda shape: torch.full(shape, 2.0 ** -6, device="cuda"), True)
    we, _, _, ve = _weights(mq, g, N, K, 64, "fp16", lambda shape: torch.full(shape, 2.0 ** -6, device="cuda"), True, (E,))
    for M in (3, 4, 30, 300, 1500):
        x = torch.randint(-4, 5, (M, K), generator=g, device="cuda").bfloat16()
        far = flat.as_strided((M, K), ((flat.numel() - K) // (M - 1) // 8 * 8, 1))
        far.copy_(x)
        assert (M - 1) * far.stride(0) * 2 > 2 ** 32
        want = (x.double() @ values.T.contiguous()).float()
        assert torch.equal(mq.w4_linear(far, w, out_dtype=torch.float32), want)
        a, b = mq.w4_quantize(far, group=32, zeros=True), mq.w4_quantize(x, group=32, zeros=True)
        assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales) and torch.equal(a.zeros, b.zeros)
        plan = mq.expert_plan(torch.rand(M, E, generator=g, device="cuda").topk(2, 1).indices.int(), E)
        rows = mq.experts_gather(x, plan)
        assert torch.equal(mq.experts_gather(far, plan), rows)
        near = mq.w4_experts_linear(x, we, plan, by_token=True, out_dtype=torch.float32)
        assert torch.equal(mq.w4_experts_linear(far, we, plan, by_token=True, out_dtype=torch.float32), near)
        assert torch.equal(near, mq.w4_experts_linear(rows, we, plan, out_dtype=torch.float32))
