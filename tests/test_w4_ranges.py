"""Products with group-scaled 4-bit weights where scales and rows are far apart: every way gives
the sums that fp32 can hold, however the scales of a row of weights follow each other.

Against float64, with the bound of test_w4_ways.py: A a group's sum of |x|, n groups, S the sum
over groups of |s| (15 + |z|) A; |y - exact| <= (3 group + 3 n + 24) 2^-23 S. All inputs are such
that 15 times a group's A, and S, stay below 2^127, and that sums of products which count are
above 2^-90."""
import pytest

import tests.w4_reference as ref

pytestmark = pytest.mark.gpu

CODE = {"fp32": 0, "bf16": 1, "fp16": 2}


@pytest.fixture(scope="module")
def mq():
    import torch
    assert torch.cuda.is_available()
    import dense_sparse_bit_amd
    return dense_sparse_bit_amd


def _dtype(name):
    import torch
    return {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[name]


def _powers(kind, shape, g):
    """Exponents of the scales of a row, group by group: what a running sum in units of the present
    scale finds hard."""
    import torch
    n = shape[-1]
    at = torch.arange(n, device="cuda")
    fp16 = {"falls": torch.where(at % 2 == 0, 14, -24), "falls once": torch.where(at < (n + 1) // 2, 14, -24),
            "rises": torch.where(at % 2 == 0, -24, 14), "steps": 14 - at * 38 // max(n - 1, 1)}
    bf16 = {"falls": torch.where(at % 2 == 0, 0, -60), "falls once": torch.where(at < (n + 1) // 2, 0, -60),
            "rises": torch.where(at % 2 == 0, -100, 50), "steps": 40 - at * 120 // max(n - 1, 1)}
    return {"fp16": fp16, "bf16": bf16}[kind[0]][kind[1]].expand(shape)


def _weights(mq, g, N, K, group, scales, batch=()):
    import torch
    codes = torch.randint(0, 16, batch + (N, K), generator=g, device="cuda", dtype=torch.uint8)
    z = torch.randint(0, 16, scales.shape, generator=g, device="cuda").to(scales.dtype)
    wide = lambda v: v.double().repeat_interleave(group, -1)[..., :K]
    return mq.w4_pack(codes, scales, z, group=group), z, (codes.double() - wide(z)) * wide(scales)


def _bound(x, s, z, group, K):
    import torch
    n = s.shape[-1]
    a = torch.nn.functional.pad(x.double().abs(), (0, n * group - K)).view(len(x), n, group).sum(2)
    S = a @ (s.double().abs() * (15 + z.double().abs())).T.contiguous()
    assert (15 * a).max() < 2.0 ** 127 and S.max() < 2.0 ** 127
    return (3 * group + 3 * n + 24) * 2.0 ** -23 * S


def _check(got, want, near):
    assert got.isfinite().all()
    assert ((got.double() - want).abs() <= near).all()


@pytest.mark.parametrize("order", ["falls", "falls once", "rises", "steps"])
@pytest.mark.parametrize("x_type,group,M,N,K,way", ref.WAYS)
def test_large_rows_and_scales_in_every_order(mq, x_type, group, M, N, K, way, order):
    """Rows of about 2^60 (fp16: 2^10) times scales 2^38 apart (fp16) or 2^60 to 2^150 (bf16): sums in
    units of a small scale leave fp32's range, where their values do not."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + 3 * N + K)
    assert mq.lib().mq_w4_linear_way(M, N, K, CODE[x_type], group) == way
    for kind, size in (("fp16", 80), ("bf16", 60)):
        shape = (N, -(-K // group))
        s = torch.ldexp(1 + torch.rand(shape, generator=g, device="cuda") / 2, _powers((kind, order), shape, g).float()).to(_dtype(kind))
        s = torch.where(torch.rand(shape, generator=g, device="cuda") < 0.5, s, -s)
        w, z, values = _weights(mq, g, N, K, group, s)
        if order == "rises" and kind == "bf16":
            size = 20
        x = torch.ldexp(torch.randn(M, K, generator=g, device="cuda"), torch.tensor(10.0 if x_type == "fp16" else size, device="cuda"))
        x = x.to(_dtype(x_type))
        want = x.double() @ values.T.contiguous()
        _check(mq.w4_linear(x, w, out_dtype=torch.float32), want, _bound(x, s, z, group, K))


@pytest.mark.parametrize("x_type,group,M,N,K,way", ref.WAYS)
def test_a_large_scale_whose_rows_are_zero_takes_nothing_away(mq, x_type, group, M, N, K, way):
    """Scales of 2^-100 and, in every second group, 2^50, where x is zero: the sums before are not
    lost in units of the large one."""
    import torch
    if K <= group:
        pytest.skip("one group")
    g = torch.Generator(device="cuda").manual_seed(M + 5 * N + K)
    shape = (N, -(-K // group))
    at = torch.arange(shape[1], device="cuda")
    s = torch.ldexp(1 + torch.rand(shape, generator=g, device="cuda") / 2, torch.where(at % 2 == 0, -100, 50).float()).bfloat16()
    w, z, values = _weights(mq, g, N, K, group, s)
    x = torch.randn(M, K, generator=g, device="cuda") * (torch.arange(K, device="cuda") // group % 2 == 0)
    x = torch.ldexp(x, torch.tensor(12.0, device="cuda")).to(_dtype(x_type))
    want = x.double() @ values.T.contiguous()
    assert want.abs().max() > 0
    _check(mq.w4_linear(x, w, out_dtype=torch.float32), want, _bound(x, s, z, group, K))


@pytest.mark.parametrize("x_type,group,M,N,K,way", ref.WAYS)
def test_scales_next_to_the_ends_of_their_type(mq, x_type, group, M, N, K, way):
    """Scales below 2^-126 and above 2^126, whose reciprocals leave fp32's normal numbers, with rows
    that keep the products in it; some columns have ordinary scales among them."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + 7 * N + K)
    shape = (N, -(-K // group))
    small = torch.randint(0, 2, shape, generator=g, device="cuda", dtype=torch.bool)
    for power, size in ((-130, 14), (126.5, -12)):
        s = torch.ldexp(torch.ones(shape, device="cuda"), torch.tensor(float(int(power)), device="cuda"))
        if power > 0:
            s = s * 1.5
        else:
            s = torch.where(small, s, torch.ldexp(s, torch.tensor(40.0, device="cuda")))
        s[::3] = 1 / 64
        s = s.bfloat16()
        w, z, values = _weights(mq, g, N, K, group, s)
        x = torch.ldexp(torch.rand(M, K, generator=g, device="cuda"), torch.tensor(float(size), device="cuda"))
        x = torch.where(torch.arange(K, device="cuda") % max(K // 8, 1) == 0, x, torch.zeros_like(x)).to(_dtype(x_type))
        want = x.double() @ values.T.contiguous()
        # outputs below 2^-126 are subnormal: half of 2^-149 for each addition
        _check(mq.w4_linear(x, w, out_dtype=torch.float32), want, _bound(x, s, z, group, K) + 2.0 ** -149 * (shape[1] + 24))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("x_type", ["bf16", "fp32"])
@pytest.mark.parametrize("T,E,k,N,K", [(1, 4, 2, 40, 520), (20, 8, 2, 100, 520), (70, 4, 2, 300, 520), (400, 4, 2, 300, 264), (2000, 8, 4, 530, 512)])
def test_experts_with_large_rows_and_falling_scales(mq, x_type, group, T, E, k, N, K):
    import torch
    g = torch.Generator(device="cuda").manual_seed(T + N)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.int()
    ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.1, -1, ids).int().contiguous()
    plan = mq.expert_plan(ids, E)
    shape = (E, N, -(-K // group))
    s = torch.ldexp(1 + torch.rand(shape, generator=g, device="cuda") / 2, _powers(("bf16", "falls"), shape, g).float()).bfloat16()
    w, z, values = _weights(mq, g, N, K, group, s, (E,))
    x = torch.ldexp(torch.randn(T, K, generator=g, device="cuda"), torch.tensor(60.0, device="cuda")).to(_dtype(x_type))
    got = mq.w4_experts_linear(x, w, plan, by_token=True, out_dtype=torch.float32)
    token, offsets = plan.row_token.long(), plan.offsets.tolist()
    real = token >= 0
    assert not got[~real].any()
    for e in range(E):
        at = torch.arange(offsets[e], offsets[e + 1], device="cuda")
        at = at[real[at]]
        if len(at):
            rows = x[token[at]]
            _check(got[at], rows.double() @ values[e].T.contiguous(), _bound(rows, s[e], z[e], group, K))


def test_rows_that_do_not_count_change_nothing(mq):
    """Rows of no token that hold NaN or infinities, between rows whose columns are computed again."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(0)
    T, E, k, N, K, group = 300, 3, 2, 130, 512, 128
    plan = mq.expert_plan(torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.int(), E)
    shape = (E, N, K // group)
    for order, size in (("falls", 60), ("rises", 20)):
        s = torch.ldexp(torch.ones(shape, device="cuda"), _powers(("bf16", order), shape, g).float()).bfloat16()
        w, z, values = _weights(mq, g, N, K, group, s, (E,))
        x = torch.ldexp(torch.randn(T, K, generator=g, device="cuda"), torch.tensor(float(size), device="cuda")).bfloat16()
        rows = mq.experts_gather(x, plan)
        want = mq.w4_experts_linear(rows, w, plan, out_dtype=torch.float32)
        assert want.isfinite().all()
        for bad in (float("nan"), float("inf")):
            rows[plan.row_token < 0] = bad
            assert torch.equal(mq.w4_experts_linear(rows, w, plan, out_dtype=torch.float32), want)
