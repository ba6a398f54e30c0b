"""Every way of the microscaled product, at sizes that take it: a host test asks the library
which way each size takes, so that another choice of ways cannot leave one without tests.

Inputs and tolerances are those of tests/test_mx.py: exact products with scales of 1; with
free scales (4 ceil(K/128) + 16) 2^-23 of the sum of magnitudes and half a step of the
output's type. A bias is one more term and one more addition.
"""
import pytest

from tests.test_mx import HALF_STEP, _dtype, _exact_operand

# mq_mx_gemm_way -> sizes (M, N, K). N odd, or a multiple of 8 (whole 16-byte stores); M ends
# inside a 16-row tile; K ends inside a group of 128. The row blocks (4 to 7) go through the
# groups four at a time, so K leaves 0 to 3 of them over; one group alone too.
WAYS = {
    0: [(19, 17, 532), (19, 16, 542), (77, 1001, 1500)],
    1: [(19, 7515, 513), (50, 3744, 692), (20, 7649, 1226)],
    2: [(19, 7890, 524), (19, 7680, 546), (49, 4169, 1255)],
    3: [(35, 9372, 1933), (35, 9373, 1933), (65, 6224, 1672), (136, 3719, 1771)],
    4: [(35, 7163, 914), (35, 7600, 921), (34, 6701, 532), (35, 6864, 604), (33, 6861, 701), (33, 6952, 671), (35, 6925, 812),
        (33, 9016, 861), (35, 6142, 33)],
    5: [(2436, 1859, 903), (1977, 2336, 1000), (2121, 2092, 520), (1368, 3624, 523), (1732, 2730, 641), (1778, 2592, 645),
        (1234, 3883, 773), (600, 7960, 773), (1708, 2704, 33)],
    6: [(1862, 4619, 905), (1093, 8016, 962), (1722, 5153, 515), (2249, 3920, 533), (1043, 8469, 652), (1939, 4728, 659),
        (1359, 6509, 769), (1798, 4928, 781), (1583, 5678, 32)],
    7: [(1666, 7650, 946), (1750, 7440, 904), (1453, 8449, 525), (1548, 9392, 532), (1558, 8142, 650), (2357, 5464, 680),
        (1955, 6602, 769), (1791, 7536, 797), (1657, 7731, 33)],
}
CASES = [(way, *size) for way, sizes in WAYS.items() for size in sizes]


# Rows quantized on the way, by their number (1; 2 to 4; 5 to 16) and by the columns (over 8192:
# two column tiles a wave); K below 8, odd, and with runs of a wave that end inside four groups
ON_THE_WAY = [(M, N, K) for M in (1, 2, 4, 5, 11, 16) for N, K in ((8192, 520), (8193, 520), (9001, 1031), (9000, 7), (333, 5),
                                                                  (12345, 2049), (70, 8191))]


@pytest.fixture(scope="module")
def mq():
    import dense_sparse_bit_amd
    return dense_sparse_bit_amd


def test_sizes_take_the_ways_they_are_here_for(mq):
    way_of = mq.lib().mq_mx_gemm_way
    for way, *size in CASES:
        assert way_of(*size) == way, size
    for way, sizes in WAYS.items():
        assert any(N % 8 == 0 for _, N, _ in sizes) and any(N % 2 for _, N, _ in sizes), way
        groups = [-(-K // 128) for _, _, K in sizes]
        assert max(groups) > 4
        if way >= 4:
            assert {g % 4 for g in groups if g > 4} == {0, 1, 2, 3} and 1 in groups
    for size in ON_THE_WAY:
        assert mq.lib().mq_mx_linear_workspace_bytes(*size) == 0, size
    # all ways there are: over sizes of any kind no other number comes back
    seen = {way_of(M, N, K) for M in (1, 16, 17, 33, 64, 100, 200, 400, 800, 2000, 5000, 70000)
            for N in (1, 16, 100, 1000, 4096, 8192, 17408, 40000) for K in (1, 128, 1000, 4096, 14336, 100000)}
    assert seen == set(WAYS)
    assert way_of(0, 16, 16) >= 0 and way_of(-1, 16, 16) == -1 and way_of(1, 0, 16) == -1 and way_of(1, 16, 1 << 21) == -2


@pytest.mark.gpu
@pytest.mark.parametrize("way,M,N,K", CASES)
def test_product_is_exact_where_fp32_is(mq, way, M, N, K):
    import torch
    print(f"[way {way}] {M}x{N}x{K}", flush=True)
    x, w = _exact_operand(mq, M, K, M + N).cuda(), _exact_operand(mq, N, K, K + 7).cuda()
    want = x.double() @ w.double().t().contiguous()
    wq, xq = mq.mx_quantize(w), mq.mx_quantize(x)
    bias = torch.randint(-50, 50, (N,), generator=torch.Generator().manual_seed(3)).float().cuda()
    for b, total in ((None, want), (bias, want + bias.double())):
        buf = torch.full((M * N + 128,), 7.0, device="cuda")
        y = buf[64:64 + M * N].view(M, N)
        for a in (xq, x.bfloat16()):
            y.zero_()
            mq.mx_linear(a, wq, bias=b, y=y)
            assert torch.equal(y.double(), total)
        assert (buf[:64] == 7).all() and (buf[64 + M * N:] == 7).all()
        for name in ("bf16", "fp16"):                         # the exact sum, rounded once
            buf = torch.full((M * N + 128,), 7.0, device="cuda", dtype=_dtype(name))
            y = buf[64:64 + M * N].view(M, N)
            mq.mx_linear(xq, wq, bias=b, y=y)
            assert torch.equal(y, total.to(_dtype(name)))
            assert (buf[:64] == 7).all() and (buf[64 + M * N:] == 7).all()


@pytest.mark.gpu
@pytest.mark.parametrize("way,M,N,K", CASES)
def test_product_with_free_scales(mq, way, M, N, K):
    import torch
    print(f"[way {way}] {M}x{N}x{K}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(M * N + K)
    draw = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    x = draw(M, K) * torch.exp(draw(K))
    w, bias = draw(N, K) * torch.exp(draw(N, 1)) / K ** 0.5, draw(N)
    wq = mq.mx_quantize(w)
    wv = mq.mx_dequantize(wq).double().t().contiguous()
    for x_type, y_type, b in (("bf16", "bf16", None), ("fp32", "fp32", bias), ("fp16", "fp16", bias), ("fp32", "bf16", bias)):
        a = x.to(_dtype(x_type))
        xv = mq.mx_dequantize(mq.mx_quantize(a)).double()
        want, size = xv @ wv, xv.abs() @ wv.abs()
        if b is not None:
            want, size = want + b.double(), size + b.double().abs()
        y = mq.mx_linear(a, wq, bias=b, out_dtype=_dtype(y_type))
        tol = (4 * -(-K // 128) + 17) * 2.0 ** -23 * size
        tol += HALF_STEP[y_type] * (want.abs() + tol) + (2.0 ** -25 if y_type == "fp16" else 0)
        err = (y.double() - want).abs()
        assert (err <= tol).all(), (x_type, y_type, float((err / tol).max()))
        # the quantized operand and a repeated call give the same bits
        assert torch.equal(mq.mx_linear(mq.mx_quantize(a), wq, bias=b, out_dtype=_dtype(y_type)), y)


@pytest.mark.gpu
@pytest.mark.parametrize("way,M,N,K", [c for c in CASES if c[3] > 128])
def test_scale_range_and_nan(mq, way, M, N, K):
    """Blocks of very small and very large scales, and ones with a NaN or an infinity: only
    their own rows (of x) and columns (of w) are NaN."""
    import torch
    print(f"[way {way}] {M}x{N}x{K}", flush=True)
    x, w = _exact_operand(mq, M, K, 1).cuda(), _exact_operand(mq, N, K, 2).cuda()
    x[:, 32:64] *= 2.0 ** -60
    w[:, 32:64] *= 2.0 ** 62
    rows, cols = sorted({0, M // 2, M - 1}), sorted({9, N // 2, N - 1})
    x[rows[0], 70], x[rows[1], K - 1], x[rows[2], 130] = float("inf"), float("nan"), -float("inf")
    w[cols[0], K - 1], w[cols[1], 5], w[cols[2], 140] = float("nan"), float("inf"), float("nan")
    want = x.double() @ w.double().t().contiguous()
    bad = torch.zeros(M, N, dtype=torch.bool, device="cuda")
    bad[rows], bad[:, cols] = True, True
    for a in (x, mq.mx_quantize(x)):
        y = mq.mx_linear(a, mq.mx_quantize(w), out_dtype=torch.float32)
        assert torch.equal(torch.isnan(y), bad)
        assert torch.equal(y[~bad].double(), want[~bad])


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", ON_THE_WAY)
def test_rows_quantized_on_the_way(mq, M, N, K):
    import torch
    print(f"[on the way] {M}x{N}x{K}", flush=True)
    x, w = _exact_operand(mq, M, K, M + N).cuda(), _exact_operand(mq, N, K, K + 7).cuda()
    want, wq = x.double() @ w.double().t().contiguous(), mq.mx_quantize(w)
    bias = torch.randint(-50, 50, (N,), generator=torch.Generator().manual_seed(3)).float().cuda()
    wide = torch.zeros(M, K + 11, device="cuda")
    wide[:, 5:5 + K] = x
    for a in (x, x.bfloat16(), x.half(), wide[:, 5:5 + K], wide.bfloat16()[:, 5:5 + K]):
        assert torch.equal(mq.mx_linear(a, wq, out_dtype=torch.float32).double(), want)
        assert torch.equal(mq.mx_linear(a, wq, bias=bias, out_dtype=torch.float32).double(), want + bias.double())
        assert torch.equal(mq.mx_linear(a, wq), mq.mx_linear(mq.mx_quantize(a), wq))
    x[M // 2, K - 1] = float("nan")
    y = mq.mx_linear(x, wq, out_dtype=torch.float32)
    assert torch.isnan(y[M // 2]).all()
    keep = torch.arange(M, device="cuda") != M // 2
    assert torch.equal(y[keep].double(), want[keep])


@pytest.mark.gpu
def test_a_prefill_chunk_of_a_whole_layer(mq):
    """The largest product that a layer of this library's benchmark makes, every output."""
    import torch
    M, N, K = 2048, 17408, 5120
    assert mq.lib().mq_mx_gemm_way(M, N, K) == 7
    x, w = _exact_operand(mq, M, K, 5).cuda(), _exact_operand(mq, N, K, 6).cuda()
    y = mq.mx_linear(x.bfloat16(), mq.mx_quantize(w), out_dtype=torch.float32)
    assert torch.equal(y.double(), x.double() @ w.double().t().contiguous())
