"""Microscaled 4-bit quantization and products against the 64-bit statements of
tests/mx_reference.py.

Quantized codes and scales are compared bit for bit. Products have two kinds of inputs:
- all scales 1: every partial sum is a multiple of 1/4 below 2^24 / 4, so fp32 holds it
  exactly and the fp32 output must be equal;
- free scales: each of the ceil(K/128) matrix instructions adds four scaled block sums
  to the fp32 accumulator. A block sum is exact; each addition may drop up to 2^-23 of
  the magnitudes added (truncation), and those are at most S = sum |x||w|. A split of K
  over up to 16 waves adds 16 more. So |y - exact| <= (4 ceil(K/128) + 16) 2^-23 S, plus
  half a step of the output's type.
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


def _check_quantized(mq, x):
    """x: device [R, K]; the library's codes, scales and values against the reference."""
    import torch
    a = mq.mx_quantize(x)
    codes, scale = ref.quantize(_np(x))
    pc, ps = ref.pack(codes, scale)
    np.testing.assert_array_equal(a.scales.cpu().numpy(), ps)
    got, want = a.codes.cpu().numpy(), pc
    np.testing.assert_array_equal(got, want)
    v = ref.values(codes, scale)
    for name in ("fp32", "bf16"):
        back = _np(mq.mx_dequantize(a, dtype=_dtype(name)))
        np.testing.assert_array_equal(back, v)
    torch.cuda.synchronize()
    return a


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
@pytest.mark.parametrize("R,K", [(1, 1), (1, 32), (2, 31), (3, 33), (16, 128), (17, 129), (15, 512), (33, 520), (7, 1000),
                                 (70, 2056)])
def test_quantize_matches_the_reference(mq, dtype, R, K):
    import torch
    print(f"[quantize] {R}x{K} {dtype}", flush=True)
    g = torch.Generator().manual_seed(R * 1000 + K)
    x = torch.randn(R, K, generator=g) * torch.exp(2 * torch.randn(R, (K + 31) // 32, generator=g)).repeat_interleave(32, 1)[:, :K]
    _check_quantized(mq, x.to(_dtype(dtype)).cuda())


def test_quantize_ties_and_saturation(mq):
    import torch
    step = torch.arange(0, 8 * 16, dtype=torch.float32) / 16          # every tie and between, peak < 8
    x = torch.zeros(4, 256)
    x[0, :128], x[1, :128] = step, -step
    x[0, 0::32] = x[1, 0::32] = 7.9375                               # blocks of scale 1
    x[2, :128], x[3, :128] = step * 2.0 ** -100, step * 2.0 ** 100
    x[2, 0::32], x[3, 0::32] = 7.9375 * 2.0 ** -100, 7.9375 * 2.0 ** 100
    x[0, 128:160] = -0.0
    _check_quantized(mq, x.cuda())
    _check_quantized(mq, x[:2].bfloat16().cuda())
    _check_quantized(mq, x[:2].half().cuda())


def test_quantize_extremes(mq):
    """Subnormals, the type's largest values, zeros and powers of two; blocks with a NaN or
    an infinity read back as NaN, their neighbours as before."""
    import torch
    x = torch.zeros(6, 160)
    x[0] = 2.0 ** -149 * torch.arange(160)
    x[1] = 2.0 ** -126 * torch.linspace(-2, 2, 160)
    x[2] = 3.4028234e38 * torch.linspace(-1, 1, 160)
    x[3] = 2.0 ** torch.arange(-80, 80).float()
    x[4] = torch.randn(160, generator=torch.Generator().manual_seed(1))
    x[4, 40], x[4, 70], x[4, 100] = float("nan"), float("inf"), -float("inf")
    _check_quantized(mq, x.cuda())
    _check_quantized(mq, x[:5].bfloat16().cuda())
    y = torch.full((2, 64), 65504.0)
    y[1] = 2.0 ** -24 * torch.arange(64)
    _check_quantized(mq, y.half().cuda())


@pytest.mark.parametrize("dtype", ["fp32", "bf16", "fp16"])
def test_quantize_strided_and_batched(mq, dtype):
    import torch
    g = torch.Generator().manual_seed(5)
    wide = torch.randn(40, 333, generator=g).to(_dtype(dtype)).cuda()
    for x in (wide[:, 8:264], wide[:, 3:300], wide[::3, 8:200], wide[:1].expand(5, 333), wide[4:5, :32]):
        _check_quantized(mq, x)
    b = torch.randn(3, 21, 300, generator=g).to(_dtype(dtype)).cuda()
    for x in (b, b[:, 2:19, 4:100], b.transpose(0, 1)):
        a = mq.mx_quantize(x)
        back = mq.mx_dequantize(a)
        for i in range(x.shape[0]):
            one = mq.mx_quantize(x[i])
            assert torch.equal(a.codes[i], one.codes) and torch.equal(a.scales[i], one.scales)
            assert torch.equal(back[i], mq.mx_dequantize(one))


def test_dequantize_rounds_once_to_fp16(mq):
    import torch
    x = torch.tensor([[6.0, 5.0, 2.0 ** -10] + [0.0] * 29, [2.0 ** 17] * 32, [1.5 * 2.0 ** -24] * 32])
    a = mq.mx_quantize(x.cuda())
    want = mq.mx_dequantize(a).cpu().to(torch.float16)
    assert torch.equal(mq.mx_dequantize(a, dtype=torch.float16).cpu(), want)


def _exact_operand(mq, R, K, seed):
    """Codes of every value with scales of 1, as a matrix whose blocks all peak at 4 or 6."""
    import torch
    g = torch.Generator().manual_seed(seed)
    v = torch.tensor(ref.GRID, dtype=torch.float32)[torch.randint(0, 8, (R, K), generator=g)]
    v = v * (2 * torch.randint(0, 2, (R, K), generator=g) - 1)
    v[:, 0::32] = 6.0 - 2.0 * torch.randint(0, 2, (R, (K + 31) // 32), generator=g)
    return v


SHAPES = [(1, 16, 32), (1, 64, 128), (1, 1, 1), (2, 17, 33), (4, 100, 520), (16, 48, 512), (17, 64, 640), (31, 33, 1000),
          (32, 256, 1024), (33, 130, 384), (64, 512, 513), (77, 1001, 1500), (100, 65, 2048), (129, 257, 4096),
          (256, 256, 256), (300, 520, 96), (1, 4096, 4096), (3, 1000, 8192), (513, 300, 1152), (1, 300, 14336)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product_is_exact_where_fp32_is(mq, M, N, K):
    import torch
    print(f"[product] {M}x{N}x{K}", flush=True)
    x, w = _exact_operand(mq, M, K, M + N), _exact_operand(mq, N, K, K + 7)
    want = x.double() @ w.double().t()
    xd = x.cuda()
    wq = mq.mx_quantize(w.cuda())
    xq = mq.mx_quantize(xd)
    assert torch.equal(mq.mx_dequantize(xq).cpu(), x)
    for a in (xq, xd, xd.bfloat16(), xd.half()):
        y = mq.mx_linear(a, wq, out_dtype=torch.float32)
        assert torch.equal(y.cpu().double(), want), (M, N, K)
    bias = torch.randint(-50, 50, (N,), generator=torch.Generator().manual_seed(3)).float()
    y = mq.mx_linear(xd, wq, bias=bias.cuda(), out_dtype=torch.float32)
    assert torch.equal(y.cpu().double(), want + bias.double())


@pytest.mark.parametrize("x_type,y_type", [("bf16", "bf16"), ("fp32", "fp32"), ("fp16", "fp16"), ("bf16", "fp32")])
@pytest.mark.parametrize("M,N,K", [(1, 1000, 1500), (5, 64, 4096), (20, 333, 992), (48, 200, 2000), (77, 1001, 1500),
                                   (200, 300, 5120), (700, 400, 320)])
def test_product_with_free_scales(mq, M, N, K, x_type, y_type):
    import torch
    g = torch.Generator().manual_seed(M * N + K)
    x = torch.randn(M, K, generator=g) * torch.exp(torch.randn(K, generator=g))
    w = torch.randn(N, K, generator=g) * torch.exp(torch.randn(N, 1, generator=g)) / K ** 0.5
    x = x.to(_dtype(x_type)).cuda()
    wq = mq.mx_quantize(w.cuda())
    xv = _np(mq.mx_dequantize(mq.mx_quantize(x)))
    wv = _np(mq.mx_dequantize(wq))
    want, size = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    y = mq.mx_linear(x, wq, out_dtype=_dtype(y_type))
    tol = (4 * -(-K // 128) + 16) * 2.0 ** -23 * size + HALF_STEP[y_type] * np.abs(want) * (1 + 2.0 ** -10)
    if y_type == "fp16":
        tol = tol + 2.0 ** -25
    err = np.abs(_np(y) - want)
    assert (err <= tol).all(), float((err / tol).max())
    # the quantized operand and a repeated call give the same bits
    again = mq.mx_linear(mq.mx_quantize(x), wq, out_dtype=_dtype(y_type))
    assert torch.equal(again, y)


@pytest.mark.parametrize("M", [1, 8, 40, 200])
def test_product_scale_range_and_nan(mq, M):
    """Blocks of very small and very large scales, and one with a NaN: only its own row
    (of x) or column (of w) is NaN."""
    import torch
    N, K = 70, 300
    x, w = _exact_operand(mq, M, K, 1), _exact_operand(mq, N, K, 2)
    x[:, 32:64] *= 2.0 ** -60
    w[:, 32:64] *= 2.0 ** 62
    x[M // 2, 70] = float("inf")
    w[9, 290] = float("nan")
    y = mq.mx_linear(x.cuda(), mq.mx_quantize(w.cuda()), out_dtype=torch.float32).cpu()
    bad = torch.zeros(M, N, dtype=torch.bool)
    bad[M // 2], bad[:, 9] = True, True
    assert torch.equal(torch.isnan(y), bad)
    want = x.double() @ w.double().t()
    assert torch.equal(y[~bad].double(), want[~bad])


@pytest.mark.parametrize("M", [0, 1, 5, 70])
def test_product_strides_and_outputs(mq, M):
    """Rows of a wider matrix, a caller's output, no tokens at all; bytes around an output
    stay as they are."""
    import torch
    N, K = 200, 264
    big = _exact_operand(mq, max(M, 1), 400, 3).cuda()
    x = big[:M, 72:72 + K]
    w = _exact_operand(mq, N, K, 4)
    wq = mq.mx_quantize(w.cuda())
    buf = torch.full((M * N + 64,), 7.0, device="cuda")
    y = buf[32:32 + M * N].view(M, N)
    out = mq.mx_linear(x, wq, y=y)
    assert out.data_ptr() == y.data_ptr() or M == 0
    want = mq.mx_dequantize(mq.mx_quantize(x)).double().cpu() @ w.double().t() if M else torch.zeros(0, N).double()
    assert torch.allclose(y.cpu().double(), want, rtol=2.0 ** -20, atol=0)
    assert (buf[:32] == 7).all() and (buf[32 + M * N:] == 7).all()


def test_calls_on_another_stream_and_in_a_graph(mq):
    """A captured chain replays with new inputs, eager work between; a side stream gives
    the same bits."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(9)
    w = mq.mx_quantize(torch.randn(512, 1024, generator=g, device="cuda"))
    for M in (1, 16, 50, 300):
        x = torch.randn(M, 1024, generator=g, device="cuda", dtype=torch.bfloat16)
        y = torch.empty(M, 512, device="cuda")
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        other = mq.mx_linear(x, w, out_dtype=torch.float32, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(other, mq.mx_linear(x, w, out_dtype=torch.float32))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            mq.mx_linear(x, w, y=y)
        for i in range(4):
            x.copy_(torch.randn(M, 1024, generator=g, device="cuda"))
            graph.replay()
            eager = mq.mx_linear(x, w, out_dtype=torch.float32)
            torch.cuda.synchronize()
            assert torch.equal(y, eager), (M, i)
