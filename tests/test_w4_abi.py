"""Host-only checks of the group-scaled and the tokens-to-rows calls: arguments the library
refuses before any launch, the sizes it states, and what the binding refuses. No GPU needed."""
import pytest


@pytest.fixture(scope="module")
def mq():
    import dense_sparse_bit_amd
    return dense_sparse_bit_amd


FAKE = 0x10000   # never dereferenced: every call below fails its checks first


@pytest.fixture(scope="module")
def lib(mq):
    import torch
    if torch.cuda.is_available():
        pytest.skip("host-only argument checks run where no GPU is visible")
    return mq.lib()


QUANTIZE = dict(x=FAKE, dtype=1, B=2, stride_b=4096, R=4, stride_r=512, K=512, group=64, scale_dtype=2, codes=FAKE, scales=FAKE,
                zeros=FAKE, stream=None)
PACK = dict(c=FAKE, B=2, stride_b=4096, R=4, stride_r=512, K=512, group=64, s=FAKE, z=FAKE, codes=FAKE, scales=FAKE, zeros=FAKE,
            stream=None)
DEQUANTIZE = dict(codes=FAKE, scales=FAKE, zeros=None, scale_dtype=1, B=2, R=4, K=512, group=32, y=FAKE, dtype=0, stream=None)
LINEAR = dict(x=FAKE, x_dtype=1, stride=512, codes=FAKE, scales=FAKE, zeros=FAKE, scale_dtype=2, group=128, M=400, N=64, K=512,
              bias=None, y=FAKE, y_dtype=1, work=FAKE, work_bytes=1 << 40, stream=None)
EXPERTS = dict(x=FAKE, x_dtype=1, stride=512, by_token=1, T=400, k=8, E=64, N=64, K=512, offsets=FAKE, row_token=FAKE, codes=FAKE,
               scales=FAKE, zeros=None, scale_dtype=2, group=128, y=FAKE, y_dtype=1, work=FAKE, work_bytes=1 << 40, stream=None)
GATHER = dict(x=FAKE, x_dtype=1, stride=512, T=40, k=8, E=64, D=512, row_token=FAKE, row_of=FAKE, weights=FAKE, rows=FAKE, rows_dtype=1,
              other=FAKE, dots=FAKE, stream=None)
COMBINE = dict(rows=FAKE, rows_dtype=1, T=40, k=8, E=64, D=512, row_of=FAKE, weights=None, x=FAKE, x_dtype=0, other=None, stride_o=0,
               dots=None, stream=None)

WEIGHTS = [(dict(codes=None), -1), (dict(codes=FAKE + 8), -1), (dict(scales=None), -1), (dict(scales=FAKE + 8), -1),
           (dict(zeros=FAKE + 2), -1), (dict(group=0), -1), (dict(group=16), -1), (dict(group=96), -1), (dict(group=256), -1),
           (dict(K=0), -1), (dict(K=-1), -1), (dict(K=(1 << 20) + 1), -2)]
TYPES = [(dict(scale_dtype=0), -1), (dict(scale_dtype=3), -1)]
MATRIX = WEIGHTS + [(dict(B=-1), -1), (dict(R=-1), -1), (dict(B=65536), -2), (dict(R=(1 << 24) + 1), -2), (dict(R=1 << 24, K=1 << 20), -2),
                    (dict(B=1 << 62, R=1 << 62), -2)]
CASES = [
    ("mq_w4_quantize", QUANTIZE, MATRIX + TYPES + [
        (dict(x=None), -1), (dict(x=FAKE + 1), -1), (dict(dtype=0, x=FAKE + 2), -1), (dict(dtype=3), -1), (dict(dtype=-1), -1),
        (dict(stride_b=-1), -1), (dict(stride_r=-1), -1), (dict(B=0, x=None, codes=None), 0), (dict(R=0, x=None, codes=None), 0)]),
    ("mq_w4_pack", PACK, MATRIX + [
        (dict(c=None), -1), (dict(s=None), -1), (dict(s=FAKE + 1), -1), (dict(z=FAKE + 1), -1), (dict(z=None), -1), (dict(zeros=None), -1),
        (dict(stride_b=-1), -1), (dict(stride_r=-1), -1), (dict(B=0, c=None), 0), (dict(R=0, c=None), 0)]),
    ("mq_w4_dequantize", DEQUANTIZE, MATRIX + TYPES + [
        (dict(y=None), -1), (dict(y=FAKE + 4), -1), (dict(dtype=3), -1), (dict(R=0, y=None), 0)]),
    ("mq_w4_linear", LINEAR, WEIGHTS + TYPES + [
        (dict(x=None), -1), (dict(x=FAKE + 1), -1), (dict(x_dtype=3), -1), (dict(y_dtype=-1), -1), (dict(stride=-1), -1), (dict(y=None), -1),
        (dict(y=FAKE + 8), -1), (dict(bias=FAKE + 2), -1), (dict(M=-1), -1), (dict(N=0), -1), (dict(M=(1 << 24) + 1), -2),
        (dict(N=(1 << 24) + 1), -2), (dict(M=1 << 24, N=1 << 24), -2), (dict(N=1 << 24, K=1 << 20), -2), (dict(M=0, x=None, y=None), 0)]),
    ("mq_w4_experts", EXPERTS, WEIGHTS + TYPES + [
        (dict(x=None), -1), (dict(x=FAKE + 1), -1), (dict(x_dtype=3), -1), (dict(y_dtype=3), -1), (dict(stride=-1), -1), (dict(y=None), -1),
        (dict(y=FAKE + 4), -1), (dict(offsets=None), -1), (dict(offsets=FAKE + 2), -1), (dict(row_token=None), -1),
        (dict(row_token=FAKE + 1), -1), (dict(T=-1), -1), (dict(k=0), -1), (dict(E=0), -1), (dict(N=0), -1), (dict(E=1025), -2),
        (dict(T=1 << 25), -2), (dict(T=0, x=None, y=None, offsets=None), 0)]),
    ("mq_experts_gather", GATHER, [
        (dict(x=None), -1), (dict(x=FAKE + 1), -1), (dict(x_dtype=3), -1), (dict(rows_dtype=3), -1), (dict(stride=-1), -1),
        (dict(rows=None), -1), (dict(rows=FAKE + 8), -1), (dict(row_token=None), -1), (dict(row_of=None), -1), (dict(row_of=FAKE + 2), -1),
        (dict(weights=FAKE + 2), -1), (dict(other=None), -1), (dict(dots=None), -1), (dict(other=FAKE + 1), -1), (dict(dots=FAKE + 2), -1),
        (dict(T=-1), -1), (dict(k=0), -1), (dict(E=-1), -1), (dict(D=0), -1), (dict(D=(1 << 20) + 1), -2), (dict(E=1025), -2),
        (dict(T=1 << 25), -2), (dict(T=0, x=None, rows=None, row_of=None), 0)]),
    ("mq_experts_combine", COMBINE, [
        (dict(rows=None), -1), (dict(rows=FAKE + 1), -1), (dict(rows_dtype=9), -1), (dict(x_dtype=9), -1), (dict(x=None), -1),
        (dict(x=FAKE + 8), -1), (dict(row_of=None), -1), (dict(weights=FAKE + 1), -1), (dict(other=FAKE), -1), (dict(dots=FAKE), -1),
        (dict(other=FAKE + 2, dots=FAKE), -1), (dict(stride_o=-1), -1), (dict(T=-1), -1), (dict(k=-1), -1), (dict(E=0), -1),
        (dict(D=-1), -1), (dict(D=(1 << 20) + 1), -2), (dict(E=1025), -2), (dict(T=1 << 25), -2), (dict(T=0, rows=None, x=None), 0)]),
]


@pytest.mark.parametrize("call,base,kw,status", [(call, base, kw, status) for call, base, all_ in CASES for kw, status in all_])
def test_refused_before_any_launch(lib, call, base, kw, status):
    assert set(kw) <= set(base)
    assert getattr(lib, call)(*{**base, **kw}.values()) == status


def test_a_missing_workspace_is_refused(lib):
    """Where a call says that it takes one; a call that is refused takes none."""
    for M in (1, 16, 40, 400, 4000):
        need = lib.mq_w4_linear_workspace_bytes(M, 64, 512, 1, 128)
        if need:
            for kw in (dict(work=None), dict(work=FAKE + 8), dict(work_bytes=need - 1)):
                assert lib.mq_w4_linear(*{**LINEAR, "M": M, **kw}.values()) == -1
    for T in (1, 16, 40, 400, 4000):
        for by_token in (0, 1):
            need = lib.mq_w4_experts_workspace_bytes(T, 8, 64, 64, 512, by_token, 1, 128)
            if need:
                for kw in (dict(work=None), dict(work=FAKE + 8), dict(work_bytes=need - 1)):
                    assert lib.mq_w4_experts(*{**EXPERTS, "T": T, "by_token": by_token, **kw}.values()) == -1
    for size in ((-1, 64, 512, 1, 128), (4, 0, 512, 1, 128), (4, 64, 512, 1, 48), (4, 64, 1 << 21, 1, 128), (4, 64, 512, 7, 128)):
        assert lib.mq_w4_linear_workspace_bytes(*size) == 0
    for size in ((4, 0, 8, 64, 512, 0, 1, 128), (4, 2, 2000, 64, 512, 0, 1, 128), (4, 2, 8, 64, 512, 0, 1, 48)):
        assert lib.mq_w4_experts_workspace_bytes(*size) == 0


def test_ways_of_products(lib):
    import tests.w4_reference as ref
    for x_type, group, M, N, K, way in ref.WAYS:
        assert lib.mq_w4_linear_way(M, N, K, {"fp32": 0, "bf16": 1, "fp16": 2}[x_type], group) == way
    assert {way for *_, way in ref.WAYS} == {0, 1, 2, 4, 5} | {8 * p + t for p in (1, 2, 4, 8) for t in range(5)}
    for size, status in (((-1, 64, 512, 1, 128), -1), ((4, 0, 512, 1, 128), -1), ((4, 64, 512, 1, 48), -1), ((4, 64, 512, 7, 128), -1),
                         ((4, 64, 1 << 21, 1, 128), -2)):
        assert lib.mq_w4_linear_way(*size) == status


def test_stated_sizes(lib):
    for R, K, group in ((1, 1, 32), (16, 128, 128), (17, 129, 64), (100, 5000, 32)):
        RT, G, Q = -(-R // 16), -(-K // 128), -(-K // 512)
        assert lib.mq_w4_codes_bytes(R, K) == RT * G * 1024
        assert lib.mq_w4_scales_bytes(R, K, group) == RT * Q * 16 * (512 // group) * 2
    assert lib.mq_w4_codes_bytes(4, 0) == 0 and lib.mq_w4_scales_bytes(4, 8, 48) == 0 and lib.mq_w4_codes_bytes(1 << 25, 8) == 0


def _cpu_w4(mq, N=16, K=128, group=128, zeros=False, batch=None):
    import torch
    from dense_sparse_bit_amd.w4 import _new
    return _new(N, K, group, batch, torch.float16, zeros, "cpu")


def test_binding_refuses(mq):
    import torch
    x, codes, s = torch.zeros(4, 128), torch.zeros(16, 128, dtype=torch.uint8), torch.zeros(16, 1, dtype=torch.float16)
    w = _cpu_w4(mq)
    refused = [
        (TypeError, lambda: mq.w4_quantize(None)), (TypeError, lambda: mq.w4_quantize(x.double())),
        (ValueError, lambda: mq.w4_quantize(x[0])), (ValueError, lambda: mq.w4_quantize(x.t())),
        (ValueError, lambda: mq.w4_quantize(x, group=16)), (ValueError, lambda: mq.w4_quantize(x, group=True)),
        (ValueError, lambda: mq.w4_quantize(x, group=None)), (TypeError, lambda: mq.w4_quantize(x, scale_dtype=torch.float32)),
        (ValueError, lambda: mq.w4_quantize(x[:, :0])), (ValueError, lambda: mq.w4_quantize(x)),
        (TypeError, lambda: mq.w4_pack(x, s)), (TypeError, lambda: mq.w4_pack(codes[0], s)), (ValueError, lambda: mq.w4_pack(codes.t(), s)),
        (TypeError, lambda: mq.w4_pack(codes, None)), (TypeError, lambda: mq.w4_pack(codes, s.float())),
        (ValueError, lambda: mq.w4_pack(codes, s, group=100)), (ValueError, lambda: mq.w4_pack(codes, s)),
        (TypeError, lambda: mq.w4_dequantize(codes)), (TypeError, lambda: mq.w4_dequantize(tuple.__new__(mq.W4, (codes,)))),
        (ValueError, lambda: mq.w4_dequantize(w)),
        (TypeError, lambda: mq.w4_linear(x.int(), w)), (ValueError, lambda: mq.w4_linear(x, w)), (ValueError, lambda: mq.w4_linear(x[0], w)),
        (ValueError, lambda: mq.w4_linear(x.clone().requires_grad_(), w)),
        (ValueError, lambda: mq.w4_linear(x, w, bias=torch.zeros(16, requires_grad=True))),
        (ValueError, lambda: mq.w4_experts_linear(x.clone().requires_grad_(), w, None)), (ValueError, lambda: mq.w4_experts_linear(x, w, None)),
        (TypeError, lambda: mq.experts_gather(None, None)), (TypeError, lambda: mq.experts_gather(x.int(), None)),
        (ValueError, lambda: mq.experts_gather(x, None)), (ValueError, lambda: mq.experts_gather(x[0], None)),
        (ValueError, lambda: mq.experts_gather(x.clone().requires_grad_(), None, rows=x)),
        (TypeError, lambda: mq.experts_combine(None, None)), (ValueError, lambda: mq.experts_combine(x, None)),
        (ValueError, lambda: mq.experts_combine(x.clone().requires_grad_(), None, y=x)),
    ]
    for error, call in refused:
        with pytest.raises(error):
            call()
    # a matrix whose tensors do not have its sizes, with the check that the device calls make
    from dense_sparse_bit_amd.w4 import _w4
    _w4(_cpu_w4(mq, zeros=True), "w", -1)
    _w4(_cpu_w4(mq, batch=3), "w", -1, 3)
    for bad in (w._replace(rows=17), w._replace(cols=129), w._replace(group=64), w._replace(group=5), w._replace(codes=w.codes[:, :, :512]),
                w._replace(zeros=w.scales[:, :, :8]), w._replace(scales=w.scales.transpose(2, 3))):
        with pytest.raises(ValueError):
            _w4(bad, "w", -1)
    for bad in (w._replace(scales=w.scales.float()), w._replace(zeros=w.scales.to(torch.bfloat16)), w._replace(scales=None),
                w._replace(codes=w.codes.char()), None, tuple(w)):
        with pytest.raises(TypeError):
            _w4(bad, "w", -1)
    with pytest.raises(ValueError):
        _w4(_cpu_w4(mq, batch=3), "w", -1, 4)


@pytest.mark.gpu
def test_binding_refuses_on_the_device(mq):
    """Sizes, types and plans that do not fit, without a launch; the same from the long way."""
    import torch
    dev = "cuda"
    x, s = torch.zeros(4, 128, device=dev), torch.zeros(16, 1, device=dev, dtype=torch.float16)
    codes = torch.zeros(16, 128, device=dev, dtype=torch.uint8)
    w = mq.w4_pack(codes, s)
    we = mq.w4_pack(codes.expand(2, 16, 128), s.expand(2, 16, 1).contiguous())
    plan = mq.expert_plan(torch.zeros(4, 2, device=dev, dtype=torch.int32), 2)
    P = plan.row_token.numel()
    rows, weights = torch.zeros(P, 128, device=dev), torch.zeros(4, 2, device=dev)
    other = torch.zeros(5, 2, device=dev)
    refused = [
        (ValueError, lambda: mq.w4_pack(codes, s[:8])), (TypeError, lambda: mq.w4_pack(codes, s, s.to(torch.bfloat16))),
        (ValueError, lambda: mq.w4_pack(codes, s, group=64)), (ValueError, lambda: mq.w4_pack(codes, s.cpu())),
        (ValueError, lambda: mq.w4_quantize(x, out=w)), (TypeError, lambda: mq.w4_quantize(x, out=x)),
        (ValueError, lambda: mq.w4_quantize(torch.zeros(16, 128, device=dev), zeros=True, out=w)),
        (ValueError, lambda: mq.w4_linear(x[:, :100], w)), (ValueError, lambda: mq.w4_linear(x, we)), (TypeError, lambda: mq.w4_linear(x, codes)),
        (ValueError, lambda: mq.w4_linear(x, w, bias=torch.zeros(15, device=dev))),
        (TypeError, lambda: mq.w4_linear(x, w, bias=torch.zeros(16, device=dev, dtype=torch.float16))),
        (ValueError, lambda: mq.w4_linear(x, w, y=torch.zeros(4, 17, device=dev))), (TypeError, lambda: mq.w4_linear(x, w, out_dtype=torch.int32)),
        (ValueError, lambda: mq.w4_linear(x, w, y=torch.zeros(65, device=dev)[1:].reshape(4, 16))),
        (ValueError, lambda: mq.w4_linear(x, w._replace(codes=w.codes.cpu()))), (TypeError, lambda: mq.w4_experts_linear(rows, we, None)),
        (ValueError, lambda: mq.w4_experts_linear(x, we, plan)), (ValueError, lambda: mq.w4_experts_linear(rows, we, plan, by_token=True)),
        (ValueError, lambda: mq.w4_experts_linear(rows, w, plan)), (TypeError, lambda: mq.experts_gather(x, tuple(plan))),
        (ValueError, lambda: mq.experts_gather(x[:3], plan)), (ValueError, lambda: mq.experts_gather(x, plan, other)),
        (TypeError, lambda: mq.experts_gather(x, plan, weights.half())), (ValueError, lambda: mq.experts_gather(x[:, :0], plan)),
        (ValueError, lambda: mq.experts_gather(x, plan, rows=rows[:, :64])), (ValueError, lambda: mq.experts_gather(x, plan, weights.cpu())),
        (ValueError, lambda: mq.experts_gather(x, plan, weights.requires_grad_(), rows=rows)),
        (ValueError, lambda: mq.experts_combine(x, plan)), (ValueError, lambda: mq.experts_combine(rows, plan, other)),
        (ValueError, lambda: mq.experts_combine(rows.t().contiguous().t(), plan)),
        (ValueError, lambda: mq.experts_combine(rows, plan, y=torch.zeros(4, 100, device=dev))),
        (TypeError, lambda: mq.experts_combine(rows, plan, out_dtype=torch.float64)),
        (ValueError, lambda: mq.experts_combine(rows, mq.ExpertPlan(plan.offsets, plan.row_token[:16], plan.row_of))),
    ]
    for error, call in refused:
        with pytest.raises(error):
            call()
    torch.cuda.synchronize()
