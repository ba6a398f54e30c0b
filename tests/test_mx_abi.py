"""Host-only checks of the microscaled and routing calls: arguments the library refuses
before any launch, the sizes it states, and what the binding refuses. No GPU needed."""
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


def _with(base, kw):
    a = dict(base)
    for k in kw:
        assert k in a
    a.update(kw)
    return list(a.values())


QUANTIZE = dict(x=FAKE, dtype=1, B=2, stride_b=4096, R=4, stride_r=512, K=512, codes=FAKE, scales=FAKE, stream=None)
DEQUANTIZE = dict(codes=FAKE, scales=FAKE, B=2, R=4, K=512, y=FAKE, dtype=0, stream=None)
GEMM = dict(xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, M=4, N=64, K=512, bias=None, y=FAKE, dtype=1, stream=None)
LINEAR = dict(x=FAKE, x_dtype=1, stride=512, wq=FAKE, ws=FAKE, M=400, N=64, K=512, bias=None, y=FAKE, y_dtype=1,
              work=FAKE, work_bytes=1 << 30, stream=None)
ROUTE = dict(logits=FAKE, dtype=0, T=4, stride=64, E=64, bias=None, score=0, groups=4, top_groups=2, group_score=0, k=8,
             renorm=1, scale=1.0, ids=FAKE, weights=FAKE, stream=None)
PLAN = dict(ids=FAKE, T=4, k=8, E=64, offsets=FAKE, row_token=FAKE, row_of=FAKE, stream=None)
UP = dict(x=FAKE, x_dtype=1, stride=512, T=400, k=8, E=64, D=512, I=128, offsets=FAKE, row_token=FAKE, row_of=FAKE, gq=FAKE,
          gs=FAKE, uq=FAKE, us=FAKE, h=FAKE, h_dtype=1, work=FAKE, work_bytes=1 << 40, stream=None)
DOWN = dict(h=FAKE, h_dtype=1, T=400, k=8, E=64, D=512, I=128, offsets=FAKE, row_of=FAKE, weights=FAKE, wq=FAKE, ws=FAKE,
            y=FAKE, y_dtype=1, work=FAKE, work_bytes=1 << 40, stream=None)


@pytest.mark.parametrize("call,base,kw,status", [
    ("mq_mx_quantize", QUANTIZE, k, s) for k, s in [
        (dict(x=None), -1), (dict(dtype=3), -1), (dict(dtype=-1), -1), (dict(B=-1), -1), (dict(R=-1), -1), (dict(K=0), -1),
        (dict(K=-4), -1), (dict(stride_b=-1), -1), (dict(stride_r=-512), -1), (dict(x=FAKE + 1), -1),
        (dict(dtype=0, x=FAKE + 2), -1), (dict(codes=None), -1), (dict(scales=None), -1), (dict(codes=FAKE + 8), -1),
        (dict(scales=FAKE + 2), -1), (dict(K=(1 << 20) + 1), -2), (dict(R=(1 << 24) + 1), -2), (dict(B=65536), -2),
        (dict(B=1 << 62, R=1 << 62), -2), (dict(R=1 << 24, K=1 << 20), -2), (dict(B=0, x=None, codes=None), 0),
        (dict(R=0, x=None, codes=None), 0)]
] + [
    ("mq_mx_dequantize", DEQUANTIZE, k, s) for k, s in [
        (dict(codes=None), -1), (dict(scales=None), -1), (dict(y=None), -1), (dict(y=FAKE + 4), -1), (dict(dtype=4), -1),
        (dict(K=0), -1), (dict(R=-2), -1), (dict(K=1 << 30), -2), (dict(R=0, y=None), 0)]
] + [
    ("mq_mx_gemm", GEMM, k, s) for k, s in [
        (dict(xq=None), -1), (dict(xs=None), -1), (dict(wq=None), -1), (dict(ws=None), -1), (dict(y=None), -1),
        (dict(y=FAKE + 8), -1), (dict(xq=FAKE + 8), -1), (dict(ws=FAKE + 1), -1), (dict(bias=FAKE + 2), -1),
        (dict(dtype=9), -1), (dict(M=-1), -1), (dict(N=0), -1), (dict(K=0), -1), (dict(M=1 << 40), -2),
        (dict(N=1 << 25), -2), (dict(N=1 << 24, K=1 << 20), -2), (dict(M=0, xq=None, y=None), 0)]
] + [
    ("mq_mx_linear", LINEAR, k, s) for k, s in [
        (dict(x=None), -1), (dict(x=FAKE + 1), -1), (dict(x_dtype=5), -1), (dict(y_dtype=5), -1), (dict(stride=-1), -1),
        (dict(wq=None), -1), (dict(ws=None), -1), (dict(y=None), -1), (dict(work=None), -1), (dict(work=FAKE + 8), -1),
        (dict(work_bytes=100), -1), (dict(bias=FAKE + 1), -1), (dict(K=-1), -1), (dict(K=1 << 21), -2),
        (dict(M=0, x=None, work=None, work_bytes=0), 0)]
] + [
    ("mq_route", ROUTE, k, s) for k, s in [
        (dict(logits=None), -1), (dict(logits=FAKE + 2), -1), (dict(dtype=7), -1), (dict(T=-1), -1), (dict(stride=-1), -1),
        (dict(E=0), -1), (dict(E=-64), -1), (dict(bias=FAKE + 1), -1), (dict(score=2), -1), (dict(group_score=-1), -1),
        (dict(groups=0), -1), (dict(groups=5), -1), (dict(top_groups=0), -1), (dict(top_groups=5), -1), (dict(k=0), -1),
        (dict(k=33), -1), (dict(E=1024, groups=1, top_groups=1, k=33), -2), (dict(E=1025, groups=1, top_groups=1), -2),
        (dict(E=128, groups=128, top_groups=64), -2), (dict(ids=None), -1), (dict(weights=None), -1), (dict(ids=FAKE + 2), -1),
        (dict(T=1 << 40), -2), (dict(T=0, logits=None, ids=None, weights=None), 0)]
] + [
    ("mq_expert_plan", PLAN, k, s) for k, s in [
        (dict(ids=None), -1), (dict(T=-1), -1), (dict(k=0), -1), (dict(E=0), -1), (dict(E=1025), -2), (dict(T=1 << 25), -2),
        (dict(offsets=None), -1), (dict(row_token=None), -1), (dict(row_of=None), -1), (dict(offsets=FAKE + 2), -1),
        (dict(row_of=FAKE + 1), -1)]
] + [
    ("mq_mx_experts_up", UP, k, s) for k, s in [
        (dict(x=None), -1), (dict(x=FAKE + 1), -1), (dict(x_dtype=3), -1), (dict(h_dtype=3), -1), (dict(stride=-8), -1),
        (dict(T=-1), -1), (dict(k=0), -1), (dict(E=0), -1), (dict(D=0), -1), (dict(I=0), -1), (dict(I=-1), -1),
        (dict(E=2000), -2), (dict(D=1 << 21), -2), (dict(offsets=None), -1), (dict(row_token=None), -1),
        (dict(row_of=None), -1), (dict(gq=None), -1), (dict(gs=None), -1), (dict(uq=None), -1), (dict(us=FAKE + 1), -1),
        (dict(h=None), -1), (dict(h=FAKE + 2), -1), (dict(work=None), -1), (dict(work_bytes=64), -1),
        (dict(work=FAKE + 4), -1), (dict(T=0, x=None, h=None, work=None), 0)]
] + [
    ("mq_mx_experts_down", DOWN, k, s) for k, s in [
        (dict(h=None), -1), (dict(h_dtype=-1), -1), (dict(y_dtype=3), -1), (dict(T=-1), -1), (dict(k=0), -1), (dict(E=0), -1),
        (dict(D=0), -1), (dict(I=0), -1), (dict(E=2000), -2), (dict(I=1 << 21), -2), (dict(offsets=None), -1),
        (dict(row_of=None), -1), (dict(weights=None), -1), (dict(weights=FAKE + 2), -1), (dict(wq=None), -1),
        (dict(ws=None), -1), (dict(y=None), -1), (dict(y=FAKE + 8), -1), (dict(work=None), -1), (dict(work_bytes=64), -1),
        (dict(T=0, h=None, y=None, work=None), 0)]
])
def test_arguments(lib, call, base, kw, status):
    assert getattr(lib, call)(*_with(base, kw)) == status


def test_sizes(mq):
    lib = mq.lib()
    assert lib.mq_mx_codes_bytes(17, 129) == 2 * 2 * 1024 and lib.mq_mx_scales_bytes(17, 129) == 2 * 256
    assert lib.mq_mx_codes_bytes(16, 640) == 5 * 1024 and lib.mq_mx_scales_bytes(16, 640) == 2 * 256
    assert lib.mq_mx_codes_bytes(0, 128) == 0 and lib.mq_mx_codes_bytes(-1, 128) == 0
    assert lib.mq_plan_rows(1, 8, 64) == 128 and lib.mq_plan_rows(1, 8, 2) == 32
    assert lib.mq_plan_rows(4096, 8, 64) == 32768 + 60 * 16
    assert lib.mq_plan_rows(0, 8, 64) == 0 and lib.mq_plan_rows(-1, 8, 64) == -1 and lib.mq_plan_rows(1, 1, 4096) == -1
    # the rows any distribution takes fit: every expert's rows rounded up to 16
    for T, k, E in ((1, 1, 1), (3, 5, 7), (100, 4, 16), (33, 2, 1024)):
        worst = min(T * k, E)
        assert lib.mq_plan_rows(T, k, E) >= 16 * (worst - 1) + 16 * (-(-(T * k - worst + 1) // 16))


def test_binding_refusals(mq):
    import torch
    x = torch.zeros(4, 64)
    w = mq.MX(torch.zeros(1, 1, 1024, dtype=torch.uint8), torch.zeros(1, 1, 256, dtype=torch.uint8), 16, 64)
    plan = mq.ExpertPlan(*(torch.zeros(n, dtype=torch.int32) for n in (3, 16)), torch.zeros(4, 2, dtype=torch.int32))
    for bad in (x, x.bfloat16()):                       # host tensors never reach the library
        with pytest.raises(ValueError, match="device tensors"):
            mq.mx_quantize(bad)
        with pytest.raises(ValueError, match="device tensors"):
            mq.mx_linear(bad, w)
    with pytest.raises(ValueError, match="device tensors"):
        mq.mx_dequantize(w)
    with pytest.raises(ValueError, match="device tensors"):
        mq.route(x, 4)
    with pytest.raises(ValueError, match="device tensors"):
        mq.expert_plan(torch.zeros(4, 2, dtype=torch.int32), 8)
    with pytest.raises(ValueError, match="device tensors"):
        mq.mx_experts_up(x, w, w, plan)
    with pytest.raises(ValueError, match="device tensors"):
        mq.mx_experts_down(x, w, plan, x)
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        mq.mx_quantize(x.double())
    with pytest.raises(TypeError, match="torch.Tensor"):
        mq.mx_quantize([1.0])
    with pytest.raises(ValueError, match="axes"):
        mq.mx_quantize(x[0])
    with pytest.raises(ValueError, match="last axis"):
        mq.mx_quantize(x.t())
    with pytest.raises(ValueError, match="no columns"):
        mq.mx_quantize(x[:, :0])
    with pytest.raises(TypeError, match="MX matrix"):
        mq.mx_dequantize(x)
    for kw, what in ((dict(score="relu"), "score"), (dict(group_score="mean"), "group_score"), (dict(groups=3), "groups"),
                     (dict(groups=4, top_groups=5), "groups"), (dict(groups=0), "groups"), (dict(k=65), "k = 65"),
                     (dict(k=0), "k = 0"), (dict(groups=8, top_groups=1, k=9), "k = 9")):
        with pytest.raises(ValueError, match=what):
            mq.route(x, **{"k": 4, **kw})
    with pytest.raises(ValueError, match="no plan"):
        mq.plan_rows(4, 4, 5000)
    with pytest.raises(ValueError, match="int32"):
        mq.expert_plan(torch.zeros(4), 8)


def test_reference_layout_and_values():
    """The host reference itself: its device layout against the values' positions, and
    quantization of the grid's own values."""
    import numpy as np
    import tests.mx_reference as ref
    rng = np.random.default_rng(0)
    x = rng.standard_normal((19, 700))
    codes, scale = ref.quantize(x)
    v = ref.values(codes, scale)
    rel = np.abs(v - x) / np.repeat(np.abs(np.pad(x, ((0, 0), (0, 4))).reshape(19, -1, 32)).max(2), 32, 1)[:, :700]
    # off by at most half the widest step (2 X) or by the part above 6 X: 2 X against a peak of 4 X .. 8 X
    assert rel.max() <= 0.25
    np.testing.assert_array_equal(ref.values(*ref.quantize(v)), v)
    c, s = ref.pack(codes, scale)
    G, G4 = c.shape[1], s.shape[1]
    c, s = c.reshape(-1), s.reshape(-1)
    for r, k in ((0, 0), (18, 699), (16, 127), (3, 128), (5, 515)):
        lane = ((k // 32) % 4) * 16 + r % 16
        byte = c[(((r // 16) * G + k // 128) * 64 + lane) * 16 + (k % 32) // 2]
        assert (byte >> (4 * (k % 2))) & 15 == codes[r, k]
        assert s[(((r // 16) * G4 + k // 512) * 64 + lane) * 4 + (k // 128) % 4] == scale[r, k // 32]
