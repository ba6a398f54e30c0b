"""What the microscaled and routing calls guard against besides wrong arguments: order of
a wave's LDS accesses, operands that are no whole tuples, plans and sizes at their limits,
a machine without the extension module."""
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def mq():
    import dense_sparse_bit_amd
    return dense_sparse_bit_amd


@pytest.mark.parametrize("source", ["mx_gemm.hip", "mx_quant.hip", "route.hip"])
def test_lanes_hand_lds_over_through_fences(source):
    """A wave barrier alone orders no memory accesses for the compiler: lanes that read
    what others of their wave stored do so behind mx_wave_sync, which fences both sides."""
    csrc = os.path.join(ROOT, "dense_sparse_bit_amd", "csrc")
    assert "__builtin_amdgcn_wave_barrier" not in open(os.path.join(csrc, source)).read()
    helper = re.search(r"void mx_wave_sync\(\) \{(.*?)\}", open(os.path.join(csrc, "mx_device.h")).read(), re.S).group(1)
    calls = re.findall(r"__builtin_amdgcn_(\w+)\(([^)]*)\)", helper)
    assert calls == [("fence", '__ATOMIC_RELEASE, "wavefront", "local"'), ("wave_barrier", ""),
                     ("fence", '__ATOMIC_ACQUIRE, "wavefront", "local"')]


def _short_operands(mq, device):
    """Instances of the public tuples with too few items, where each call takes one."""
    import torch
    zeros = lambda *shape, dtype=torch.float32: torch.zeros(*shape, dtype=dtype, device=device)
    x, h, weights = zeros(4, 64), zeros(32, 64), zeros(4, 2)
    plan = mq.ExpertPlan(*(zeros(*shape, dtype=torch.int32) for shape in ((3,), (32,), (4, 2))))
    w = mq.MX(zeros(1, 1, 1024, dtype=torch.uint8), zeros(1, 1, 256, dtype=torch.uint8), 16, 64)
    e = mq.MX(zeros(2, 1, 1, 1024, dtype=torch.uint8), zeros(2, 1, 1, 256, dtype=torch.uint8), 16, 64)
    for n in range(4):
        a = tuple.__new__(mq.MX, w[:n])
        yield from ((lambda a=a: mq.mx_dequantize(a)), (lambda a=a: mq.mx_linear(a, w)))
        if device == "cpu":                      # the rest comes after checks that host tensors do not pass
            continue
        yield from ((lambda a=a: mq.mx_linear(x, a)), (lambda a=a: mq.mx_quantize(x, out=a)),
                    (lambda a=a: mq.mx_experts_up(x, a, e, plan)), (lambda a=a: mq.mx_experts_up(x, e, a, plan)),
                    (lambda a=a: mq.mx_experts_down(h, a, plan, weights)))
        if n < 3:
            p = tuple.__new__(mq.ExpertPlan, plan[:n])
            yield from ((lambda p=p: mq.mx_experts_up(x, e, e, p)), (lambda p=p: mq.mx_experts_down(h, e, p, weights)))


@pytest.mark.parametrize("device", ["cpu", pytest.param("cuda", marks=pytest.mark.gpu)])
def test_tuples_with_items_missing_are_refused(mq, device):
    import torch
    if device == "cpu" and torch.cuda.is_available():
        pytest.skip("the host's own order of checks, where no GPU is visible")
    for call in _short_operands(mq, device):
        with pytest.raises(TypeError, match="must be an"):
            call()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [4, 40])
def test_rows_past_the_last_experts_are_no_rows(mq, T):
    """A slot whose row lies after the last expert's adds zero, token by token and in row
    blocks alike, whatever the workspace held before."""
    import torch
    E, k, D, I = 4, 2, 72, 96
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.zeros(T, k, dtype=torch.int32, device="cuda")
    plan = mq.expert_plan(ids, E)
    rows = plan.row_token.numel()
    assert int(plan.offsets[E]) < rows
    w = mq.mx_quantize(torch.randn(E, D, I, generator=g, device="cuda"))
    h = torch.randn(rows, I, generator=g, device="cuda")
    weights = torch.rand(T, k, generator=g, device="cuda")
    lib, stream = mq.lib(), torch.cuda.current_stream().cuda_stream
    need = lib.mq_mx_experts_down_workspace_bytes(T, k, E, D, I)
    results = []
    for row in (rows - 1, int(plan.offsets[E]), -1):
        row_of = plan.row_of.clone()
        row_of[T // 2, 1] = row
        work = torch.full((need + 16,), 255, dtype=torch.uint8, device="cuda")          # NaN in fp32
        y = torch.empty(T, D, device="cuda")
        assert lib.mq_mx_experts_down(h.data_ptr(), 0, T, k, E, D, I, plan.offsets.data_ptr(), row_of.data_ptr(),
                                      weights.data_ptr(), w.codes.data_ptr(), w.scales.data_ptr(), y.data_ptr(), 0,
                                      work.data_ptr(), need, stream) == 0
        torch.cuda.synchronize()
        results.append(y)
    assert torch.isfinite(results[2]).all()
    assert torch.equal(results[0], results[2]) and torch.equal(results[1], results[2])


def test_no_workspace_for_calls_that_are_refused(mq):
    """The sizes of a workspace go by the checks of the call that takes it: a program learns
    of a refusal before it allocates. 2^24 slots make more than 2^24 rows of a plan."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("host-only argument checks run where no GPU is visible")
    lib, p = mq.lib(), 0x10000
    up = lambda T, k, E, D, I: lib.mq_mx_experts_up(p, 1, D, T, k, E, D, I, p, p, p, p, p, p, p, p, 1, None, 0, None)
    down = lambda T, k, E, D, I: lib.mq_mx_experts_down(p, 1, T, k, E, D, I, p, p, p, p, p, p, 1, None, 0, None)
    for T, k, E, D, I in ((1 << 21, 8, 1024, 512, 256), (1 << 24, 1, 2, 64, 64), (100, 4, 1024, 1 << 20, 1 << 11),
                          (100, 4, 1024, 1 << 11, 1 << 20), (100, 0, 8, 64, 64), (100, 4, 8, 0, 64), (100, 4, 8, 64, 0)):
        assert up(T, k, E, D, I) < 0 and down(T, k, E, D, I) < 0
        assert lib.mq_mx_experts_up_workspace_bytes(T, k, E, D, I) == 0, (T, k, E, D, I)
        assert lib.mq_mx_experts_down_workspace_bytes(T, k, E, D, I) == 0, (T, k, E, D, I)
    # refused for the missing workspace alone
    assert up(100, 4, 8, 64, 64) == -1 and lib.mq_mx_experts_up_workspace_bytes(100, 4, 8, 64, 64) > 0
    assert down(100, 4, 8, 64, 64) == -1 and lib.mq_mx_experts_down_workspace_bytes(100, 4, 8, 64, 64) > 0


def _python(code):
    return subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True, timeout=300,
                          env={**os.environ, "HIP_VISIBLE_DEVICES": "-1"})


WITHOUT = "import sys; sys.modules['dense_sparse_bit_amd._binding'] = None; "


def test_package_without_the_extension_module():
    """The package imports, says so, and passes its host tests."""
    r = _python(WITHOUT + "import dense_sparse_bit_amd as mq; assert mq._binding is None; import pytest; "
                "sys.exit(pytest.main(['-q', '-x', '-p', 'no:cacheprovider', '-m', 'not gpu', "
                "'tests/test_abi.py', 'tests/test_mx_abi.py']))")
    assert r.returncode == 0, r.stdout + r.stderr
    assert "RuntimeWarning: _binding.so is missing" in r.stderr, r.stderr


def test_extension_module_of_another_torch_is_not_loaded(mq):
    if mq._binding is None:
        pytest.skip("no extension module here")
    r = _python("import torch; torch.__version__ = '9.9'; import dense_sparse_bit_amd as mq; assert mq._binding is None")
    assert r.returncode == 0, r.stdout + r.stderr
    assert "RuntimeWarning" in r.stderr and "this is torch 9.9" in r.stderr, r.stderr
    r = _python("import dense_sparse_bit_amd as mq; assert mq._binding is not None")
    assert r.returncode == 0 and "RuntimeWarning" not in r.stderr, r.stdout + r.stderr


@pytest.mark.gpu
def test_the_long_way_gives_the_same_bits(mq, monkeypatch):
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    draw = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    E, k, D, I = 8, 2, 200, 96
    x, w, bias, router = draw(40, D), draw(64, D), draw(64), draw(40, E)
    wg, wu, wd = draw(E, I, D), draw(E, I, D), draw(E, D, I)

    def calls():
        for T in (40, 3, 0):
            a = mq.mx_quantize(x[:T])
            b = mq.mx_quantize(wg)
            yield from (*a[:2], *b[:2], mq.mx_dequantize(a, dtype=torch.float16), mq.mx_dequantize(b))
            q = mq.mx_quantize(w, out=mq.mx_quantize(w))
            yield from (mq.mx_linear(x[:T], q, bias=bias), mq.mx_linear(a, q, out_dtype=torch.float32),
                        mq.mx_linear(x[:T], q, y=torch.empty(T, 64, device="cuda", dtype=torch.float16)))
            ids, weights = mq.route(router[:T], k, score="sigmoid", groups=4, top_groups=2, group_score="top2", scale=1.5)
            plan = mq.expert_plan(ids, E)
            yield from (ids, weights, *plan)
            up, down = (mq.mx_quantize(wg), mq.mx_quantize(wu)), mq.mx_quantize(wd)
            h = mq.mx_experts_up(x[:T], *up, plan, out_dtype=torch.float32)
            yield from (h, mq.mx_experts_down(h, down, plan, weights), mq.mx_experts(x[:T], *up, down, plan, weights))

    assert mq._binding is not None
    short = list(calls())
    for module in ("mx", "experts"):
        monkeypatch.setattr(sys.modules[f"dense_sparse_bit_amd.{module}"], "_binding", None)
    for i, (a, b) in enumerate(zip(short, calls(), strict=True)):
        assert torch.equal(a, b) and a.dtype == b.dtype, i


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 50])
def test_layer_rounds_h_to_the_type_asked_for(mq, T):
    """mx_experts is mx_experts_up and mx_experts_down with h in h_dtype; bf16 by default."""
    import torch
    E, k, D, I = 4, 2, 136, 80
    g = torch.Generator(device="cuda").manual_seed(T)
    draw = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    x, w = draw(T, D), [mq.mx_quantize(draw(*s)) for s in ((E, I, D), (E, I, D), (E, D, I))]
    ids, weights = mq.route(draw(T, E), k)
    plan = mq.expert_plan(ids, E)
    layer = lambda **kw: mq.mx_experts(x, *w, plan, weights, out_dtype=torch.float32, **kw)
    results = {}
    for dtype in (torch.bfloat16, torch.float16, torch.float32):
        h = mq.mx_experts_up(x, *w[:2], plan, out_dtype=dtype)
        results[dtype] = mq.mx_experts_down(h, w[2], plan, weights, out_dtype=torch.float32)
        assert torch.equal(layer(h_dtype=dtype), results[dtype]), dtype
    assert torch.equal(layer(), results[torch.bfloat16])
    assert not torch.equal(results[torch.bfloat16], results[torch.float32])
    with pytest.raises(TypeError, match="float32, bfloat16 or float16"):
        layer(h_dtype=torch.int32)


def _fp32_rows(mq, T, k, E, D, I):
    """Bytes of a down product's workspace that hold fp32 rows."""
    lib = mq.lib()
    round16 = lambda n: -(-n // 16) * 16
    P = lib.mq_plan_rows(T, k, E)
    rest = round16(lib.mq_mx_codes_bytes(P, I)) + round16(lib.mq_mx_scales_bytes(P, I)) + \
        round16(4 * (4 + 4 * (P // 16 // 8 + E + 2)))
    return P, lib.mq_mx_experts_down_workspace_bytes(T, k, E, D, I) - rest


@pytest.mark.parametrize("D", [72, 1000, 2880, 4096, 5120, 7168])
def test_rows_of_down_products_stay_within_their_bound(mq, D):
    """Parts of at most 200 MiB, as long as two blocks of 256 columns take no more; then of at
    most 1024 columns. Never more columns than there are."""
    seen = set()
    for T in (9, 17, 300, 3000, 4096, 6000, 8192, 10000, 12500, 16384, 20000, 32768, 65536, 200000):
        P, rows = _fp32_rows(mq, T, 8, 64, D, 256)
        assert 0 < rows <= (P * -(-D // 4) * 4 + 3) * 4
        small = P * 512 * 4 <= 200 << 20
        assert rows <= (200 << 20 if small else P * 1024 * 4), (T, P, rows)
        seen.add(small)
    assert seen == {True, False}


@pytest.mark.gpu
def test_down_products_of_more_rows_than_a_part_of_the_cache_holds(mq):
    """More than 102400 rows: two parts of at most 1024 columns, the second a shorter one."""
    import numpy as np
    import torch
    from tests.test_mx_large import _check_layer
    T, k, E, D, I = 14000, 8, 8, 1101, 40
    rng = np.random.default_rng(5)
    ids = rng.integers(0, E, (T, k)).astype(np.int32)
    ids[rng.random((T, k)) < 0.02] = -1
    P, rows = _fp32_rows(mq, T, k, E, D, I)
    assert P > 102400 and rows == P * 768 * 4
    _check_layer(mq, ids, E, D, I, torch.bfloat16, "bf16", [0, 1, 6999, 13998, 13999])
