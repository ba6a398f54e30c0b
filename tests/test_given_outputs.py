"""Outputs that a caller gives are written in place, and autograd is told so: a backward pass whose
saved tensors were overwritten is an error, not a gradient of other values."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mq():
    import torch
    assert torch.cuda.is_available()
    import dense_sparse_bit_amd
    return dense_sparse_bit_amd


@pytest.fixture(params=["short way", "long way"])
def way(request, monkeypatch):
    if request.param == "long way":
        from dense_sparse_bit_amd import experts, mx, w4
        for module in (experts, mx, w4):
            monkeypatch.setattr(module, "_binding", None)
    return request.param


def _layer(mq):
    import torch
    g = torch.Generator(device="cuda").manual_seed(0)
    T, E, k, D = 20, 4, 2, 128
    ids, weights = mq.route(torch.randn(T, E, generator=g, device="cuda"), k)
    plan = mq.expert_plan(ids, E)
    codes = torch.randint(0, 16, (E, D, D), generator=g, device="cuda", dtype=torch.uint8)
    w = mq.w4_pack(codes, torch.rand(E, D, 1, generator=g, device="cuda").half())
    return torch.randn(T, D, generator=g, device="cuda"), plan, weights, w, torch.randn(T, E, generator=g, device="cuda")


def test_overwritten_operands_of_a_gradient_are_an_error(mq, way):
    import torch
    x, plan, weights, w, logits = _layer(mq)
    T, D = x.shape
    P = plan.row_token.numel()
    mxw = mq.mx_quantize(torch.randn(D, D, device="cuda"))
    calls = {
        "rows": [lambda b: mq.w4_experts_linear(x, w, plan, by_token=True, y=b), lambda b: mq.experts_gather(x, plan, rows=b),
                 lambda b: mq.mx_linear(torch.randn(P, D, device="cuda"), mxw, y=b),
                 lambda b: mq.w4_linear(torch.randn(P, D, device="cuda"), w._replace(codes=w.codes[0], scales=w.scales[0]), y=b)],
        "x": [lambda b: mq.experts_combine(torch.randn(P, D, device="cuda"), plan, weights, y=b),
              lambda b: mq.w4_dequantize(mq.w4_quantize(x), out=b), lambda b: mq.mx_dequantize(mq.mx_quantize(x), out=b)],
        "weights": [lambda b: mq.route(logits, 2, weights=b)],
    }
    for what, writes in calls.items():
        for write in writes:
            v = weights.clone().requires_grad_()
            if what == "rows":                       # the weights' gradient keeps the rows
                buffer = mq.w4_experts_linear(x, w, plan, by_token=True, out_dtype=torch.float32)
                y = mq.experts_combine(buffer, plan, v)
            elif what == "x":
                buffer = x.clone()
                y = mq.experts_gather(buffer, plan, v)
            else:                                    # the rows' gradient keeps the weights
                buffer = weights.clone()
                v = torch.randn(P, D, device="cuda", requires_grad=True)
                y = mq.experts_combine(v, plan, buffer)
            before = buffer._version
            write(buffer)
            assert buffer._version > before
            with pytest.raises(RuntimeError, match="inplace"):
                torch.autograd.grad(y, v, torch.ones_like(y))
    # ids too; a buffer that nothing kept is written as before
    ids = torch.empty(T, 2, dtype=torch.int32, device="cuda")
    before = ids._version
    mq.route(logits, 2, ids=ids)
    assert ids._version > before


def test_outputs_of_inference_mode(mq, way):
    """Their versions are not counted, and they are written."""
    import torch
    x, plan, weights, w, logits = _layer(mq)
    with torch.inference_mode():
        rows = torch.empty(plan.row_token.numel(), x.shape[1], device="cuda")
        y, ids, v = torch.empty_like(x), torch.empty_like(plan.row_of), torch.empty_like(weights)
        mq.w4_experts_linear(x, w, plan, by_token=True, y=rows)
        mq.experts_combine(rows, plan, weights, y=y)
        mq.route(logits, 2, ids=ids, weights=v)
        assert torch.equal(y, mq.experts_combine(rows, plan, weights)) and torch.equal(v, mq.route(logits, 2)[1])
    with torch.no_grad():
        assert mq.experts_combine(rows, plan, weights, y=y) is y


def test_outputs_over_the_input_are_refused(mq, way):
    """Workgroups would overwrite rows that others still read. Memory before, behind and beside it is not refused."""
    import torch
    x, plan, weights, w, _ = _layer(mq)
    T, D = x.shape
    P = plan.row_token.numel()
    one = w._replace(codes=w.codes[0], scales=w.scales[0])
    both = torch.zeros(2 * P, D, device="cuda")
    cases = [(lambda a, y: mq.w4_linear(a, one, y=y), T, T), (lambda a, y: mq.w4_experts_linear(a, w, plan, y=y), P, P),
             (lambda a, y: mq.w4_experts_linear(a, w, plan, by_token=True, y=y), T, P), (lambda a, y: mq.experts_gather(a, plan, rows=y), T, P),
             (lambda a, y: mq.experts_combine(a, plan, weights, y=y), P, T)]
    for call, m, n in cases:
        a = both[:m]
        for y in (both[:n], both[m - 1:m - 1 + n], both.view(-1)[4:4 + n * D].view(n, D)):
            with pytest.raises(ValueError, match="shares memory"):
                call(a, y)
        both.normal_()
        apart = call(a.clone(), torch.empty(n, D, device="cuda"))
        assert torch.equal(call(a, both[m:m + n] if m + n <= len(both) else torch.empty(n, D, device="cuda")), apart)
        shifted = both[n:n + m]
        want = call(shifted.clone(), torch.empty(n, D, device="cuda"))
        assert torch.equal(call(shifted, both[:n]), want)
