"""The gradients of experts_gather and experts_combine where only some of them are wanted: the same
bits as where all are, and no memory for the others."""
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
        from dense_sparse_bit_amd import experts
        monkeypatch.setattr(experts, "_binding", None)
    return request.param


def _inputs(mq, T, E, k, D, dtype):
    import torch
    g = torch.Generator(device="cuda").manual_seed(T + k)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.int()
    ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.1, -1, ids).int().contiguous()
    plan = mq.expert_plan(ids, E)
    rand = lambda *size: torch.randn(*size, generator=g, device="cuda").to(dtype)
    P = plan.row_token.numel()
    return plan, rand(T, D), rand(P, D), torch.rand(T, k, generator=g, device="cuda"), rand(P, D), rand(T, D)


@pytest.mark.parametrize("T,E,k,D", [(1, 4, 2, 128), (37, 8, 3, 100), (64, 64, 8, 4096), (50, 16, 11, 260)])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_each_gradient_by_itself(mq, way, dtype, T, E, k, D):
    import torch
    plan, x, rows, weights, drows, dy = _inputs(mq, T, E, k, D, {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype])
    for call, operand, given in ((lambda a, v: mq.experts_gather(a, plan, v), x, drows), (lambda a, v: mq.experts_combine(a, plan, v), rows, dy)):
        a, v = operand.clone().requires_grad_(), weights.clone().requires_grad_()
        both = torch.autograd.grad(call(a, v), (a, v), given)
        # asked for one of two
        out = call(a, v)
        assert torch.equal(torch.autograd.grad(out, a, given, retain_graph=True)[0], both[0])
        assert torch.equal(torch.autograd.grad(out, v, given)[0], both[1])
        # one leaf
        assert torch.equal(torch.autograd.grad(call(a, weights), a, given)[0], both[0])
        assert torch.equal(torch.autograd.grad(call(operand, v), v, given)[0], both[1])
        # dy with rows that share their memory
        if given is dy:
            one = dy[:1].expand(T, D)
            want = torch.autograd.grad(call(a, v), (a, v), one.contiguous())
            assert torch.equal(torch.autograd.grad(call(operand, v), v, one)[0], want[1])


def test_a_routers_gradient_takes_no_memory_for_the_rows(mq, way):
    """Weights alone want a gradient: one of the rows (P x D) is not made for it."""
    import torch
    T, E, k, D = 256, 64, 8, 4096
    plan, x, rows, weights, drows, dy = _inputs(mq, T, E, k, D, torch.float32)
    P = rows.shape[0]
    v = weights.clone().requires_grad_()
    for out, given in ((mq.experts_combine(rows, plan, v), dy), (mq.experts_gather(x, plan, v), drows)):
        torch.autograd.grad(out, v, given, retain_graph=True)
        torch.cuda.synchronize()
        before = torch.cuda.memory_allocated()
        torch.cuda.reset_peak_memory_stats()
        torch.autograd.grad(out, v, given)
        assert torch.cuda.max_memory_allocated() - before < P * D * 4 // 2


def test_a_second_derivative_of_one_gradient_is_an_error(mq, way):
    import torch
    plan, x, rows, weights, drows, dy = _inputs(mq, 20, 4, 2, 128, torch.float32)
    v = weights.clone().requires_grad_()
    dv, = torch.autograd.grad(mq.experts_combine(rows, plan, v), v, dy.requires_grad_(), create_graph=True)
    with pytest.raises(RuntimeError):
        dv.sum().backward()
