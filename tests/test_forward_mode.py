"""Calls without a forward-mode derivative refuse inputs that carry a tangent: a result without one
would say that the derivative is zero."""
import pytest


@pytest.fixture(scope="module")
def mq():
    import dense_sparse_bit_amd
    return dense_sparse_bit_amd


def _calls(mq, device):
    """(operands' sizes, which of them carry a tangent in turn, the call)"""
    import torch
    from dense_sparse_bit_amd.w4 import _new
    ids = torch.zeros(4, 2, dtype=torch.int32, device=device)
    if device == "cuda":
        plan = mq.expert_plan(ids, 2)
        codes, s = torch.zeros(2, 16, 128, dtype=torch.uint8, device=device), torch.zeros(2, 16, 1, device=device).half()
        w, we = mq.w4_pack(codes[0], s[0]), mq.w4_pack(codes, s)
    else:
        P = mq.plan_rows(4, 2, 2)
        plan = mq.ExpertPlan(torch.zeros(3, dtype=torch.int32), torch.zeros(P, dtype=torch.int32), ids)
        w, we = _new(16, 128, 128, None, torch.float16, False, "cpu"), _new(16, 128, 128, 2, torch.float16, False, "cpu")
    P = plan.row_token.numel()
    return [(((4, 128), (16,)), lambda x, b: mq.w4_linear(x, w, bias=b)), (((P, 128),), lambda x: mq.w4_experts_linear(x, we, plan)),
            (((4, 128),), lambda x: mq.w4_experts_linear(x, we, plan, by_token=True)),
            (((4, 128), (4, 2)), lambda x, v: mq.experts_gather(x, plan, v)), (((P, 128), (4, 2)), lambda r, v: mq.experts_combine(r, plan, v))]


def _refused(mq, device):
    import torch
    from torch.autograd import forward_ad
    for sizes, call in _calls(mq, device):
        for which in range(len(sizes)):
            for grad in (False, True):
                with forward_ad.dual_level():
                    given = [torch.ones(size, device=device) for size in sizes]
                    given[which] = forward_ad.make_dual(given[which].requires_grad_(grad), torch.ones_like(given[which]))
                    for mode in (torch.no_grad, torch.enable_grad):
                        with mode(), pytest.raises(ValueError, match="forward-mode" if not grad else "forward-mode|no gradient"):
                            call(*given)


def test_tangents_are_refused(mq):
    _refused(mq, "cpu")


@pytest.mark.gpu
def test_tangents_are_refused_on_the_device(mq):
    """By the short way too; operands without a tangent are not, in a dual level either."""
    import torch
    from torch.autograd import forward_ad
    _refused(mq, "cuda")
    with forward_ad.dual_level():
        for sizes, call in _calls(mq, "cuda"):
            call(*[torch.ones(size, device="cuda") for size in sizes])
    for sizes, call in _calls(mq, "cuda"):
        given = tuple(torch.ones(size, device="cuda") for size in sizes)
        with pytest.raises((RuntimeError, ValueError, TypeError)):
            torch.func.jvp(call, given, given)
