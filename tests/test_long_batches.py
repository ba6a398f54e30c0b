"""Batches of more rows than a grid's axis holds: each workgroup takes several, one after the other.
Whole numbers, so that sums and dots are exact in any order."""
import pytest

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mq():
    import torch
    assert torch.cuda.is_available()
    import dense_sparse_bit_amd
    return dense_sparse_bit_amd


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("T,E,k,D", [(70001, 16, 2, 40), (66003, 12, 9, 20), (140001, 8, 1, 3)])
def test_tokens_and_rows_with_their_gradients(mq, dtype, T, E, k, D):
    import torch
    t = {"fp32": torch.float32, "bf16": torch.bfloat16}[dtype]
    g = torch.Generator(device="cuda").manual_seed(T)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.int()
    ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.1, -1, ids).int().contiguous()
    plan = mq.expert_plan(ids, E)
    P = plan.row_token.numel()
    whole = lambda *size: torch.randint(-2, 3, size, generator=g, device="cuda").to(t)
    live = plan.row_of >= 0
    at = plan.row_of.long().clamp(min=0)
    x, drows = whole(T, D).requires_grad_(), whole(P, D)
    weights = whole(T, k).float().requires_grad_()
    rows = mq.experts_gather(x, plan, weights)
    want = torch.zeros(P, D, device="cuda")
    want[at[live]] = (x.detach().float()[:, None, :] * weights.detach()[:, :, None])[live]
    assert torch.equal(rows.detach().float(), want)
    mine = drows.float()[at] * live[:, :, None]
    dx, dw = torch.autograd.grad(rows, (x, weights), drows)
    assert torch.equal(dx.float(), (mine * weights.detach()[:, :, None]).sum(1))
    assert torch.equal(dw, (mine * x.detach().float()[:, None, :]).sum(2))

    given, dy = whole(P, D).requires_grad_(), whole(T, D)
    y = mq.experts_combine(given, plan, weights)
    mine = given.detach().float()[at] * live[:, :, None]
    assert torch.equal(y.detach().float(), (mine * weights.detach()[:, :, None]).sum(1))
    dgiven, dw = torch.autograd.grad(y, (given, weights), dy)
    want = torch.zeros(P, D, device="cuda")
    want[at[live]] = (dy.float()[:, None, :] * weights.detach()[:, :, None])[live]
    assert torch.equal(dgiven.float(), want)
    assert torch.equal(dw, (mine * dy.float()[:, None, :]).sum(2))


def test_matrices_of_many_rows(mq):
    """More 16-row tiles than a grid's axis: what the first and the last rows become is what they become alone."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    R, K = 16 * 32768 * 2 + 40, 33
    x = torch.randn(R, K, generator=g, device="cuda").bfloat16()
    whole = mq.w4_quantize(x, group=32, zeros=True)
    back = mq.w4_dequantize(whole)
    s, z = torch.rand(R, 2, generator=g, device="cuda").half(), torch.randint(0, 16, (R, 2), generator=g, device="cuda").half()
    codes = torch.randint(0, 16, (R, K), generator=g, device="cuda", dtype=torch.uint8)
    packed = mq.w4_pack(codes, s, z, group=32)
    values = mq.w4_dequantize(packed)
    each = lambda v: v.repeat_interleave(32, 1)[:, :K].float()
    assert torch.equal(values, (codes.float() - each(z)) * each(s))
    for first in (0, 16 * 32767, 16 * 32768, 16 * 65536 - 32, 16 * 65536):
        rows = slice(first, min(first + 48, R))
        part = mq.w4_quantize(x[rows], group=32, zeros=True)
        tiles = slice(first // 16, first // 16 + part.codes.shape[0])
        assert torch.equal(whole.codes[tiles], part.codes) and torch.equal(whole.scales[tiles], part.scales) and torch.equal(whole.zeros[tiles], part.zeros)
        assert torch.equal(back[rows], mq.w4_dequantize(part))
