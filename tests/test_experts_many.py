"""The experts' products with more experts than a wave has lanes, up to MQ_MAX_EXPERTS: the
search for a row's expert goes through several rounds of 64, the list of row blocks through
several waves' sums, and at 1024 experts the rows after the last one's have no entry of their
own. High-numbered experts are the popular ones. Tolerances: tests/test_experts.py."""
import numpy as np
import pytest

from tests.test_mx_large import _check_layer, _layer

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mq():
    import torch
    assert torch.cuda.is_available()
    import dense_sparse_bit_amd
    return dense_sparse_bit_amd


def _ids(T, k, E, seed):
    """Half of the slots among the last eight experts, a fourth with the very last one, the
    others anywhere; some without."""
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, E, (T, k))
    high = rng.random((T, k))
    ids = np.where(high < 0.5, E - 1 - rng.integers(0, 8, (T, k)), ids)
    ids = np.where(high < 0.25, E - 1, ids)
    ids[rng.random((T, k)) < 0.05] = -1
    ids[0, 0] = E - 1
    return ids.astype(np.int32)


@pytest.mark.parametrize("E", [65, 128, 257, 1023, 1024])
@pytest.mark.parametrize("T,k", [(1, 8), (3, 4), (8, 8), (9, 4), (16, 6), (17, 4), (300, 4), (700, 2)])
def test_many_experts(mq, T, k, E):
    """Token by token, split over K and in row blocks; every row of no token is zero, those
    after the last expert's among them."""
    import torch
    print(f"[experts] {T} {k} {E}", flush=True)
    ids, D, I = _ids(T, k, E, T + E), 132, 40
    tokens = list(range(T)) if T <= 17 else sorted({0, 1, T // 2, T - 2, T - 1, *np.flatnonzero((ids == E - 1).any(1))[-4:].tolist()})
    _check_layer(mq, ids, E, D, I, torch.bfloat16, "fp32", tokens)
    x, (wg, wu, _), plan, _ = _layer(mq, ids, E, D, I, torch.bfloat16)
    rows = plan.row_token.numel()
    assert int(plan.offsets[E]) < rows
    h = torch.full((rows, I), float("nan"), device="cuda")
    mq.mx_experts_up(x, wg, wu, plan, h=h)
    assert (h[plan.row_token < 0] == 0).all() and not torch.isnan(h).any()


@pytest.mark.parametrize("E", [256, 1024])
def test_each_expert_has_rows_and_none_are_left(mq, E):
    """The rows of the last expert end where the plan's do."""
    import torch
    ids = np.random.default_rng(E).permutation(E).reshape(E // 4, 4).astype(np.int32)
    x, _, plan, _ = _layer(mq, ids, E, 64, 32, torch.float32)
    assert int(plan.offsets[E]) == plan.row_token.numel()
    _check_layer(mq, ids, E, 64, 32, torch.float32, "bf16", list(range(0, E // 4, 7)))


@pytest.mark.parametrize("E", [129, 1024])
def test_no_slot_has_an_expert(mq, E):
    """All rows lie after the last expert's."""
    import torch
    for T in (2, 40):
        ids = np.full((T, 2), -1, dtype=np.int32)
        x, (wg, wu, wd), plan, weights = _layer(mq, ids, E, 96, 48, torch.bfloat16)
        h = torch.full((plan.row_token.numel(), 48), float("nan"), device="cuda")
        assert (mq.mx_experts_up(x, wg, wu, plan, h=h) == 0).all()
        y = torch.full((T, 96), float("nan"), device="cuda")
        assert (mq.mx_experts_down(h, wd, plan, weights, y=y) == 0).all()


@pytest.mark.parametrize("T", [2, 12, 40, 300])
def test_nan_stays_in_its_rows_and_columns(mq, T):
    """A NaN of x in the rows of its token, one of the weights in its expert's rows and column;
    in y in the tokens that have such a row."""
    import torch
    E, D, I = 5, 300, 72
    ids = np.stack([np.random.default_rng(t).permutation(E - 1)[:2] for t in range(T)]).astype(np.int32)
    ids[0], ids[1] = (0, 1), (2, 3)
    x, _, plan, weights = _layer(mq, ids, E, D, I, torch.float32)
    g = torch.Generator(device="cuda").manual_seed(1)
    wg, wu = torch.randn(2, E, I, D, generator=g, device="cuda")
    wd = torch.randn(E, D, I, generator=g, device="cuda")
    x[0, D - 1] = float("nan")
    wg[1, 7, 3], wu[2, I - 1, 290] = float("inf"), float("nan")
    gate, up, down = (mq.mx_quantize(w) for w in (wg, wu, wd))
    h = mq.mx_experts_up(x, gate, up, plan, out_dtype=torch.float32)
    bad = torch.zeros_like(h, dtype=torch.bool)
    row_of = plan.row_of.cpu().numpy()
    bad[row_of[0]] = True
    bad[row_of[ids == 1], 7] = True
    bad[row_of[ids == 2], I - 1] = True
    assert torch.equal(torch.isnan(h), bad)
    y = mq.mx_experts_down(h, down, plan, weights, out_dtype=torch.float32)
    marked = torch.from_numpy(((ids == 1) | (ids == 2)).any(1)).cuda()
    marked[0] = True
    assert torch.equal(torch.isnan(y), marked[:, None].expand_as(y))
    # and of the down weights in its column of the expert's tokens
    wd[3, 9, 0] = float("nan")
    clean = torch.randn(h.shape, generator=g, device="cuda")
    y = mq.mx_experts_down(clean, mq.mx_quantize(wd), plan, weights, out_dtype=torch.float32)
    want = torch.zeros_like(y, dtype=torch.bool)
    want[:, 9] = torch.from_numpy((ids == 3).any(1)).cuda()
    assert torch.equal(torch.isnan(y), want)


@pytest.mark.parametrize("T", [1, 40])
def test_silu_over_its_range(mq, T):
    """silu(g) u for every half of a whole number g in [-120, 120], with gate and up exact, as
    fp32: relative error at most (1.25 |g| + 8) 2^-24 (the exponential's argument is rounded;
    then an exponential, a sum, a reciprocal and two products of a unit or half of one), and
    below g = -87, where the value leaves fp32's normal range, 2^-119."""
    import torch
    gates = np.arange(-240, 241) / 2
    I, D = len(gates), 32
    w = np.zeros((I, D))
    w[:, 0], w[:, 1] = 4, -4                                    # a peak of 4 or 6: a scale of 1
    for i, g in enumerate(gates):
        left, at = abs(g), 2
        while left > 0:
            w[i, at] = next(v for v in (6, 4, 3, 2, 1.5, 1, 0.5) if v <= left)
            left -= w[i, at]
            at += 1
        w[i, 2:] *= np.sign(g)
    assert (w.sum(1) == gates).all()
    x = torch.ones(T, D, device="cuda")
    gate = torch.from_numpy(w).float().cuda()[None]
    up = torch.zeros(1, I, D, device="cuda")
    up[:, :, 0] = 1.0
    gate_q, up_q = mq.mx_quantize(gate), mq.mx_quantize(up)
    assert torch.equal(mq.mx_dequantize(gate_q), gate) and torch.equal(mq.mx_dequantize(up_q), up)
    plan = mq.expert_plan(torch.zeros(T, 1, dtype=torch.int32, device="cuda"), 1)
    h = mq.mx_experts_up(x, gate_q, up_q, plan, out_dtype=torch.float32)[:T].double().cpu().numpy()
    want = gates / (1 + np.exp(-gates))
    tol = np.where(gates < -87, 2.0 ** -119, (1.25 * np.abs(gates) + 8) * 2.0 ** -24 * np.abs(want))
    assert (np.abs(h - want) <= tol).all()
