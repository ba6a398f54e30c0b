"""Tokens to the rows of their experts and back, with gradients, against plain statements
in 64 bits.

- gather: a copy, or one fp32 product, then one rounding: equal to the same in torch.
- combine: k products and k additions in fp32, each off by half a step (2^-24) of at most the
  sum of |w r|; then half a step of the output's type.
- dots: D products and additions in fp32 in some order: at most D + 8 times 2^-24 of the sum of
  the magnitudes. On whole numbers whose sums stay below 2^24 everything is exact.
"""
import pytest

pytestmark = pytest.mark.gpu

HALF_STEP = {"fp32": 2.0 ** -24, "bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
KINDS = ("fp32", "bf16", "fp16")


@pytest.fixture(scope="module")
def mq():
    import torch
    assert torch.cuda.is_available()
    import dense_sparse_bit_amd
    return dense_sparse_bit_amd


def _dtype(name):
    import torch
    return {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[name]


def _gen(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def _plan(mq, g, T, E, k):
    """Ids with losses, strangers (another rank's experts) and, in places, one expert twice."""
    import torch
    ids = torch.randint(-1, E + 1, (T, k), generator=g, device="cuda", dtype=torch.int32)
    return ids, mq.expert_plan(ids, E)


def _whole(g, *shape):
    import torch
    return torch.randint(-4, 5, shape, generator=g, device="cuda").float()


def _slots(plan):
    """(t, j, p) of the slots that have a row."""
    import torch
    t, j = torch.nonzero(plan.row_of >= 0, as_tuple=True)
    return t, j, plan.row_of[t, j].long()


SIZES = [(1, 4, 1, 1), (1, 64, 8, 4096), (2, 3, 2, 7), (5, 8, 3, 8), (17, 2, 9, 100), (33, 16, 8, 1000), (64, 5, 1, 2056), (100, 40, 17, 515),
         (300, 8, 2, 4100)]


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("dtype", KINDS)
def test_gather_matches_torch(mq, dtype, weighted):
    import torch
    for T, E, k, D in SIZES:
        g = _gen(T * D)
        _, plan = _plan(mq, g, T, E, k)
        x = torch.randn(T, D, generator=g, device="cuda").to(_dtype(dtype))
        weights = torch.randn(T, k, generator=g, device="cuda") if weighted else None
        t, j, p = _slots(plan)
        want = torch.zeros(plan.row_token.numel(), D, device="cuda")
        want[p] = x[t].float() * (weights[t, j][:, None] if weighted else 1.0)
        got = mq.experts_gather(x, plan, weights)
        assert got.dtype == x.dtype and torch.equal(got, want.to(x.dtype)), (T, E, k, D)
        rows = torch.full_like(got, float("nan"))
        assert mq.experts_gather(x, plan, weights, rows=rows) is rows and torch.equal(rows, got)


@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("dtype,out", [("fp32", "fp32"), ("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"), ("fp32", "bf16")])
def test_combine_matches_the_sum(mq, dtype, out, weighted):
    import torch
    for T, E, k, D in SIZES:
        g = _gen(T * D + 1)
        _, plan = _plan(mq, g, T, E, k)
        rows = torch.randn(plan.row_token.numel(), D, generator=g, device="cuda").to(_dtype(dtype))
        rows[plan.row_token < 0] = float("nan")        # nobody's rows are not read
        weights = torch.randn(T, k, generator=g, device="cuda") if weighted else None
        t, j, p = _slots(plan)
        each = torch.zeros(T, k, D, dtype=torch.float64, device="cuda")
        each[t, j] = rows[p].double() * (weights[t, j][:, None].double() if weighted else 1.0)
        want, most = each.sum(1), each.abs().sum(1)
        got = mq.experts_combine(rows, plan, weights, out_dtype=_dtype(out))
        assert got.dtype == _dtype(out)
        sums = 2 * k * 2.0 ** -24 * most
        bound = sums + HALF_STEP[out] * (want.abs() + sums) + (2.0 ** -25 if out == "fp16" else 0)
        assert ((got.double() - want).abs() <= bound).all(), (T, E, k, D)
        y = torch.empty(T, D, device="cuda", dtype=_dtype(out))
        assert mq.experts_combine(rows, plan, weights, y=y) is y and torch.equal(y, got)


def test_slots_without_a_row_add_their_weight_times_zero(mq):
    """As in the experts' products: a NaN weight is seen, a finite one is nothing."""
    import torch
    ids = torch.tensor([[0, -1], [-1, -1], [1, 5]], dtype=torch.int32, device="cuda")
    plan = mq.expert_plan(ids, 2)
    rows = torch.ones(plan.row_token.numel(), 40, device="cuda")
    weights = torch.tensor([[2.0, 3.0], [1.0, 1.0], [1.0, float("nan")]], device="cuda")
    y = mq.experts_combine(rows, plan, weights)
    assert (y[0] == 2).all() and (y[1] == 0).all() and y[2].isnan().all()
    assert (mq.experts_combine(rows, plan)[:, 0] == torch.tensor([1.0, 0.0, 1.0], device="cuda")).all()


def test_no_tokens_and_no_experts(mq):
    import torch
    for T in (0, 5):
        ids = torch.full((T, 2), -1, dtype=torch.int32, device="cuda")
        plan = mq.expert_plan(ids, 4)
        x = torch.randn(T, 30, device="cuda", requires_grad=True)
        w = torch.rand(T, 2, device="cuda", requires_grad=True)
        rows = mq.experts_gather(x, plan, w)
        assert rows.shape == (plan.row_token.numel(), 30) and (rows == 0).all()
        y = mq.experts_combine(rows, plan, w)
        assert y.shape == (T, 30) and (y == 0).all()
        dx, dw = torch.autograd.grad(y, (x, w), torch.ones_like(y))
        assert dx.shape == x.shape and dw.shape == w.shape and (dx == 0).all() and (dw == 0).all()


def test_strided_rows_of_x(mq):
    import torch
    g = _gen(3)
    for dtype in KINDS:
        wide = torch.randn(40, 300, generator=g, device="cuda").to(_dtype(dtype))
        x = wide[::2, 3:204]
        _, plan = _plan(mq, g, 20, 4, 3)
        assert torch.equal(mq.experts_gather(x, plan), mq.experts_gather(x.contiguous(), plan))
        one = x[:1].expand(20, 201)
        assert torch.equal(mq.experts_gather(one, plan), mq.experts_gather(one.contiguous(), plan))


# ------------------------------------------------------------------------------ gradients
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("dtype", KINDS)
def test_gradients_of_whole_numbers_are_exact(mq, dtype, weighted):
    """Formula and difference quotients, both exact: 9 values of at most 4 times weights of at most 4
    per slot, 17 slots, and dots of 4100 products of at most 16 stay below 2^24; a sum of 17
    products up to 16 is whole up to 272, which fp16 and bf16 (256) round, so bf16 sums are
    compared after the same rounding."""
    import torch
    kind = _dtype(dtype)
    for T, E, k, D in SIZES:
        g = _gen(T + D)
        _, plan = _plan(mq, g, T, E, k)
        t, j, p = _slots(plan)
        P = plan.row_token.numel()
        v = _whole(g, T, k) if weighted else torch.ones(T, k, device="cuda")
        # gather
        x = _whole(g, T, D).to(kind).requires_grad_()
        w = v.clone().requires_grad_() if weighted else None
        rows = mq.experts_gather(x, plan, w)
        given = _whole(g, P, D).to(kind)
        given[plan.row_token < 0] = float("nan")
        got = torch.autograd.grad(rows, (x, w) if weighted else (x,), given)
        each = torch.zeros(T, k, D, device="cuda")
        each[t, j] = given[p].float()
        assert got[0].dtype == kind and torch.equal(got[0], (each * v[:, :, None]).sum(1).to(kind))
        if weighted:
            assert torch.equal(got[1], (each * x.detach().float()[:, None, :]).sum(2))
        # the function is linear in x and in the weights: its change is its gradient times theirs
        step = _whole(g, T, D).to(kind)
        with torch.no_grad():
            change = (mq.experts_gather(x + step, plan, w).double() - rows.double())[p]
        if dtype == "fp32":
            assert (change * given[p].double()).sum() == (got[0].double() * step.double()).sum()
        # combine
        r = _whole(g, P, D).to(kind).requires_grad_()
        y = mq.experts_combine(r, plan, w)
        dy = _whole(g, T, D).to(kind)
        got = torch.autograd.grad(y, (r, w) if weighted else (r,), dy)
        want = torch.zeros(P, D, device="cuda")
        want[p] = dy[t].float() * v[t, j][:, None]
        assert got[0].dtype == kind and torch.equal(got[0], want.to(kind))
        each = torch.zeros(T, k, D, device="cuda")
        each[t, j] = r.detach()[p].float()
        if weighted:
            assert torch.equal(got[1], (each * dy.float()[:, None, :]).sum(2))
            with torch.no_grad():
                if dtype == "fp32":
                    step = _whole(g, T, k)
                    change = mq.experts_combine(r, plan, w + step).double() - y.double()
                    assert (change * dy.double()).sum() == (got[1].double() * step.double()).sum()


@pytest.mark.parametrize("dtype,out", [("fp32", "fp32"), ("bf16", "bf16"), ("fp16", "fp16"), ("bf16", "fp32"), ("fp32", "bf16")])
def test_gradients_of_free_values(mq, dtype, out):
    import torch
    for T, E, k, D in SIZES:
        g = _gen(T + D + 7)
        _, plan = _plan(mq, g, T, E, k)
        t, j, p = _slots(plan)
        P = plan.row_token.numel()
        weights = torch.randn(T, k, generator=g, device="cuda").requires_grad_()
        r = torch.randn(P, D, generator=g, device="cuda").to(_dtype(dtype)).requires_grad_()
        y = mq.experts_combine(r, plan, weights, out_dtype=_dtype(out))
        dy = torch.randn(T, D, generator=g, device="cuda").to(_dtype(out))
        dr, dw = torch.autograd.grad(y, (r, weights), dy)
        want = torch.zeros(P, D, device="cuda")
        want[p] = dy[t].float() * weights.detach()[t, j][:, None]
        assert torch.equal(dr, want.to(r.dtype))
        each = torch.zeros(T, k, D, dtype=torch.float64, device="cuda")
        each[t, j] = r.detach()[p].double() * dy[t].double()
        assert ((dw.double() - each.sum(2)).abs() <= (D + 8) * 2.0 ** -24 * each.abs().sum(2)).all()


def test_gradients_that_are_not_contiguous_and_partial_wants(mq):
    import torch
    g = _gen(1)
    T, E, k, D = 30, 4, 3, 50
    _, plan = _plan(mq, g, T, E, k)
    P = plan.row_token.numel()
    x = _whole(g, T, D)
    w = _whole(g, T, k)
    for needs in ((True, False), (False, True)):
        xl, wl = x.clone().requires_grad_(needs[0]), w.clone().requires_grad_(needs[1])
        mq.experts_gather(xl, plan, wl).sum().backward()           # an expanded gradient
        assert (xl.grad is not None, wl.grad is not None) == needs
        rl = _whole(g, P, D).requires_grad_(needs[0])
        wl = w.clone().requires_grad_(needs[1])
        mq.experts_combine(rl, plan, wl).sum().backward()
        assert (rl.grad is not None, wl.grad is not None) == needs
    # twice the same leaf; a transposed gradient
    xl = x.clone().requires_grad_()
    y = mq.experts_combine(mq.experts_gather(xl, plan), plan, w) + xl
    dy = _whole(g, D, T).t()
    (dx,) = torch.autograd.grad(y, xl, dy)
    live = (plan.row_of >= 0).float() * w
    assert torch.equal(dx, dy * (1 + live.sum(1, keepdim=True)))
    # a strided x with its weights' gradient
    wide = _whole(g, T, 2 * D)
    wl = w.clone().requires_grad_()
    rows = mq.experts_gather(wide[:, 3:3 + D], plan, wl)
    given = _whole(g, P, D)
    (dw,) = torch.autograd.grad(rows, wl, given)
    wl2 = w.clone().requires_grad_()
    (dw2,) = torch.autograd.grad(mq.experts_gather(wide[:, 3:3 + D].contiguous(), plan, wl2), wl2, given)
    assert torch.equal(dw, dw2)


@pytest.mark.parametrize("k", [1, 3, 8, 9, 20])
def test_slots_without_a_row_have_no_gradient(mq, k):
    """Their dots are 0 whatever the token holds, and a NaN in rows of no token goes nowhere."""
    import torch
    g = _gen(4)
    T, E, D = 40, 6, 75
    ids, plan = _plan(mq, g, T, E, k)
    lost = plan.row_of < 0
    assert lost.any()
    for D in (72, 75):
        x, w = torch.randn(T, D, generator=g, device="cuda"), torch.rand(T, k, generator=g, device="cuda")
        x[::3] = float("nan")
        x[1::3, 5] = float("inf")
        wl = w.clone().requires_grad_()
        given = torch.randn(plan.row_token.numel(), D, generator=g, device="cuda")
        (dw,) = torch.autograd.grad(mq.experts_gather(x, plan, wl), wl, given)
        assert (dw[lost] == 0).all() and (dw[::3][~lost[::3]]).isnan().all()
        wl = w.clone().requires_grad_()
        rows = torch.randn(plan.row_token.numel(), D, generator=g, device="cuda")
        rows[plan.row_token < 0] = float("nan")
        (dw,) = torch.autograd.grad(mq.experts_combine(rows, plan, wl), wl, x)
        assert (dw[lost] == 0).all() and (dw[::3][~lost[::3]]).isnan().all()


def test_changed_inputs_and_second_derivatives_are_refused(mq):
    import torch
    g = _gen(2)
    _, plan = _plan(mq, g, 10, 4, 2)
    w = torch.rand(10, 2, device="cuda", requires_grad=True)
    x = torch.randn(10, 20, device="cuda", requires_grad=True)
    rows = mq.experts_gather(x, plan, w)
    plan.row_of.add_(0)
    with pytest.raises(RuntimeError):
        rows.sum().backward()
    _, plan = _plan(mq, g, 10, 4, 2)
    rows = mq.experts_gather(x, plan, w)
    (dx,) = torch.autograd.grad(rows, x, torch.ones_like(rows), create_graph=True)
    with pytest.raises(RuntimeError):
        dx.sum().backward()


def test_same_bits_every_time_and_on_other_streams(mq):
    import torch
    g = _gen(5)
    T, E, k, D = 200, 8, 4, 1000
    _, plan = _plan(mq, g, T, E, k)
    x = torch.randn(T, D, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.rand(T, k, generator=g, device="cuda")
    given = torch.randn(plan.row_token.numel(), D, generator=g, device="cuda").to(torch.bfloat16)

    def once(stream=None):
        xl, wl = x.clone().requires_grad_(), w.clone().requires_grad_()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        rows = mq.experts_gather(xl, plan, wl, stream=stream)
        y = mq.experts_combine(rows, plan, wl, stream=stream)
        if stream is not None:
            torch.cuda.current_stream().wait_stream(stream)
        return (rows.detach(), y.detach()) + torch.autograd.grad((rows, y), (xl, wl), (given, torch.ones_like(y)))

    want = once()
    torch.cuda.synchronize()
    for stream in (None, torch.cuda.Stream(), None):
        got = once(stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)


def test_forward_and_backward_in_a_graph(mq):
    """A whole step, captured, with its own leaves, replayed among eager steps."""
    import torch
    g = _gen(6)
    T, E, k, D = 50, 8, 2, 300
    ids, plan = _plan(mq, g, T, E, k)
    x, w = torch.randn(T, D, generator=g, device="cuda"), torch.rand(T, k, generator=g, device="cuda")
    given = torch.randn(T, D, generator=g, device="cuda")

    def step(xl, wl, ids, given):
        plan = mq.expert_plan(ids, E)
        y = mq.experts_combine(mq.experts_gather(xl, plan), plan, wl)
        return (y.detach(),) + torch.autograd.grad(y, (xl, wl), given)

    fx, fw, fids, fgiven = x.clone().requires_grad_(), w.clone().requires_grad_(), ids.clone(), given.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(fx, fw, fids, fgiven)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(fx, fw, fids, fgiven)
    for i in range(4):
        x2, w2 = torch.randn(T, D, generator=g, device="cuda"), torch.rand(T, k, generator=g, device="cuda")
        ids2 = torch.randint(-1, E, (T, k), generator=g, device="cuda", dtype=torch.int32)
        with torch.no_grad():
            fx.copy_(x2), fw.copy_(w2), fids.copy_(ids2)
        want = step(x2.requires_grad_(), w2.requires_grad_(), ids2, given)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert torch.equal(a, b)


def test_a_layer_of_plain_experts_trains_through_them(mq):
    """route, plan, gather, experts in torch, combine: gradients of tokens, experts' matrices
    and the router against the same layer written token by token, in 64 bits."""
    import torch
    g = _gen(8)
    T, E, k, D = 40, 4, 2, 24
    x = torch.randn(T, D, generator=g, device="cuda").requires_grad_()
    router = torch.randn(E, D, generator=g, device="cuda").requires_grad_()
    experts = (torch.randn(E, D, D, generator=g, device="cuda") / 5).requires_grad_()
    logits = x @ router.t()
    ids, _ = mq.route(logits.detach(), k)
    weights = torch.softmax(logits, 1).gather(1, ids.long())
    plan = mq.expert_plan(ids, E)
    rows = mq.experts_gather(x, plan)
    ends = plan.offsets.tolist()
    out = torch.cat([rows[ends[e]:ends[e + 1]] @ experts[e].t() for e in range(E)] + [rows[ends[E]:]])
    y = mq.experts_combine(out, plan, weights)
    dy = torch.randn(T, D, generator=g, device="cuda")
    got = torch.autograd.grad(y, (x, router, experts), dy)
    x64, r64, e64 = (v.detach().double().requires_grad_() for v in (x, router, experts))
    w64 = torch.softmax(x64 @ r64.t(), 1).gather(1, ids.long())
    each = torch.stack([torch.stack([e64[int(ids[t, j])] @ x64[t] for j in range(k)]) for t in range(T)])
    want = torch.autograd.grad((w64[:, :, None] * each).sum(1), (x64, r64, e64), dy.double())
    for a, b in zip(got, want):
        # The longest way, to the router's gradient: a logit's 24 products, a softmax (8), an expert's 24, a dot's
        # 24, the softmax's gradient (8), a sum over 40 tokens: 128 roundings of half a step (2^-24), each of
        # sums whose magnitudes add up to at most 25 times the largest value: 3200 of them, and a fourth for
        # the products of errors and for exp.
        assert (a.double() - b).abs().max() <= 4000 * 2.0 ** -24 * b.abs().max()


def test_the_long_way_gives_the_same_bits(mq, monkeypatch):
    import torch
    if mq._binding is None:
        pytest.skip("no extension module here")
    g = _gen(9)
    _, plan = _plan(mq, g, 30, 8, 3)
    x = torch.randn(30, 70, generator=g, device="cuda")
    w = torch.rand(30, 3, generator=g, device="cuda")
    m = torch.randn(8, 40, 70, generator=g, device="cuda")

    def calls():
        xl, wl = x.clone().requires_grad_(), w.clone().requires_grad_()
        rows = mq.experts_gather(xl, plan, wl)
        y = mq.experts_combine(rows, plan, wl, out_dtype=torch.bfloat16)
        grads = torch.autograd.grad(y, (xl, wl), torch.ones_like(y))
        wq = mq.w4_quantize(m, group=32, zeros=True)
        packed = mq.w4_pack(torch.arange(70 * 40, device="cuda").reshape(40, 70).to(torch.uint8) % 16,
                            torch.rand(40, 2, device="cuda", generator=_gen(1)).half(), group=64)
        return (rows, y, *grads, wq.codes, wq.scales, wq.zeros, mq.w4_dequantize(wq), packed.codes, packed.scales,
                mq.w4_linear(x, packed), mq.w4_experts_linear(x, wq, plan, by_token=True), mq.w4_experts_linear(rows.detach(), wq, plan))

    short = calls()
    for name in ("experts", "w4"):
        monkeypatch.setattr(f"dense_sparse_bit_amd.{name}._binding", None)
    for a, b in zip(calls(), short):
        assert a.dtype == b.dtype and torch.equal(a, b)


def test_a_graph_kept_freed_and_differentiated_twice(mq):
    """A kept graph gives the same again, a freed one and a second derivative are errors, and a
    thread of its own runs one while another goes on."""
    import threading
    import torch
    g = _gen(11)
    _, plan = _plan(mq, g, 20, 4, 2)
    x = torch.randn(20, 24, generator=g, device="cuda").requires_grad_()
    w = torch.rand(20, 2, generator=g, device="cuda").requires_grad_()
    dy = torch.randn(20, 24, generator=g, device="cuda")
    y = mq.experts_combine(mq.experts_gather(x, plan, w), plan, w)
    first = torch.autograd.grad(y, (x, w), dy, retain_graph=True)
    again = torch.autograd.grad(y, (x, w), dy)
    for a, b in zip(first, again):
        assert torch.equal(a, b)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(y, (x, w), dy)
    for d in (dy, dy.clone().requires_grad_()):
        y = mq.experts_combine(mq.experts_gather(x, plan, w), plan, w)
        dx, dw = torch.autograd.grad(y, (x, w), d, create_graph=True)
        assert torch.equal(dx, first[0]) and torch.equal(dw, first[1])
        for v in (dx, dw):
            with pytest.raises(RuntimeError):
                v.sum().backward(retain_graph=True)
    with torch.no_grad():
        assert not mq.experts_gather(x, plan, w).requires_grad
    results = [None] * 4

    def work(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            torch.cuda.current_stream().wait_stream(torch.cuda.default_stream())
            xl, wl = x.detach().clone().requires_grad_(), w.detach().clone().requires_grad_()
            for _ in range(10):
                y = mq.experts_combine(mq.experts_gather(xl, plan, wl), plan, wl)
                results[i] = torch.autograd.grad(y, (xl, wl), dy)
            torch.cuda.current_stream().synchronize()
    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for r in results:
        assert torch.equal(r[0], first[0]) and torch.equal(r[1], first[1])
