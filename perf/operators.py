"""The microscaled 4-bit operators and the routing to experts: cases, plain forms, exact values.

Microscaled 4-bit format: 32 consecutive inputs of a row share a power-of-two scale
X = 2^(e - 127) (one byte e); each value is one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a
sign, times X. Quantization takes X = 2^(floor(log2(amax)) - 2), at least 2^-127, and
rounds value / X to the nearest of these, ties to the even code, values above 6 to 6.

Operators (entry points of dense_sparse_bit_amd):
  quantize  mx_quantize, mx_dequantize: a matrix to 4 bits and read back
  linear    mx_linear: y = Q(x) Q(w)^T + bias
  route     route, expert_plan: logits -> experts and weights of each token -> rows by expert
  up        mx_experts_up: h = silu(Q(x) Q(w_gate)^T) * (Q(x) Q(w_up)^T), each row with its expert
  down      mx_experts_down: y[t] = sum_j weight[t, j] * (Q(h[row(t, j)]) Q(w_down)^T)

run() computes the plain form (elementary torch operations, 32 bits; router scores in
64, because experts are chosen by comparing them) or, where `own` is true, calls the
library. exact() computes the same from the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # a ragged batch in fp32, a column slice of a wider matrix, a tail block of 8
        {"name": "quantize_ragged", "op": "quantize", "rows": 333, "cols": 5000, "dtype": "fp32", "strided": True},
        # a whole MLP weight matrix, as a loader quantizes it
        {"name": "quantize_weight", "op": "quantize", "rows": 17408, "cols": 5120, "dtype": "bf16", "strided": False},
        # one token through an attention projection
        {"name": "linear_token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "x": "bf16", "y": "bf16", "bias": False},
        # a decode batch through an MLP projection
        {"name": "linear_batch", "op": "linear", "M": 32, "N": 14336, "K": 4096, "x": "bf16", "y": "bf16", "bias": False},
        # sizes that fit no tile, with a bias and other types
        {"name": "linear_odd", "op": "linear", "M": 77, "N": 1001, "K": 1500, "x": "fp16", "y": "fp32", "bias": True},
        # a prefill chunk through the MLP up projection
        {"name": "linear_prefill", "op": "linear", "M": 2048, "N": 17408, "K": 5120, "x": "bf16", "y": "bf16",
         "bias": False},
        # routing of one decode token
        {"name": "route_token", "op": "route", "T": 1, "E": 128, "k": 8, "dtype": "bf16", "score": "softmax",
         "bias": False, "groups": 1, "top_groups": 1, "group_score": "max", "renormalize": True, "masked": False},
        # routing of a prefill chunk with a balancing bias and groups; some experts masked
        {"name": "route_prefill", "op": "route", "T": 4096, "E": 256, "k": 8, "dtype": "fp32", "score": "sigmoid",
         "bias": True, "groups": 8, "top_groups": 4, "group_score": "top2", "renormalize": True, "masked": True},
        # one decode token through its experts
        {"name": "up_token", "op": "up", "T": 1, "E": 64, "k": 8, "D": 4096, "I": 1024, "x": "bf16", "y": "bf16"},
        {"name": "down_token", "op": "down", "T": 1, "E": 64, "k": 8, "D": 4096, "I": 1024, "x": "bf16", "y": "bf16"},
        # a prefill chunk through the experts, uneven loads, some slots without an expert
        {"name": "up_prefill", "op": "up", "T": 4096, "E": 64, "k": 8, "D": 4096, "I": 1024, "x": "bf16", "y": "bf16"},
        {"name": "down_prefill", "op": "down", "T": 4096, "E": 64, "k": 8, "D": 4096, "I": 1024, "x": "bf16",
         "y": "bf16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "route", "up", "down"])
    kind = lambda: rng.choice(["bf16", "bf16", "fp32", "fp16"])
    if op == "quantize":
        cols = _log(rng, 32, 17408)
        rows = _log(rng, 1, min(17408, 17408 * 5120 // cols))
        return {"op": op, "rows": rows, "cols": cols, "dtype": kind(), "strided": rng.random() < 0.4}
    if op == "linear":
        K, N = _log(rng, 64, 14336), _log(rng, 16, 17408)
        M = _log(rng, 1, min(2048, 2048 * 17408 * 5120 // (N * K)))
        return {"op": op, "M": M, "N": N, "K": K, "x": kind(), "y": kind(), "bias": rng.random() < 0.4}
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, max(4, 8 // groups), 512 // groups)
        top = rng.randint(1, groups)
        k = rng.randint(1, min(16, top * (E // groups)))
        T = _log(rng, 1, min(16384, 4096 * 256 // E))
        return {"op": op, "T": T, "E": E, "k": k, "dtype": kind(), "score": rng.choice(["softmax", "sigmoid"]),
                "bias": rng.random() < 0.5, "groups": groups, "top_groups": top,
                "group_score": rng.choice(["max", "top2"]), "renormalize": rng.random() < 0.7,
                "masked": rng.random() < 0.4}
    E = _log(rng, 4, 64)
    k = rng.randint(1, min(8, E))
    T = _log(rng, 1, 4096)
    D, I = 8 * _log(rng, 16, 512), 8 * _log(rng, 8, 128)
    return {"op": op, "T": T, "E": E, "k": k, "D": D, "I": I, "x": kind(), "y": kind()}


# ------------------------------------------------------------------------------ work
def work(case):
    size = {"fp32": 4, "bf16": 2, "fp16": 2}
    fp4 = lambda r, c: r * c / 2 + r * math.ceil(c / 32)
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (size[case["dtype"]] + 2), "flops": 4 * n}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * size[case["x"]] + fp4(N, K) + M * N * size[case["y"]] + (4 * N if case["bias"] else 0),
                "flops": 2 * M * N * K}
    if op == "route":
        T, E, k = case["T"], case["E"], case["k"]
        return {"bytes": T * E * size[case["dtype"]] + T * k * (4 + 4 + 4 + 4) + 4 * E, "flops": 20 * T * E}
    T, E, k, D, I = (case[n] for n in ("T", "E", "k", "D", "I"))
    active = E * (1 - (1 - min(k / E, 1.0)) ** T)
    if op == "up":
        return {"bytes": 2 * active * fp4(I, D) + T * D * size[case["x"]] + T * k * I * size[case["y"]],
                "flops": 4 * T * k * D * I}
    return {"bytes": active * fp4(D, I) + T * k * I * size[case["x"]] + T * D * size[case["y"]] + 8 * T * k,
            "flops": 2 * T * k * D * I}


# ------------------------------------------------------------------------------ inputs
def _gen(seed, case):
    g = torch.Generator(device="cuda")
    g.manual_seed((int(seed) * 1000003 + sum(ord(c) for c in case["op"])) % (1 << 62))
    return g


def _activations(g, rows, cols, dtype):
    """Normal values, every hundredth channel or so ten times as large."""
    x = torch.randn(rows, cols, generator=g, device="cuda")
    big = torch.rand(cols, generator=g, device="cuda") < 0.01
    return (x * torch.where(big, 10.0, 1.0)).to(dtype)


def _weights(g, *shape):
    w = torch.randn(*shape, generator=g, device="cuda", dtype=torch.bfloat16)
    return w * (1.0 / math.sqrt(shape[-1]))


def _ids(g, case):
    """Experts of each token: distinct, some experts far more popular; for more than
    one token about one slot in fifty has none (-1)."""
    T, E, k = case["T"], case["E"], case["k"]
    logits = torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
    ids = logits.topk(k, dim=1).indices.to(torch.int32)
    if T > 1:
        ids = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.02, -1, ids).to(torch.int32)
    w = torch.rand(T, k, generator=g, device="cuda") + 0.1
    return ids.contiguous(), w / w.sum(1, keepdim=True)


def _inputs(case, seed):
    g = _gen(seed, case)
    op = case["op"]
    if op == "quantize":
        pad = 24 if case["strided"] else 0
        x = _activations(g, case["rows"], case["cols"] + pad, DTYPES[case["dtype"]])
        return {"x": x[:, 8:8 + case["cols"]] if pad else x}
    if op == "linear":
        bias = torch.randn(case["N"], generator=g, device="cuda") if case["bias"] else None
        return {"x": _activations(g, case["M"], case["K"], DTYPES[case["x"]]),
                "w": _weights(g, case["N"], case["K"]), "bias": bias}
    if op == "route":
        T, E = case["T"], case["E"]
        logits = 2 * torch.randn(T, E, generator=g, device="cuda") + torch.randn(E, generator=g, device="cuda")
        if case["masked"]:
            hide = torch.rand(T, E, generator=g, device="cuda") < 0.1
            hide[T // 2] = True                       # one token with no expert at all
            logits = torch.where(hide, -math.inf, logits)
        bias = 0.1 * torch.randn(E, generator=g, device="cuda") if case["bias"] else None
        return {"logits": logits.to(DTYPES[case["dtype"]]), "bias": bias}
    ids, weights = _ids(g, case)
    T, E, D, I = (case[n] for n in ("T", "E", "D", "I"))
    if op == "up":
        return {"x": _activations(g, T, D, DTYPES[case["x"]]), "ids": ids,
                "w_gate": _weights(g, E, I, D), "w_up": _weights(g, E, I, D)}
    total = plan_rows(T, case["k"], E)
    gate, up = torch.randn(2, total, I, generator=g, device="cuda")
    h = (gate * torch.sigmoid(gate) * up).to(DTYPES[case["x"]])
    return {"h": h, "ids": ids, "weights": weights, "w_down": _weights(g, E, D, I)}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import dense_sparse_bit_amd as mq
        s["mq"] = mq
        quantize, plan = mq.mx_quantize, mq.expert_plan
    else:
        quantize, plan = plain_quantize, plain_plan
    if "h" in s:                                       # rows of no token are zero
        row_token = plain_plan(s["ids"], case["E"])[1]
        s["h"][row_token < 0] = 0
    for name in ("w", "w_gate", "w_up", "w_down"):
        if name in s:
            s[name] = quantize(s[name])
    if case["op"] in ("up", "down"):
        s["plan"] = plan(s["ids"], case["E"])
    return s


# ------------------------------------------------------------------------------ run
def run(s):
    return _run_own(s, s["mq"]) if own else _run_plain(s)


def _run_own(s, mq):
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        return mq.mx_dequantize(mq.mx_quantize(s["x"]), dtype=torch.bfloat16)
    if op == "linear":
        return mq.mx_linear(s["x"], s["w"], bias=s["bias"], out_dtype=DTYPES[case["y"]])
    if op == "route":
        ids, weights = mq.route(s["logits"], case["k"], score=case["score"], bias=s["bias"], groups=case["groups"],
                                top_groups=case["top_groups"], group_score=case["group_score"],
                                renormalize=case["renormalize"])
        plan = mq.expert_plan(ids, case["E"])
        return ids, weights, plan.offsets, plan.row_token, plan.row_of
    if op == "up":
        return mq.mx_experts_up(s["x"], s["w_gate"], s["w_up"], s["plan"], out_dtype=DTYPES[case["y"]])
    return mq.mx_experts_down(s["h"], s["w_down"], s["plan"], s["weights"], out_dtype=DTYPES[case["y"]])


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        return plain_values(plain_quantize(s["x"])).to(torch.bfloat16)
    if op == "linear":
        y = plain_values(plain_quantize(s["x"])) @ plain_values(s["w"]).t()
        if s["bias"] is not None:
            y = y + s["bias"]
        return y.to(DTYPES[case["y"]])
    if op == "route":
        ids, weights = plain_route(s["logits"], s["bias"], case)
        return (ids, weights) + plain_plan(ids, case["E"])
    offsets, row_token, row_of = s["plan"]
    ids = s["ids"].long()
    if op == "up":
        x = plain_values(plain_quantize(s["x"]))
        h = torch.zeros(row_token.numel(), case["I"], device="cuda")
        for e in torch.unique(ids[ids >= 0]).tolist():
            t, j = torch.nonzero(ids == e, as_tuple=True)
            gate = x[t] @ plain_values(_expert(s["w_gate"], e)).t()
            up = x[t] @ plain_values(_expert(s["w_up"], e)).t()
            h[row_of[t, j].long()] = gate / (1 + torch.exp(-gate)) * up
        return h.to(DTYPES[case["y"]])
    h = plain_values(plain_quantize(s["h"]))
    y = torch.zeros(case["T"], case["D"], device="cuda")
    for e in torch.unique(ids[ids >= 0]).tolist():
        t, j = torch.nonzero(ids == e, as_tuple=True)
        y[t] += s["weights"][t, j][:, None] * (h[row_of[t, j].long()] @ plain_values(_expert(s["w_down"], e)).t())
    return y.to(DTYPES[case["y"]])


def _expert(w, e):
    codes, scales, cols = w
    return codes[e], scales[e], cols


def plan_rows(T, k, E):
    """Rows of an expert plan: each expert's rows start at a multiple of 16."""
    n = T * k
    return (n + 15 * min(n, E)) // 16 * 16


# ------------------------------------------------------------------------------ plain forms
def plain_quantize(x):
    """(codes, two to a byte, low nibble first; scale bytes; columns) of the last axis."""
    cols = x.shape[-1]
    v = x.float()
    if cols % 32:
        v = torch.nn.functional.pad(v, (0, 32 - cols % 32))
    v = v.reshape(*v.shape[:-1], -1, 32)
    exponent = torch.frexp(v.abs().amax(-1, keepdim=True)).exponent - 1 - 2
    exponent = torch.where(v.abs().amax(-1, keepdim=True) == 0, -127, exponent.clamp(-127))
    q = torch.ldexp(v.abs(), -exponent).clamp(max=6.0)
    step = torch.where(q < 2, 0.5, torch.where(q < 4, 1.0, 2.0))
    q = torch.round(q / step) * step
    code = sum((q >= value).to(torch.uint8) for value in VALUES[1:]) + 8 * torch.signbit(v).to(torch.uint8)
    code = code.reshape(*x.shape[:-1], -1)
    return code[..., 0::2] | (code[..., 1::2] << 4), (exponent[..., 0] + 127).to(torch.uint8), cols


def plain_values(a):
    codes, scales, cols = a
    code = torch.stack((codes & 15, codes >> 4), dim=-1).reshape(*codes.shape[:-1], -1, 32)
    table = torch.tensor(VALUES + tuple(-v for v in VALUES), device=codes.device)
    v = torch.ldexp(table[code.int()], scales.int()[..., None] - 127)
    return v.reshape(*codes.shape[:-1], -1)[..., :cols]


def plain_route(logits, bias, case):
    T, E = logits.shape
    k, groups = case["k"], case["groups"]
    x = logits.double()
    if case["score"] == "softmax":
        top = x.amax(1, keepdim=True)
        e = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
        score = e / e.sum(1, keepdim=True).clamp(min=1e-300)
    else:
        score = 1 / (1 + torch.exp(-x))
    # both scores grow with the logit: without a bias its own order is theirs
    order = x if bias is None else torch.where(x == -math.inf, -math.inf, score + bias.double())
    if case["top_groups"] < groups:
        if case["group_score"] == "max":
            value = order.reshape(T, groups, -1).amax(2)
        else:
            both = score if bias is None else score + bias.double()
            both = torch.where(order == -math.inf, -math.inf, both).reshape(T, groups, -1)
            best = both.sort(dim=2, descending=True).values[..., :2]
            value = torch.where(best == -math.inf, 0.0, best).sum(2)
            value = torch.where(best[..., 0] == -math.inf, -math.inf, value)
        rank = torch.sort(value, dim=1, descending=True, stable=True).indices.argsort(dim=1)
        keep = (rank < case["top_groups"]).repeat_interleave(E // groups, dim=1)
        order = torch.where(keep, order, -math.inf)
    value, ids = torch.sort(order, dim=1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    weights = torch.where(value == -math.inf, 0.0, score.gather(1, ids))
    ids = torch.where(value == -math.inf, -1, ids)
    if case["renormalize"]:
        total = weights.sum(1, keepdim=True)
        weights = torch.where(total > 0, weights / total, 0.0)
    return ids.to(torch.int32), weights.float()


def plain_plan(ids, E):
    """(offsets [E+1], row_token [rows], row_of [T, k]): rows by expert, in the order of
    the slots, each expert's rows from a multiple of 16 on; -1 where there is none."""
    T, k = ids.shape
    flat = ids.reshape(-1).long()
    valid = (flat >= 0) & (flat < E)
    key = torch.where(valid, flat, E)
    count = (key[:, None] == torch.arange(E, device=ids.device)).sum(0)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    offsets[1:] = ((count + 15) // 16 * 16).cumsum(0)
    slot = torch.sort(key, stable=True).indices
    first = torch.zeros(E + 1, dtype=torch.int64, device=ids.device)
    first[1:] = count.cumsum(0)
    k_sorted = key[slot]
    row = torch.where(k_sorted < E, offsets[k_sorted] + torch.arange(T * k, device=ids.device) - first[k_sorted], -1)
    row_of = torch.empty(T * k, dtype=torch.int64, device=ids.device)
    row_of[slot] = row
    row_token = torch.full((plan_rows(T, k, E) + 1,), -1, dtype=torch.int64, device=ids.device)
    row_token[row_of] = torch.where(valid, torch.arange(T * k, device=ids.device) // k, -1)
    row_token = row_token[:-1]
    return offsets.to(torch.int32), row_token.to(torch.int32), row_of.reshape(T, k).to(torch.int32)


# ------------------------------------------------------------------------------ exact values
def _nearest(x):
    """The values 4-bit codes and shared scales give x, in 64 bits: the nearest grid
    point by distance, the even code where two are as near."""
    cols = x.shape[-1]
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    grid = torch.tensor(VALUES, dtype=torch.float64, device=x.device)
    for c in range(0, cols, 32 * 64):
        part = x[..., c:c + 32 * 64].double()
        n = part.shape[-1]
        blocks = torch.zeros(*part.shape[:-1], -(-n // 32) * 32, dtype=torch.float64, device=x.device)
        blocks[..., :n] = part
        blocks = blocks.reshape(*part.shape[:-1], -1, 32)
        peak = blocks.abs().max(dim=-1, keepdim=True).values
        e = torch.floor(torch.log2(torch.where(peak > 0, peak, 1.0)))
        power = lambda n: torch.ldexp(torch.ones_like(n), n)
        e = torch.where(power(e) > peak, e - 1, e)      # log2 rounds next to a power of two
        e = torch.where(power(e + 1) <= peak, e + 1, e)
        scale = power(torch.where(peak > 0, e - 2, -127.0).clamp(min=-127.0))
        m = blocks.abs() / scale
        best = torch.zeros_like(m)
        for i in range(1, 8):
            middle = (grid[i - 1] + grid[i]) / 2
            up = (m > middle) | ((m == middle) & (i % 2 == 0))
            best = torch.where(up, grid[i], best)
        v = torch.copysign(best * scale, blocks)
        out[..., c:c + n] = v.reshape(*part.shape[:-1], -1)[..., :n]
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "quantize":
        return _nearest(s["x"])
    if op == "linear":
        y = torch.matmul(_nearest(s["x"]), _nearest(s["w"]).t().contiguous())
        return y if s["bias"] is None else y + s["bias"].double()
    if op == "route":
        return _exact_route(s, case)
    T, E, k = case["T"], case["E"], case["k"]
    slots = s["ids"].cpu().tolist()
    rows = _exact_rows(slots, E)
    if op == "up":
        x = _nearest(s["x"])
        h = torch.zeros(plan_rows(T, k, E), case["I"], dtype=torch.float64, device="cuda")
        for e, (start, members) in rows.items():
            xe = x[torch.tensor([t for t, _ in members], device="cuda")]
            gate = torch.matmul(xe, _nearest(s["w_gate"][e]).t().contiguous())
            up = torch.matmul(xe, _nearest(s["w_up"][e]).t().contiguous())
            h[start:start + len(members)] = gate * torch.special.expit(gate) * up
        return h
    y = torch.zeros(T, case["D"], dtype=torch.float64, device="cuda")
    for e, (start, members) in rows.items():
        o = torch.matmul(_nearest(s["h"][start:start + len(members)]), _nearest(s["w_down"][e]).t().contiguous())
        t = torch.tensor([t for t, _ in members], device="cuda")
        j = torch.tensor([j for _, j in members], device="cuda")
        y.index_add_(0, t, o * s["weights"].double()[t, j][:, None])
    return y


def _exact_rows(slots, E):
    """{expert: (first row, [(token, slot), ...])} of the experts that have rows."""
    members = {}
    for t, row in enumerate(slots):
        for j, e in enumerate(row):
            if 0 <= e < E:
                members.setdefault(e, []).append((t, j))
    out, start = {}, 0
    for e in sorted(members):
        out[e] = (start, members[e])
        start += -(-len(members[e]) // 16) * 16
    return out


def _exact_route(s, case):
    import numpy as np
    T, E, k, groups = case["T"], case["E"], case["k"], case["groups"]
    logits = s["logits"].double().cpu().numpy()
    bias = None if s["bias"] is None else s["bias"].double().cpu().numpy()
    per = E // groups
    ids, weights = np.full((T, k), -1, dtype=np.int32), np.zeros((T, k))
    for t in range(T):
        x = logits[t]
        live = np.flatnonzero(x > -math.inf)
        if not live.size:
            continue
        p = np.zeros(E)
        if case["score"] == "softmax":
            p[live] = np.exp(x[live] - x[live].max())
            p /= math.fsum(p)
        else:
            p[live] = 1.0 / (1.0 + np.exp(-x[live]))
        key = x if bias is None else np.where(x > -math.inf, p + bias, -math.inf)
        if case["top_groups"] < groups:
            worth = []
            for i in range(groups):
                mine = live[(live >= i * per) & (live < (i + 1) * per)]
                if not mine.size:
                    worth.append(-math.inf)
                elif case["group_score"] == "max":
                    worth.append(key[mine].max())
                else:
                    sums = p[mine] if bias is None else key[mine]
                    worth.append(np.sort(sums)[::-1][:2].sum())
            chosen = sorted(range(groups), key=lambda i: (-worth[i], i))[:case["top_groups"]]
            live = live[np.isin(live // per, chosen)]
        best = live[np.lexsort((live, -key[live]))][:k]
        w = p[best]
        if case["renormalize"] and w.sum() > 0:
            w = w / w.sum()
        ids[t, :len(best)], weights[t, :len(best)] = best, w
    rows = _exact_rows(ids.tolist(), E)
    offsets = np.zeros(E + 1, dtype=np.int32)
    row_token = np.full(plan_rows(T, k, E), -1, dtype=np.int32)
    row_of = np.full((T, k), -1, dtype=np.int32)
    for e, (start, members) in rows.items():
        offsets[e + 1] = -(-len(members) // 16) * 16
        for i, (t, j) in enumerate(members):
            row_token[start + i], row_of[t, j] = t, start + i
    offsets = np.cumsum(offsets, dtype=np.int32)
    put = lambda a: torch.from_numpy(a).cuda()
    return put(ids), put(weights), put(offsets), put(row_token), put(row_of)
