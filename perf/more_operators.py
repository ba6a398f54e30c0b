"""Products with group-scaled 4-bit weights, tokens by expert and back: cases, plain forms, exact values.

Group-scaled 4-bit weights: g = 32, 64 or 128 consecutive inputs of a row share a 16-bit
scale s and zero point z (8 where there are no zero points); a weight is s * (code - z),
its code 0 .. 15. Quantization without zero points: s = max|w| / 7, code =
round(w / s) + 8; with them: s = (hi - lo) / 15 over the group's range with 0 in it,
z = round(-lo / s), code = round(w / s) + z; ties to even, codes clamped to 0 .. 15.

Operators (entry points of dense_sparse_bit_amd):
  quantize  w4_quantize, w4_dequantize: a matrix to such weights and read back
  linear    w4_linear: y = x W^T + bias, x as it is
  experts   w4_experts_linear: the same for the rows of a plan, each with its expert's matrix
  gather    experts_gather: each token's row to the rows of its experts, with its gradient
  combine   experts_combine: y[t] = sum_j weight[t, j] * row(t, j), with its gradient

run() computes the plain form (elementary torch operations, 32 bits) or, where `own` is
true, calls the library. exact() computes the same from the definition in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
SIZE = {"fp32": 4, "bf16": 2, "fp16": 2}


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # a ragged batch in fp32, a column slice of a wider matrix, a last group of 8, with zero points
        {"name": "quantize_ragged", "op": "quantize", "rows": 333, "cols": 5000, "group": 64, "zeros": True, "scale": "bf16",
         "x": "fp32", "y": "fp32", "strided": True},
        # a whole MLP weight matrix, as a loader quantizes it
        {"name": "quantize_weight", "op": "quantize", "rows": 17408, "cols": 5120, "group": 128, "zeros": False,
         "scale": "fp16", "x": "bf16", "y": "bf16", "strided": False},
        # one token through an attention projection
        {"name": "linear_token", "op": "linear", "M": 1, "N": 4096, "K": 4096, "group": 128, "zeros": False, "scale": "fp16",
         "x": "bf16", "y": "bf16", "bias": False},
        # a decode batch through an MLP projection, weights with zero points
        {"name": "linear_batch", "op": "linear", "M": 32, "N": 14336, "K": 4096, "group": 128, "zeros": True, "scale": "fp16",
         "x": "bf16", "y": "bf16", "bias": False},
        # sizes that fit no tile, small groups, a bias and other types
        {"name": "linear_odd", "op": "linear", "M": 77, "N": 1001, "K": 1500, "group": 32, "zeros": True, "scale": "bf16",
         "x": "fp16", "y": "fp32", "bias": True},
        # a prefill chunk through the MLP up projection
        {"name": "linear_prefill", "op": "linear", "M": 2048, "N": 17408, "K": 5120, "group": 128, "zeros": False,
         "scale": "fp16", "x": "bf16", "y": "bf16", "bias": False},
        # one decode token through its experts
        {"name": "experts_token", "op": "experts", "T": 1, "E": 64, "k": 8, "N": 1024, "K": 4096, "by_token": True,
         "group": 128, "zeros": False, "scale": "fp16", "x": "bf16", "y": "bf16"},
        # a prefill chunk's rows through their experts, uneven loads, some slots without an expert
        {"name": "experts_prefill", "op": "experts", "T": 4096, "E": 64, "k": 8, "N": 4096, "K": 1024, "by_token": False,
         "group": 64, "zeros": True, "scale": "bf16", "x": "bf16", "y": "bf16"},
        # one decode token to the rows of its experts
        {"name": "gather_token", "op": "gather", "T": 1, "E": 64, "k": 8, "D": 4096, "x": "bf16", "weighted": False,
         "grad": False},
        # a training batch to its experts' rows, and the gradient back to the tokens
        {"name": "gather_train", "op": "gather", "T": 4096, "E": 64, "k": 8, "D": 4096, "x": "bf16", "weighted": False,
         "grad": True},
        # a small ragged batch's rows back to its tokens
        {"name": "combine_small", "op": "combine", "T": 37, "E": 8, "k": 2, "D": 4096, "x": "bf16", "y": "bf16",
         "grad": False},
        # a training batch's rows back to its tokens, gradients of rows and weights
        {"name": "combine_train", "op": "combine", "T": 4096, "E": 64, "k": 8, "D": 4096, "x": "bf16", "y": "bf16",
         "grad": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "experts", "gather", "combine"])
    kind = lambda: rng.choice(["bf16", "bf16", "fp32", "fp16"])
    weights = {"group": rng.choice([32, 64, 128, 128]), "zeros": rng.random() < 0.5, "scale": rng.choice(["fp16", "bf16"])}
    if op == "quantize":
        cols = _log(rng, 32, 17408)
        rows = _log(rng, 1, min(17408, 17408 * 5120 // (2 * cols)))
        return {"op": op, "rows": rows, "cols": cols, **weights, "x": kind(), "y": kind(), "strided": rng.random() < 0.4}
    if op == "linear":
        x = kind()
        K, N = _log(rng, 64, 14336), _log(rng, 16, 17408)
        most = 2048 * 17408 * 5120 // (N * K * (3 if x == "fp32" else 1))
        return {"op": op, "M": _log(rng, 1, min(2048, most)), "N": N, "K": K, **weights, "x": x, "y": kind(),
                "bias": rng.random() < 0.4}
    E = _log(rng, 4, 64)
    k = rng.randint(1, min(8, E))
    if op == "experts":
        T, N, K = _log(rng, 1, 4096), _log(rng, 64, 4096), _log(rng, 64, 4096)
        x = kind()
        T = max(1, min(T, 4096 * 8 * 4096 * 1024 // (k * N * K * (3 if x == "fp32" else 1))))
        return {"op": op, "T": T, "E": E, "k": k, "N": N, "K": K, "by_token": rng.random() < 0.5, **weights, "x": x,
                "y": kind()}
    x, D = kind(), _log(rng, 64, 8192)
    T = _log(rng, 1, min(8192, 4096 * 8 * 4096 * 2 // (k * D * SIZE[x])))
    case = {"op": op, "T": T, "E": E, "k": k, "D": D, "x": x}
    if op == "gather":
        return {**case, "weighted": rng.random() < 0.3, "grad": rng.random() < 0.6}
    return {**case, "y": kind(), "grad": rng.random() < 0.6}


# ------------------------------------------------------------------------------ work
def _weight_bytes(case, N, K):
    return N * K / 2 + N * math.ceil(K / case["group"]) * (4 if case["zeros"] else 2)


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return {"bytes": n * (SIZE[case["x"]] + SIZE[case["y"]]), "flops": 4 * n}
    if op == "linear":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": M * K * SIZE[case["x"]] + _weight_bytes(case, N, K) + M * N * SIZE[case["y"]]
                + (4 * N if case["bias"] else 0), "flops": 2 * M * N * K}
    T, E, k = case["T"], case["E"], case["k"]
    rows = plan_rows(T, k, E)
    if op == "experts":
        N, K = case["N"], case["K"]
        active = E * (1 - (1 - min(k / E, 1.0)) ** T)
        return {"bytes": active * _weight_bytes(case, N, K) + (T if case["by_token"] else T * k) * K * SIZE[case["x"]]
                + rows * N * SIZE[case["y"]], "flops": 2 * T * k * N * K}
    D, size = case["D"], SIZE[case["x"]]
    if op == "gather":
        forward, backward = (T + rows) * D * size, (T * k + T) * D * size
        scale = 2 if case["weighted"] else 1
        return {"bytes": forward + (backward if case["grad"] else 0), "flops": T * k * D * (scale + (2 * scale if case["grad"] else 0))}
    forward, backward = T * k * D * size + T * D * SIZE[case["y"]], T * D * SIZE[case["y"]] + rows * D * size
    return {"bytes": forward + (backward if case["grad"] else 0), "flops": T * k * D * (5 if case["grad"] else 2)}


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


def _codes(g, case, *shape):
    """Codes, scales and zero points as a checkpoint holds them: [..., N, K] and [..., N, groups]."""
    kind = DTYPES[case["scale"]]
    codes = torch.randint(0, 16, shape, generator=g, device="cuda", dtype=torch.uint8)
    per = shape[:-1] + (-(-shape[-1] // case["group"]),)
    scales = ((0.5 + torch.rand(per, generator=g, device="cuda")) * (0.2 / math.sqrt(shape[-1]))).to(kind)
    zeros = torch.randint(4, 12, per, generator=g, device="cuda").to(kind) if case["zeros"] else None
    return codes, scales, zeros


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
        x = (_activations(g, case["rows"], case["cols"] + pad, torch.float32) / math.sqrt(case["cols"])).to(DTYPES[case["x"]])
        return {"x": x[:, 8:8 + case["cols"]] if pad else x}
    if op == "linear":
        bias = torch.randn(case["N"], generator=g, device="cuda") if case["bias"] else None
        return {"x": _activations(g, case["M"], case["K"], DTYPES[case["x"]]), "w": _codes(g, case, case["N"], case["K"]),
                "bias": bias}
    ids, weights = _ids(g, case)
    T, E = case["T"], case["E"]
    rows = plan_rows(T, case["k"], E)
    if op == "experts":
        x = _activations(g, T if case["by_token"] else rows, case["K"], DTYPES[case["x"]])
        return {"x": x, "ids": ids, "w": _codes(g, case, E, case["N"], case["K"])}
    D, kind = case["D"], DTYPES[case["x"]]
    normal = lambda n, t: torch.randn(n, D, generator=g, device="cuda").to(t)
    if op == "gather":
        return {"x": normal(T, kind), "ids": ids, "weights": weights if case["weighted"] else None,
                "given": normal(rows, kind) if case["grad"] else None}
    return {"rows": normal(rows, kind), "ids": ids, "weights": weights,
            "given": normal(T, DTYPES[case["y"]]) if case["grad"] else None}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import dense_sparse_bit_amd as mq
        s["mq"] = mq
        if "w" in s:
            s["w"] = mq.w4_pack(*s["w"], group=case["group"])
        if "ids" in s:
            s["plan"] = mq.expert_plan(s["ids"], case["E"])
        if case.get("grad"):
            for name in ("x", "rows", "weights"):
                if s.get(name) is not None:
                    s[name].requires_grad_()
    elif "ids" in s:
        s["plan"] = plain_plan(s["ids"], case["E"])
    return s


# ------------------------------------------------------------------------------ run
def run(s):
    return _run_own(s, s["mq"]) if own else _run_plain(s)


def _run_own(s, mq):
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        w = mq.w4_quantize(s["x"], group=case["group"], zeros=case["zeros"], scale_dtype=DTYPES[case["scale"]])
        return mq.w4_dequantize(w, dtype=DTYPES[case["y"]])
    if op == "linear":
        return mq.w4_linear(s["x"], s["w"], bias=s["bias"], out_dtype=DTYPES[case["y"]])
    if op == "experts":
        return mq.w4_experts_linear(s["x"], s["w"], s["plan"], by_token=case["by_token"], out_dtype=DTYPES[case["y"]])
    if op == "gather":
        rows = mq.experts_gather(s["x"], s["plan"], weights=s["weights"])
        if not case["grad"]:
            return rows
        leaves = (s["x"],) if s["weights"] is None else (s["x"], s["weights"])
        return (rows.detach(),) + torch.autograd.grad(rows, leaves, s["given"])
    y = mq.experts_combine(s["rows"], s["plan"], s["weights"], out_dtype=DTYPES[case["y"]])
    if not case["grad"]:
        return y
    return (y.detach(),) + torch.autograd.grad(y, (s["rows"], s["weights"]), s["given"])


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "quantize":
        return plain_values(*plain_quantize(s["x"], case), case["group"]).to(DTYPES[case["y"]])
    if op == "linear":
        y = s["x"].float() @ plain_values(*s["w"], case["group"]).t()
        if s["bias"] is not None:
            y = y + s["bias"]
        return y.to(DTYPES[case["y"]])
    offsets, row_token, row_of = s["plan"]
    ids = s["ids"].long()
    live = (ids >= 0) & (ids < case["E"])
    t, j = torch.nonzero(live, as_tuple=True)
    p = row_of[t, j].long()
    if op == "experts":
        codes, scales, zeros = s["w"]
        x = s["x"].float()
        y = torch.zeros(row_token.numel(), case["N"], device="cuda")
        for e in torch.unique(ids[live]).tolist():
            mine = ids[t, j] == e
            w = plain_values(codes[e], scales[e], None if zeros is None else zeros[e], case["group"])
            y[p[mine]] = x[t[mine] if case["by_token"] else p[mine]] @ w.t()
        return y.to(DTYPES[case["y"]])
    weights = s["weights"]
    if op == "gather":
        x = s["x"].float()
        v = x[t] if weights is None else x[t] * weights[t, j][:, None]
        rows = torch.zeros(row_token.numel(), case["D"], device="cuda")
        rows[p] = v
        rows = rows.to(s["x"].dtype)
        if not case["grad"]:
            return rows
        back = torch.zeros(case["T"], case["k"], case["D"], device="cuda")
        back[t, j] = s["given"][p].float()
        dx = (back if weights is None else back * weights[:, :, None]).sum(1).to(s["x"].dtype)
        return (rows, dx) if weights is None else (rows, dx, (back * x[:, None, :]).sum(2))
    rows = torch.zeros(case["T"], case["k"], case["D"], device="cuda")
    rows[t, j] = s["rows"][p].float()
    y = (rows * weights[:, :, None]).sum(1).to(DTYPES[case["y"]])
    if not case["grad"]:
        return y
    dy = s["given"].float()
    drows = torch.zeros(row_token.numel(), case["D"], device="cuda")
    drows[p] = dy[t] * weights[t, j][:, None]
    return y, drows.to(s["rows"].dtype), (rows * dy[:, None, :]).sum(2)


def plan_rows(T, k, E):
    """Rows of an expert plan: each expert's rows start at a multiple of 16."""
    n = T * k
    return (n + 15 * min(n, E)) // 16 * 16


# ------------------------------------------------------------------------------ plain forms
def _groups(x, group):
    """The last axis in whole groups, zeros behind its end."""
    pad = -x.shape[-1] % group
    if pad:
        x = torch.nn.functional.pad(x, (0, pad))
    return x.reshape(*x.shape[:-1], -1, group)


def plain_quantize(x, case):
    """(codes, one to a byte; scales; zero points or None) of the last axis. Quotients are
    taken in 64 bits, because a scale or a code next to a border goes by them."""
    kind = DTYPES[case["scale"]]
    v = _groups(x.float(), case["group"])
    if case["zeros"]:
        lo, hi = v.amin(-1).clamp(max=0), v.amax(-1).clamp(min=0)
        scales = ((hi - lo).double() / 15).float().to(kind)
    else:
        scales = (v.abs().amax(-1).double() / 7).float().to(kind)
    step = torch.where(scales == 0, 1.0, scales.double())
    zeros = torch.round(-lo.double() / step).clamp(0, 15) if case["zeros"] else torch.full_like(step, 8)
    codes = (torch.round(v.double() / step[..., None]) + zeros[..., None]).clamp(0, 15)
    codes = codes.reshape(*x.shape[:-1], -1)[..., :x.shape[-1]].to(torch.uint8)
    return codes, scales, zeros.to(kind) if case["zeros"] else None


def plain_values(codes, scales, zeros, group):
    v = _groups(codes, group).float()
    v = (v - (8.0 if zeros is None else zeros.float()[..., None])) * scales.float()[..., None]
    return v.reshape(*codes.shape[:-1], -1)[..., :codes.shape[-1]]


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
def _exact_weights(codes, scales, zeros, group):
    """The weights in 64 bits, group by group."""
    w = codes.double()
    for i in range(scales.shape[-1]):
        part = w[..., i * group:(i + 1) * group]
        part -= 8.0 if zeros is None else zeros[..., i:i + 1].double()
        part *= scales[..., i:i + 1].double()
    return w


def _exact_quantize(x, case):
    group, kind = case["group"], DTYPES[case["scale"]]
    out = torch.empty(x.shape, dtype=torch.float64, device=x.device)
    for c in range(0, x.shape[-1], group):
        v = x[:, c:c + group].double()
        if case["zeros"]:
            lo, hi = v.min(1, keepdim=True).values.clamp(max=0), v.max(1, keepdim=True).values.clamp(min=0)
            s = ((hi - lo).float().double() / 15).float().to(kind).double()
        else:
            s = (v.abs().max(1, keepdim=True).values / 7).float().to(kind).double()
        live = s > 0
        q = torch.where(live, v / torch.where(live, s, 1.0), 0.0)
        nearest = torch.floor(q + 0.5)
        nearest = torch.where((q + 0.5 == nearest) & (nearest % 2 != 0), nearest - 1, nearest)
        low = torch.full_like(s, -8.0)
        if case["zeros"]:
            z = torch.where(live, -lo / torch.where(live, s, 1.0), 0.0)
            up = torch.floor(z + 0.5)
            up = torch.where((z + 0.5 == up) & (up % 2 != 0), up - 1, up)
            low = -torch.minimum(up, torch.full_like(up, 15.0))
        out[:, c:c + group] = torch.minimum(torch.maximum(nearest, low), low + 15) * s
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op == "quantize":
        return _exact_quantize(s["x"], case)
    if op == "linear":
        y = torch.matmul(s["x"].double(), _exact_weights(*s["w"], case["group"]).t().contiguous())
        return y if s["bias"] is None else y + s["bias"].double()
    T, E, k = case["T"], case["E"], case["k"]
    slots = s["ids"].cpu().tolist()
    experts = _exact_rows(slots, E)
    total = plan_rows(T, k, E)
    put = lambda a: torch.tensor(a, dtype=torch.int64, device="cuda")
    if op == "experts":
        codes, scales, zeros = s["w"]
        y = torch.zeros(total, case["N"], dtype=torch.float64, device="cuda")
        for e, (start, members) in experts.items():
            n = len(members)
            x = s["x"][put([t for t, _ in members])] if case["by_token"] else s["x"][start:start + n]
            w = _exact_weights(codes[e], scales[e], None if zeros is None else zeros[e], case["group"])
            y[start:start + n] = torch.matmul(x.double(), w.t().contiguous())
        return y
    weights = None if s["weights"] is None else s["weights"].double()
    D = case["D"]
    zero = lambda *n: torch.zeros(*n, dtype=torch.float64, device="cuda")
    rows, dx, dweights, y, drows = zero(total, D), zero(T, D), zero(T, k), zero(T, D), zero(total, D)
    for start, members in experts.values():
        n = len(members)
        t, j = put([t for t, _ in members]), put([j for _, j in members])
        v = zero(n, 1) + 1.0 if weights is None else weights[t, j][:, None]
        if op == "gather":
            x = s["x"][t].double()
            rows[start:start + n] = v * x
            if case["grad"]:
                given = s["given"][start:start + n].double()
                dx.index_add_(0, t, v * given)
                dweights[t, j] = torch.linalg.vecdot(x, given)
        else:
            r = s["rows"][start:start + n].double()
            y.index_add_(0, t, v * r)
            if case["grad"]:
                given = s["given"][t].double()
                drows[start:start + n] = v * given
                dweights[t, j] = torch.linalg.vecdot(r, given)
    if op == "gather":
        if not case["grad"]:
            return rows
        return (rows, dx) if weights is None else (rows, dx, dweights)
    return (y, drows, dweights) if case["grad"] else y


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
