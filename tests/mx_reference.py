"""Plain 64-bit statements of the microscaled format, the routing and the plan, on the
host (numpy), sharing nothing with the library."""
import math

import numpy as np

GRID = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=np.float64)


def quantize(x):
    """(code index 0..15, scale byte) of x [R, K] float64: codes [R, K], bytes [R, ceil(K/32)].
    A block with a NaN or an infinity has byte 255 and codes 0."""
    R, K = x.shape
    nb = -(-K // 32)
    codes = np.zeros((R, K), dtype=np.uint8)
    scale = np.zeros((R, nb), dtype=np.uint8)
    for r in range(R):
        for b in range(nb):
            v = x[r, 32 * b:32 * b + 32]
            if not np.isfinite(v).all():
                scale[r, b] = 255
                continue
            peak = np.abs(v).max()
            e = max(math.frexp(peak)[1] - 3, -127) if peak > 0 else -127
            scale[r, b] = e + 127
            m = np.abs(v) / 2.0 ** e
            c = np.zeros(len(v), dtype=np.uint8)
            for i in range(1, 8):
                mid = (GRID[i - 1] + GRID[i]) / 2
                c[(m > mid) | ((m == mid) & (i % 2 == 0))] = i
            codes[r, 32 * b:32 * b + 32] = c + 8 * np.signbit(v)
    return codes, scale


def values(codes, scale):
    v = GRID[codes & 7] * np.where(codes & 8, -1.0, 1.0)
    s = np.repeat(scale.astype(np.int64), 32, axis=1)[:, :codes.shape[1]]
    return np.where(s == 255, np.nan, np.ldexp(v, s - 127))


def pack(codes, scale):
    """The device layout of include/mq.h, element by element from its formulas."""
    R, K = codes.shape
    RT, G = -(-R // 16), -(-K // 128)
    G4 = -(-G // 4)
    c = np.zeros(RT * G * 1024, dtype=np.uint8)
    s = np.zeros(RT * G4 * 256, dtype=np.uint8)
    r, k = np.meshgrid(np.arange(R), np.arange(K), indexing="ij")
    at = (((r // 16) * G + k // 128) * 64 + ((k // 32) % 4) * 16 + r % 16) * 16 + (k % 32) // 2
    np.add.at(c, at.ravel(), (codes << (4 * (k % 2))).astype(np.uint8).ravel())
    r, b = np.meshgrid(np.arange(R), np.arange(scale.shape[1]), indexing="ij")
    k = 32 * b
    s[(((r // 16) * G4 + k // 512) * 64 + ((k // 32) % 4) * 16 + r % 16) * 4 + (k // 128) % 4] = scale
    return c.reshape(RT, G, 1024), s.reshape(RT, G4, 256)


def route(logits, k, score, bias, groups, top_groups, group_score, renormalize, scale=1.0):
    T, E = logits.shape
    ids, weights = np.full((T, k), -1, dtype=np.int32), np.zeros((T, k))
    per = E // groups
    for t in range(T):
        x = logits[t]
        with np.errstate(all="ignore"):
            if score == "softmax":
                top = x.max() if x.max() > -math.inf else 0.0
                p = np.exp(x - top)
                p = p / p.sum() if p.sum() != 0 else p
            else:
                p = 1 / (1 + np.exp(-x))
            both = p if bias is None else p + bias
        key = np.where(x == -math.inf, -math.inf, x if bias is None else both)
        if np.isnan(key).any() or np.isnan(p).any():
            weights[t] = math.nan
            continue
        live = [e for e in range(E) if key[e] > -math.inf]
        if top_groups < groups:
            worth = []
            for g in range(groups):
                mine = [e for e in live if e // per == g]
                if not mine:
                    worth.append(-math.inf)
                elif group_score == "max":
                    worth.append(max(key[e] for e in mine))
                else:
                    worth.append(sum(sorted((both[e] for e in mine), reverse=True)[:2]))
            keep = sorted(range(groups), key=lambda g: (-worth[g], g))[:top_groups]
            live = [e for e in live if e // per in keep]
        best = sorted(live, key=lambda e: (-key[e], e))[:k]
        w = p[best]
        if renormalize:
            w = w / w.sum() if w.sum() > 0 else 0 * w
        ids[t, :len(best)] = best
        weights[t, :len(best)] = w * scale
    return ids, weights


def plan(ids, E):
    T, k = ids.shape
    n = T * k
    rows = (n + 15 * min(n, E)) // 16 * 16
    offsets = np.zeros(E + 1, dtype=np.int32)
    row_token, row_of = np.full(rows, -1, dtype=np.int32), np.full((T, k), -1, dtype=np.int32)
    for e in range(E):
        slots = [(t, j) for t in range(T) for j in range(k) if ids[t, j] == e]
        for i, (t, j) in enumerate(slots):
            row_token[offsets[e] + i] = t
            row_of[t, j] = offsets[e] + i
        offsets[e + 1] = offsets[e] + -(-len(slots) // 16) * 16
    return offsets, row_token, row_of
