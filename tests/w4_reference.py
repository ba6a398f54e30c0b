"""Plain 64-bit statements of the group-scaled 4-bit format on the host (numpy), sharing
nothing with the library."""
import numpy as np

MAX16 = {"fp16": 65504.0, "bf16": float(np.ldexp(255.0, 120))}


def round16(v, kind):
    """fp64 values that fp32 holds, rounded to fp16 or bf16 (ties to even)."""
    if kind == "fp16":
        with np.errstate(over="ignore"):
            return v.astype(np.float32).astype(np.float16).astype(np.float64)
    bits = v.astype(np.float32).view(np.uint32).astype(np.uint64)
    bits = (bits + 0x7fff + (bits >> 16 & 1)) & 0xffff0000
    return bits.astype(np.uint32).view(np.float32).astype(np.float64)


def _div32(a, b):
    """fp32 a / b, rounded once."""
    return (a / b).astype(np.float32).astype(np.float64)


def quantize(x, group, kind, with_zeros):
    """(codes [R, K], scales, zeros [R, groups] or None) of x [R, K] float64 (fp32 values)."""
    R, K = x.shape
    n = -(-K // group)
    codes = np.zeros((R, K), dtype=np.uint8)
    scales, zeros = np.zeros((R, n)), np.full((R, n), 0.0 if with_zeros else 8.0)
    for g in range(n):
        v = x[:, g * group:(g + 1) * group]
        bad = ~np.isfinite(v).all(1)
        v = np.where(bad[:, None], 0.0, v)
        if with_zeros:
            lo, hi = np.minimum(v.min(1), 0), np.maximum(v.max(1), 0)
            with np.errstate(over="ignore"):
                s = _div32((hi - lo).astype(np.float32).astype(np.float64), 15.0)
        else:
            s = _div32(np.abs(v).max(1), 7.0)
        s = round16(np.minimum(s, MAX16[kind]), kind)
        safe = np.where(s > 0, s, 1.0)
        z = np.where(s > 0, np.clip(np.rint(-lo / safe), 0, 15), 0.0) if with_zeros else np.full(R, 8.0)
        q = np.where(s[:, None] > 0, np.rint(v / safe[:, None]), 0.0)
        codes[:, g * group:(g + 1) * group] = np.where(bad[:, None], z[:, None] * 0 + (0 if with_zeros else 8),
                                                       np.clip(q + z[:, None], 0, 15))
        scales[:, g] = np.where(bad, np.nan, s)
        zeros[:, g] = np.where(bad, 0.0 if with_zeros else 8.0, z)
    return codes, scales, zeros if with_zeros else None


def values(codes, scales, zeros, group):
    K = codes.shape[-1]
    s = np.repeat(scales, group, axis=-1)[..., :K]
    z = 8.0 if zeros is None else np.repeat(zeros, group, axis=-1)[..., :K]
    return (codes.astype(np.float64) - z) * s


def pack(codes):
    """The bytes of codes [R, K] in the library's layout: [row tiles, column tiles, 1024]."""
    R, K = codes.shape
    RT, G = -(-R // 16), -(-K // 128)
    c = np.zeros((RT * 16, G * 128), dtype=np.uint8)
    c[:R, :K] = codes
    # [tile, row, tile, word, quarter, half, byte] -> [tile, tile, quarter, row, word, byte]
    c = c.reshape(RT, 16, G, 4, 4, 2, 4)
    b = c[..., 0, :] | c[..., 1, :] << 4
    return np.ascontiguousarray(b.transpose(0, 2, 4, 1, 3, 5)).reshape(RT, G, 1024)


def pack_scales(s, R, K, group):
    """[R, ceil(K/group)] in the library's layout [row tiles, quads, 16, 512/group]."""
    RT, Q, per = -(-R // 16), -(-K // 512), 512 // group
    out = np.zeros((RT * 16, Q * per))
    out[:R, :s.shape[1]] = s
    return out.reshape(RT, 16, Q, per).transpose(0, 2, 1, 3)
