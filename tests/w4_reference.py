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


# Products that between them take every way of the library's (type of x, group, M, N, K, way):
# few rows, tiles of each size, K in 1, 2, 4 and 8 parts; N and K that fit no tile.
WAYS = [("bf16", 32, 1, 50, 150, 0), ("fp32", 32, 4, 90, 200, 0), ("fp32", 128, 5, 20, 100, 1), ("fp16", 64, 13, 70, 1030, 1),
        ("bf16", 32, 3, 8211, 150, 1), ("fp16", 128, 64, 2049, 8190, 2), ("fp32", 128, 100, 4099, 1500, 2), ("bf16", 64, 64, 4100, 1030, 2),
        ("bf16", 64, 20, 33, 200, 1), ("fp16", 128, 64, 4090, 2050, 2), ("bf16", 32, 90, 3001, 4090, 4), ("fp16", 128, 250, 2050, 1027, 2),
        ("bf16", 128, 202, 2050, 8190, 5),
        ("bf16", 128, 301, 30, 100, 8), ("fp16", 64, 300, 17, 1030, 16), ("fp32", 128, 300, 20, 500, 16), ("bf16", 32, 299, 40, 2100, 32),
        ("fp16", 128, 290, 36, 4097, 64), ("bf16", 128, 770, 4100, 129, 9), ("fp16", 32, 1501, 8200, 140, 9),
        ("fp16", 32, 1003, 1030, 4090, 17), ("fp32", 32, 400, 1030, 1030, 33), ("fp16", 32, 2047, 33, 5130, 65),
        ("fp16", 64, 200, 16385, 8190, 10), ("fp32", 128, 1001, 4100, 4096, 10), ("fp32", 64, 200, 8208, 4096, 18),
        ("fp32", 128, 80, 8208, 5120, 34), ("fp32", 64, 60, 8190, 5119, 66), ("bf16", 32, 770, 12200, 4000, 11),
        ("bf16", 128, 2050, 12290, 160, 11), ("fp32", 32, 400, 12290, 2049, 19), ("fp16", 64, 80, 12300, 8192, 35),
        ("bf16", 32, 80, 8191, 8190, 67), ("fp32", 128, 80, 8190, 4095, 67), ("bf16", 128, 2047, 12287, 127, 12),
        ("fp32", 128, 1001, 16381, 130, 12), ("fp32", 128, 1000, 4095, 4094, 20), ("fp16", 128, 199, 8190, 8190, 36),
        ("fp32", 128, 199, 4093, 4095, 68)]
