"""Every kernel instance that a dense product with group-scaled 4-bit weights can reach: each type of
rows, each group, with and without zero points, in each kernel of few rows and each tile.

Whole numbers: |x| <= 4 and |c - z| <= 15 over up to 7178 inputs are below 2^19 in all with scales
2^-6, exact in fp32 in any order, so outputs must be equal. Experts' products of few rows with long
rows likewise; those by tiles are in test_w4_ways.py."""
import pytest

TYPES = {"fp32": 0, "bf16": 1, "fp16": 2}
# (M, N, K, way of mq_w4_linear_way); columns and inputs that fill no tile
SIZES = {
    ("bf16", 32): [(1, 18, 67, 0), (5, 20, 67, 1), (231, 277, 805, 2), (49, 3521, 1802, 4), (151, 2535, 1690, 5), (298, 18, 67, 8),
        (2427, 18, 4064, 65), (1037, 11661, 77, 11)],
    ("bf16", 64): [(2, 17, 67, 0), (5, 18, 68, 1), (164, 373, 814, 2), (242, 808, 2329, 4), (211, 1719, 1893, 5), (266, 18, 67, 8),
        (2025, 17, 4580, 65), (178, 5252, 6561, 34), (2646, 6710, 66, 11), (966, 13945, 130, 12)],
    ("bf16", 128): [(1, 17, 67, 0), (5, 17, 65, 1), (218, 1926, 130, 2), (247, 803, 2705, 4), (177, 1902, 1976, 5), (272, 18, 69, 8),
        (2100, 19, 4178, 65), (34, 15833, 5782, 34), (1929, 9198, 69, 11), (1406, 17429, 79, 12)],
    ("fp16", 32): [(1, 17, 66, 0), (5, 17, 69, 1), (131, 465, 795, 2), (52, 3330, 1680, 4), (50, 5986, 1707, 5), (265, 19, 67, 8),
        (2166, 17, 4331, 65), (2010, 6041, 73, 11)],
    ("fp16", 64): [(2, 17, 65, 0), (7, 17, 66, 1), (230, 276, 777, 2), (18, 6737, 2131, 4), (85, 3717, 1990, 5), (268, 17, 68, 8),
        (1979, 19, 4534, 65), (215, 4024, 7178, 34), (1151, 15453, 67, 11), (2544, 9559, 68, 12)],
    ("fp16", 128): [(1, 17, 67, 0), (5, 17, 67, 1), (116, 3432, 129, 2), (212, 933, 2626, 4), (147, 2363, 1919, 5), (303, 17, 67, 8),
        (1960, 18, 4149, 65), (1946, 388, 5912, 34), (2244, 8147, 72, 11), (2529, 5763, 138, 12)],
    ("fp32", 32): [(2, 17, 66, 0), (5, 18, 66, 1), (132, 478, 655, 2), (268, 18, 66, 8), (2201, 17, 1447, 65), (468, 12711, 75, 11)],
    ("fp32", 64): [(1, 17, 69, 0), (6, 18, 67, 1), (204, 315, 642, 2), (282, 21, 66, 8), (1976, 21, 1333, 65), (2052, 193, 5286, 66),
        (1900, 5529, 68, 11), (1226, 10318, 67, 12)],
    ("fp32", 128): [(3, 17, 65, 0), (5, 18, 67, 1), (150, 412, 648, 2), (258, 17, 69, 8), (1975, 17, 1357, 65), (1992, 157, 3727, 66),
        (2516, 4036, 66, 11), (788, 17219, 67, 12)],
}
CASES = [(x_type, group, *size) for (x_type, group), sizes in SIZES.items() for size in sizes]
# one row, and up to four, in a kernel of their own
CASES += [(x_type, group, M, 50, 700, 0) for x_type in TYPES for group in (32, 64, 128) for M in (1, 4)]


def _kernel(way):
    return way if way < 8 else 8 + way % 8


def test_the_sizes_reach_every_kernel():
    """(host) The library takes the stated ways, and nothing else for any of 100000 other sizes."""
    import math
    import random
    import dense_sparse_bit_amd as mq
    way_of = mq.lib().mq_w4_linear_way
    for x_type, group, M, N, K, way in CASES:
        assert way_of(M, N, K, TYPES[x_type], group) == way
    there = {(x_type, group, _kernel(way)) for x_type, group, *_, way in CASES}
    rng = random.Random(0)
    size = lambda most: int(math.exp(rng.uniform(0, math.log(most))))
    for _ in range(100000):
        x_type, group = rng.choice(list(TYPES)), rng.choice((32, 64, 128))
        way = way_of(size(1 << 16), size(1 << 16), size(1 << 16), TYPES[x_type], group)
        assert (x_type, group, _kernel(way)) in there


@pytest.fixture(scope="module")
def mq():
    import torch
    assert torch.cuda.is_available()
    import dense_sparse_bit_amd
    return dense_sparse_bit_amd


def _weights(mq, g, shape, group, zeros):
    import torch
    codes = torch.randint(0, 16, shape, generator=g, device="cuda", dtype=torch.uint8)
    s = torch.full(shape[:-1] + (-(-shape[-1] // group),), 2.0 ** -6, device="cuda").half()
    z = torch.randint(0, 16, s.shape, generator=g, device="cuda").half() if zeros else None
    wide = 8 if z is None else z.double().repeat_interleave(group, -1)[..., :shape[-1]]
    return mq.w4_pack(codes, s, z, group=group), (codes.double() - wide) / 64


def _rows(g, M, K, x_type):
    import torch
    return torch.randint(-4, 5, (M, K), generator=g, device="cuda").to({"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}[x_type])


@pytest.mark.gpu
@pytest.mark.parametrize("x_type,group,M,N,K,way", CASES)
def test_every_instance_of_whole_numbers_is_exact(mq, x_type, group, M, N, K, way):
    import torch
    g = torch.Generator(device="cuda").manual_seed(M + N + K)
    for zeros in (False, True):
        w, values = _weights(mq, g, (N, K), group, zeros)
        x = _rows(g, M, K, x_type)
        want = (x.double() @ values.T.contiguous()).float()
        assert torch.equal(mq.w4_linear(x, w, out_dtype=torch.float32), want)


@pytest.mark.gpu
@pytest.mark.parametrize("x_type", list(TYPES))
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T,E,k,N,K", [(1, 4, 3, 50, 2300), (3, 6, 2, 70, 4100), (20, 8, 2, 100, 2300), (20, 8, 2, 100, 900)])
def test_experts_of_few_rows(mq, x_type, group, T, E, k, N, K):
    import torch
    g = torch.Generator(device="cuda").manual_seed(T + K)
    ids = torch.rand(T, E, generator=g, device="cuda").topk(k, 1).indices.int()
    plan = mq.expert_plan(ids, E)
    token = plan.row_token.long()
    offsets = plan.offsets.tolist()
    for zeros in (False, True):
        w, values = _weights(mq, g, (E, N, K), group, zeros)
        x = _rows(g, T, K, x_type)
        rows = torch.where((token >= 0)[:, None], x[token.clamp(min=0)], torch.zeros((), dtype=x.dtype, device="cuda"))
        want = torch.zeros(len(token), N, dtype=torch.float64, device="cuda")
        for e in range(E):
            at = slice(offsets[e], offsets[e + 1])
            want[at] = rows[at].double() @ values[e].T.contiguous()
        assert torch.equal(mq.w4_experts_linear(x, w, plan, by_token=True, out_dtype=torch.float32), want.float())
        assert torch.equal(mq.w4_experts_linear(rows, w, plan, out_dtype=torch.float32), want.float())
