"""Every kernel of the 4-bit products that a plan can choose (test_w4_plan.py
holds the list and counts what these sizes reach), with more stages than its
ring holds: against the definition in 64 bits, and equal for integers."""
import pytest
import torch

import dense_ref as D
import experts_ref as R
import trellis_quantized_moe_exl3_amd as M
from test_gpu_w4 import TYPES, _gen, _offsets, _run, _split, _stack

pytestmark = pytest.mark.gpu

# rows, K, N, experts, group
TILES = [(1, 4352, 8, 1, 128), (1, 4544, 8, 16, 64), (1, 4672, 8, 3, 32), (2, 4224, 3968, 14, 128), (3, 4352, 2552, 7, 32),
         (3, 5568, 2624, 13, 64), (5, 4224, 2248, 1, 128), (5, 64, 11248, 58, 64), (10, 128, 5432, 52, 128),
         (14, 32, 4024, 26, 32), (18, 4928, 6080, 1, 64), (25, 4416, 4056, 1, 32), (37, 4224, 3800, 1, 32),
         (37, 5248, 288, 11, 128), (249, 448, 3200, 12, 64), (285, 448, 3264, 10, 32), (461, 2304, 472, 53, 64),
         (463, 4864, 24, 37, 64), (508, 4160, 232, 1, 64), (526, 704, 11768, 1, 32), (585, 2240, 408, 57, 32),
         (930, 512, 1200, 59, 128), (1158, 512, 5224, 1, 128), (1196, 448, 6152, 1, 64), (1199, 5600, 8, 28, 32),
         (1242, 4256, 8, 1, 32), (1297, 4160, 8, 1, 64), (2500, 2560, 56, 56, 128), (3247, 2560, 56, 56, 128),
         (3876, 4352, 24, 1, 128), (5859, 4480, 24, 5, 128)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("T,K,N,E,group", TILES)
def test_tiles(T, K, N, E, group, glu, dtype):
    g = _gen(T + K + N)
    d = M.make_w4_desc(K, N, E, group, D.DT[dtype], M.ACT_GELU_TANH)
    x, _ = D.inside(D.gauss(g, (T, K), 1.0, dtype))
    base = None if glu else D.inside(D.gauss(g, (T, N), 1.0, dtype))[0]
    bounds = _split(g, T, E)
    for zeros in (False, True):
        stacks = [_stack(g, E, N, K, group, dtype, zeros) for _ in range(2 if glu else 1)]
        y = _run(d, x, stacks, _offsets(bounds), base, dtype)
        ref, bound = R.w4(x, stacks, bounds, base, M.ACT_GELU_TANH, dtype)
        D.assert_close(y, ref, bound, f"zeros {zeros}")
        assert torch.equal(y, _run(d, x, stacks, _offsets(bounds), base, dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,N,E,group", TILES)
def test_integers_are_exact_in_every_tile(T, K, N, E, group, dtype):
    # |x| <= 2, |q - z| <= 15, scales 1/4 to 2, K <= 8192: every sum is a multiple of
    # 1/4 below 2^19, and the sums of x (16 + q) stay below 128 x 62, so fp32 holds
    # all of them
    g = _gen(T * 5 + K)
    d = M.make_w4_desc(K, N, E, group, D.DT[dtype])
    x, _ = D.inside(D.ints(g, (T, K), 2, dtype))
    bounds = _split(g, T, E)
    for zeros in (False, True):
        s = _stack(g, E, N, K, group, dtype, zeros, exact=True)
        y = _run(d, x, [s], _offsets(bounds), None, dtype)
        assert torch.equal(y, R.w4(x, [s], bounds, None, None, dtype)[0].to(dtype)), zeros


# Rows for which a plan takes the 64-row tile and the 128-row tile (a pair the other
# way round), experts whose last tiles are partial
TAILS = [(T, 2056, 3) for T in (1100, 2100)]


def tails(group):
    """K of one stage up to three rounds of the wide tiles' ring of three."""
    return range(group, 3 * 384 + 1, group)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("T,N,E", TAILS)
@pytest.mark.parametrize("group", [32, 64, 128])
def test_every_end_of_k(T, N, E, group, glu, dtype):
    for K in tails(group):
        g = _gen(T + K)
        d = M.make_w4_desc(K, N, E, group, D.DT[dtype])
        # NaN behind each row, and behind the last
        x, _ = D.inside(D.gauss(g, (T, K), 1.0, dtype))
        bounds = [0, T // 3 + 8, T - 40, T]
        zeros = K // group % 2 == 0
        stacks = [_stack(g, E, N, K, group, dtype, zeros) for _ in range(2 if glu else 1)]
        y = _run(d, x, stacks, _offsets(bounds), None, dtype)
        ref, bound = R.w4(x, stacks, bounds, None, M.ACT_SILU, dtype)
        D.assert_close(y, ref, bound, f"K {K}, zeros {zeros}")


# Calls with a list for crowded experts' tiles of 16 rows and more beside one for the
# others': with test_every_tile's, all pairs of tiles that a plan can choose
LISTS = [(143, 32, 11816, 5, 32), (161, 32, 2192, 82, 32), (190, 32, 496, 152, 32), (223, 32, 4240, 112, 32),
         (273, 32, 7032, 159, 32), (1148, 32, 72, 639, 32), (2040, 128, 136, 986, 32), (4835, 896, 192, 124, 128),
         (11790, 2432, 144, 100, 128), (16201, 512, 64, 16, 32), (18288, 896, 152, 866, 64), (20875, 832, 160, 431, 64),
         (32015, 2176, 24, 29, 128)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("T,K,N,E,group", LISTS)
def test_lists(T, K, N, E, group, glu, dtype):
    g = _gen(T + K + E)
    d = M.make_w4_desc(K, N, E, group, D.DT[dtype])
    x, _ = D.inside(D.gauss(g, (T, K), 1.0, dtype))
    a, b = E // 3, E - E // 3
    half = _split(g, T // 2, E)
    spreads = [("spread", _split(g, T, E, 1, 2)), ("one", [0] * (a + 1) + [T] * b),
               ("half at one", [v if e <= a else v + T - T // 2 for e, v in enumerate(half)]),
               ("two", [0] * (a + 1) + [T // 2 - 5] * (b - 1) + [T])]
    for i, (what, bounds) in enumerate(spreads):
        assert len(bounds) == E + 1
        stacks = [_stack(g, E, N, K, group, dtype, i % 2 == 0) for _ in range(2 if glu else 1)]
        y = _run(d, x, stacks, _offsets(bounds), None, dtype)
        ref, bound = R.w4(x, stacks, bounds, None, M.ACT_SILU, dtype)
        rows = slice(bounds[0], bounds[-1])
        D.assert_close(y[rows], ref[rows], bound[rows], what)
        assert (y[:bounds[0]] == 77.0).all() and (y[bounds[-1]:] == 77.0).all(), what
