"""Products with 4-bit weights and group scales, dense and by expert, against
their definition in 64 bits: values within bounds derived from the types, and
integer inputs for which the result has to be equal."""
import pytest
import torch

import dense_ref as D
import experts_ref as R
import trellis_quantized_moe_exl3_amd as M

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _split(g, R_, E, lead=0, tail=0):
    """Row boundaries of E experts, some of them empty, between the first `lead`
    and the last `tail` rows."""
    cuts = torch.sort(torch.randint(0, R_ - lead - tail + 1, (E - 1,), generator=g, device="cuda")).values.tolist()
    return [lead + v for v in [0] + cuts + [R_ - lead - tail]]


def _offsets(bounds):
    t = torch.tensor([-5] + bounds + [-5], dtype=torch.int32, device="cuda")
    return t[1:-1]   # (4-byte aligned)


def _run(d, x, stacks, offsets, base, dtype, status=0):
    T = x.shape[0]
    y, big = D.inside(torch.zeros(T, d.n_out, dtype=dtype, device="cuda"), 3, 24)
    big.fill_(77.0)
    ws = D.poisoned(M.w4_workspace_size(d, T))
    w = [M.make_w4(*s) for s in stacks]
    if len(w) == 2:
        M.w4_glu(d, x, w[0], w[1], y, ws, offsets=offsets)
    else:
        M.w4_linear(d, x, w[0], y, ws, offsets=offsets, base=base)
    assert M.status(ws) == status
    assert (big[T:] == 77.0).all() and (big[:, d.n_out:] == 77.0).all()
    return y


def _stack(g, E, N, K, group, dtype, zeros=True, exact=False):
    """A stack with NaN scales right behind it."""
    c, s, z = R.w4_stack(g, E, N, K, group, dtype, zeros, exact)
    return c, D.followed(s), z


# rows, K, N, experts, group
SHAPES = [(1, 32, 8, 1, 32), (1, 2048, 4096, 1, 128), (2, 64, 24, 1, 64), (5, 416, 72, 3, 32), (16, 1024, 136, 1, 128),
          (17, 384, 200, 2, 64), (31, 1376, 1032, 5, 32), (64, 4096, 256, 1, 64), (64, 1024, 520, 40, 128),
          (65, 256, 128, 1, 32), (100, 8192, 64, 7, 128), (130, 896, 264, 1, 128), (257, 640, 328, 300, 64),
          (333, 1376, 1032, 5, 32), (515, 512, 1000, 12, 128), (1100, 288, 2056, 2, 32), (2000, 1088, 136, 3, 64),
          (1500, 512, 512, 1024, 64), (4000, 256, 512, 1, 128)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,N,E,group", SHAPES)
def test_linear(T, K, N, E, group, dtype):
    g = _gen(T + K)
    d = M.make_w4_desc(K, N, E, group, D.DT[dtype])
    x, _ = D.inside(D.gauss(g, (T, K), 1.0, dtype))
    base, _ = D.inside(D.gauss(g, (T, N), 1.0, dtype))
    for zeros, b in ((True, None), (False, base)):
        s = _stack(g, E, N, K, group, dtype, zeros)
        bounds = _split(g, T, E)
        y = _run(d, x, [s], None if E == 1 else _offsets(bounds), b, dtype)
        ref, bound = R.w4(x, [s], bounds, b, None, dtype)
        D.assert_close(y, ref, bound, f"zeros {zeros}", 2 * R.half_step(dtype))
        if b is not None:   # in place
            z, _ = D.inside(base)
            M.w4_linear(d, x, M.make_w4(*s), z, D.poisoned(M.w4_workspace_size(d, T)), offsets=_offsets(bounds), base=z)
            assert torch.equal(z, y)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,N,E,group", SHAPES)
def test_glu(T, K, N, E, group, dtype):
    g = _gen(T + N)
    x, _ = D.inside(D.gauss(g, (T, K), 1.0, dtype))
    for act, zeros in ((M.ACT_SILU, (False, True)), (M.ACT_GELU_TANH, (True, True))):
        d = M.make_w4_desc(K, N, E, group, D.DT[dtype], act)
        stacks = [_stack(g, E, N, K, group, dtype, z) for z in zeros]
        bounds = _split(g, T, E)
        h = _run(d, x, stacks, None if E == 1 else _offsets(bounds), None, dtype)
        ref, bound = R.w4(x, stacks, bounds, None, act, dtype)
        D.assert_close(h, ref, bound, f"act {act}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,N,E,group", SHAPES)
def test_integers_are_exact(T, K, N, E, group, dtype):
    # |x| <= 2, |q - z| <= 15, scales 1/4 to 2: every sum is a multiple of 1/4
    # below 2^22 (K <= 8192: 8192 x 30 x 2), and the sums of x (16 + q) stay below
    # 128 x 62, so fp32 holds all of them
    g = _gen(T * 3 + K)
    d = M.make_w4_desc(K, N, E, group, D.DT[dtype])
    x, _ = D.inside(D.ints(g, (T, K), 2, dtype))
    base, _ = D.inside(D.ints(g, (T, N), 3, dtype))
    s = _stack(g, E, N, K, group, dtype, True, exact=True)
    bounds = _split(g, T, E)
    y = _run(d, x, [s], _offsets(bounds), base, dtype)
    ref, _ = R.w4(x, [s], bounds, base, None, dtype)
    assert torch.equal(y, ref.to(dtype))


# Sizes that between them take tiles of every shape, several tiles of columns a
# block, and two launches over lists of tiles (a second one for crowded experts);
# the kernels that they leave out are test_gpu_w4_tiles.py's
VARIANTS = [(64, 288, 1032, 6, 32), (24, 2048, 12296, 6, 64), (24, 288, 12296, 6, 32), (24, 896, 12296, 1, 128),
            (40, 288, 1032, 50, 32), (150, 800, 4104, 50, 32), (150, 896, 12296, 50, 128), (300, 2016, 4104, 50, 32),
            (300, 288, 20008, 50, 32), (800, 832, 1032, 50, 64), (150, 288, 4104, 1, 32), (300, 288, 20008, 1, 32),
            (150, 2048, 20008, 6, 128), (2000, 288, 1032, 50, 32), (800, 2048, 264, 50, 64), (1300, 416, 776, 7, 32)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("T,K,N,E,group", VARIANTS)
def test_every_tile(T, K, N, E, group, glu, dtype):
    g = _gen(T + K + E)
    d = M.make_w4_desc(K, N, E, group, D.DT[dtype])
    x, _ = D.inside(D.gauss(g, (T, K), 1.0, dtype))
    base = None if glu else D.inside(D.gauss(g, (T, N), 1.0, dtype))[0]
    # rows spread, rows crowded at the last expert or at two in between (some
    # empty, some with a row or two), and all of them at one
    few = min(E - 1, T // 8)
    spreads = {"spread": _split(g, T, E, 1, 2), "last": list(range(E)) + [T] if E <= T else None,
               "two": [0] * (E // 3 + 1) + [T // 2] * (E - E // 3 - 1) + [T], "one": [0] * (E // 2 + 1) + [T] * (E - E // 2),
               "first": [0] + [T - few + i for i in range(few)] + [T] * (E - few)}
    for i, (what, bounds) in enumerate(spreads.items()):
        if bounds is None:
            continue
        assert len(bounds) == E + 1 and all(a <= b for a, b in zip(bounds, bounds[1:]))
        stacks = [_stack(g, E, N, K, group, dtype, (i + j) % 2 == 0) for j in range(2 if glu else 1)]
        y = _run(d, x, stacks, _offsets(bounds), base, dtype)
        ref, bound = R.w4(x, stacks, bounds, base, M.ACT_SILU, dtype)
        rows = slice(bounds[0], bounds[-1])
        D.assert_close(y[rows], ref[rows], bound[rows], what)
        assert (y[:bounds[0]] == 77.0).all() and (y[bounds[-1]:] == 77.0).all(), what
        if E == 1:
            break


# Narrow tiles whose k eight wavefronts share: each of them, k that does not come
# out even, wavefronts without any
EIGHTS = [(1, 1024, 8, 1, 128), (3, 1056, 1000, 1, 32), (2, 1024, 8184, 1, 128), (4, 1088, 6000, 1, 64), (9, 1376, 520, 1, 32),
          (16, 2112, 4096, 1, 64), (15, 1056, 8184, 1, 32), (12, 4096, 8000, 1, 128), (17, 4160, 4088, 1, 64),
          (100, 4128, 2040, 1, 32), (9, 1152, 264, 4, 64), (40, 1440, 136, 6, 32), (3, 65536, 8, 1, 128)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("T,K,N,E,group", EIGHTS)
def test_tiles_of_eight_wavefronts(T, K, N, E, group, glu, dtype):
    g = _gen(T + K + E)
    d = M.make_w4_desc(K, N, E, group, D.DT[dtype])
    x, _ = D.inside(D.gauss(g, (T, K), 1.0, dtype))
    base = None if glu else D.inside(D.gauss(g, (T, N), 1.0, dtype))[0]
    bounds = _split(g, T, E)
    for zeros in (False, True):
        stacks = [_stack(g, E, N, K, group, dtype, zeros) for j in range(2 if glu else 1)]
        y = _run(d, x, stacks, _offsets(bounds), base, dtype)
        ref, bound = R.w4(x, stacks, bounds, base, M.ACT_SILU, dtype)
        D.assert_close(y, ref, bound, f"zeros {zeros}")
        assert torch.equal(y, _run(d, x, stacks, _offsets(bounds), base, dtype))


@pytest.mark.parametrize("T,E", [(100, 1024), (128, 1024), (3000, 1024), (200, 1), (5000, 2)])
def test_lists_of_many_and_few_experts(T, E):
    # one row here and there, the last expert crowded
    g = _gen(E)
    dtype = torch.bfloat16
    K, N = 256, 264
    d = M.make_w4_desc(K, N, E, 128, M.DT_BF16)
    x = D.gauss(g, (T, K), 1.0, dtype)
    s = _stack(g, E, N, K, 128, dtype)
    for crowd in (0, T // 2, T - 1):
        cuts = torch.sort(torch.randint(0, T - crowd + 1, (E - 1,), generator=g, device="cuda")).values.tolist()
        bounds = [0] + cuts + [T]
        y = _run(d, x, [s], _offsets(bounds), None, dtype)
        ref, bound = R.w4(x, [s], bounds, None, None, dtype)
        D.assert_close(y, ref, bound, f"crowd {crowd}")


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("T,E", [(9, 3), (64, 5), (200, 4), (700, 9), (3000, 2)])
def test_rows_outside_the_offsets_stay(T, E, glu):
    g = _gen(T)
    dtype = torch.bfloat16
    K, N, group = 256, 136, 64
    d = M.make_w4_desc(K, N, E, group, M.DT_BF16)
    x = D.gauss(g, (T, K), 1.0, dtype)
    stacks = [_stack(g, E, N, K, group, dtype) for _ in range(2 if glu else 1)]
    lead, tail = 2, T // 3
    bounds = _split(g, T, E, lead, tail)
    x[:lead], x[T - tail:] = float("nan"), float("inf")
    y = _run(d, x, stacks, _offsets(bounds), None, dtype)
    assert (y[:lead] == 77.0).all() and (y[T - tail:] == 77.0).all()
    ref, bound = R.w4(x[:T - tail], stacks, bounds, None, M.ACT_SILU, dtype)
    D.assert_close(y[lead:T - tail], ref[lead:], bound[lead:], "rows")
    # no expert has a row
    y = _run(d, x, stacks, _offsets([T // 2] * (E + 1)), None, dtype)
    assert (y == 77.0).all()


@pytest.mark.parametrize("T", [1, 7, 40, 300, 2000])
@pytest.mark.parametrize("dtype", TYPES)
def test_a_rows_infinities_stay_with_it(T, dtype):
    g = _gen(T)
    K, N, E, group = 512, 200, 3, 32
    d = M.make_w4_desc(K, N, E, group, D.DT[dtype])
    x = D.gauss(g, (T, K), 1.0, dtype)
    s = _stack(g, E, N, K, group, dtype)
    bounds = _split(g, T, E)
    clean = _run(d, x, [s], _offsets(bounds), None, dtype)
    x[T // 2, 5], x[T - 1, K - 1] = float("inf"), float("nan")
    y = _run(d, x, [s], _offsets(bounds), None, dtype)
    touched = torch.zeros(T, dtype=torch.bool)
    touched[T // 2] = touched[T - 1] = True
    assert torch.equal(y[~touched], clean[~touched])
    assert not torch.isfinite(y[touched]).any()
    # another expert's scales
    e = next((e for e in range(E) if bounds[e + 1] > bounds[e]), 0)
    x = D.gauss(g, (T, K), 1.0, dtype)
    clean = _run(d, x, [s], _offsets(bounds), None, dtype)
    s[1][e] = float("nan")
    y = _run(d, x, [s], _offsets(bounds), None, dtype)
    rows = torch.zeros(T, dtype=torch.bool)
    rows[bounds[e]:bounds[e + 1]] = True
    assert torch.isnan(y[rows]).all() and torch.equal(y[~rows], clean[~rows])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 40, 300])
def test_large_activations_and_any_zero(T, dtype):
    # x up to the type's range (2^100 in bf16), zeros of 0 to 255
    g = _gen(T)
    K, N, group = 256, 72, 64
    d = M.make_w4_desc(K, N, 1, group, D.DT[dtype])
    c, s, z = _stack(g, 1, N, K, group, dtype)
    z = torch.randint(0, 256, z.shape, generator=g, device="cuda", dtype=torch.uint8)
    big = 2.0 ** 100 if dtype == torch.bfloat16 else 65504.0
    x = (D.gauss(g, (T, K), 0.2, torch.float32).clamp(-1, 1) * big).to(dtype)
    s = s * (2.0 ** -12)
    y = _run(d, x, [(c, s, z)], None, None, dtype)
    ref, bound = R.w4(x, [(c, s, z)], [0, T], None, None, dtype)
    D.assert_close(y, ref, bound, "y")


@pytest.mark.parametrize("bad", [[0, 9, 5, 40], [-1, 3, 9, 40], [0, 3, 9, 41], [40, 0, 0, 0], [0, 2 ** 31 - 1, 3, 40],
                                 [-2 ** 31, 5, 9, 40]])
def test_bad_offsets_are_reported(bad):
    g = _gen(3)
    dtype = torch.bfloat16
    K, N, E, group = 256, 72, 3, 64
    d = M.make_w4_desc(K, N, E, group, M.DT_BF16)
    x = D.gauss(g, (40, K), 1.0, dtype)
    for n in (1, 2):
        stacks = [_stack(g, E, N, K, group, dtype) for _ in range(n)]
        _run(d, x, stacks, _offsets(bad), None, dtype, M.STATUS_BAD_INDEX)
        _run(d, x, stacks, _offsets([0, 3, 9, 40]), None, dtype)


@pytest.mark.parametrize("case", ["descend", "below", "beyond", "swapped", "extremes"])
def test_bad_offsets_of_listed_tiles_are_reported(case):
    # (overlapping experts have more tiles than the rows have: the lists and the
    # launches end where the call's size says)
    g = _gen(4)
    dtype = torch.bfloat16
    T, K, N, E = 700, 256, 136, 40
    d = M.make_w4_desc(K, N, E, 64, M.DT_BF16)
    x, s = D.gauss(g, (T, K), 1.0, dtype), _stack(g, E, N, K, 64, dtype)
    bounds = _split(g, T, E)
    if case == "descend":
        bounds[5:] = [T if i % 2 else 0 for i in range(E + 1 - 5)]
    elif case == "below":
        bounds[0] = -7
    elif case == "beyond":
        bounds[-1] = T + 1
    elif case == "swapped":
        bounds = bounds[::-1]
    else:
        bounds = [2 ** 31 - 1 if i % 2 else -2 ** 31 for i in range(E + 1)]
    _run(d, x, [s], _offsets(bounds), None, dtype, M.STATUS_BAD_INDEX)
    _run(d, x, [s, s], _offsets(bounds), None, dtype, M.STATUS_BAD_INDEX)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T", [1, 40, 700])
def test_one_expert_out_of_a_stack(T, dtype):
    # its zeros begin at an odd multiple of 8 bytes
    g = _gen(T)
    K, N, E, group = 1376, 1032, 4, 32
    d = M.make_w4_desc(K, N, 1, group, D.DT[dtype])
    x = D.gauss(g, (T, K), 1.0, dtype)
    stacks = [_stack(g, E, N, K, group, dtype) for _ in range(2)]
    for e in (1, 3):
        one = [tuple(t[e] for t in s) for s in stacks]
        assert one[0][2].data_ptr() % 16 == 8
        for n in (1, 2):
            y = _run(d, x, one[:n], None, None, dtype)
            ref, bound = R.w4(x, [tuple(t[e:e + 1] for t in s) for s in stacks[:n]], [0, T], None, M.ACT_SILU, dtype)
            D.assert_close(y, ref, bound, f"expert {e}, {n}")


@pytest.mark.parametrize("T", [6, 600])
def test_stacks_past_four_gib(T):
    g = _gen(T)
    dtype = torch.float16
    E, N, K, group = 600, 2048, 8192, 128
    d = M.make_w4_desc(K, N, E, group, M.DT_F16)
    c = torch.zeros(E, N, K // 2, dtype=torch.uint8, device="cuda")
    s = torch.ones(E, N, K // group, dtype=dtype, device="cuda")
    z = torch.full((E, N, K // group), 3, dtype=torch.uint8, device="cuda")
    named = [0, 255, 256, 511, 512, E - 1]   # (4 GiB of codes: 512)
    bounds = [0] * (E + 1)
    for i, e in enumerate(named):
        c[e], s[e], z[e] = (t[0] for t in R.w4_stack(g, 1, N, K, group, dtype))
        bounds[e + 1:] = [(i + 1) * (T // 6)] * (E - e)
    x = D.gauss(g, (T, K), 1.0, dtype)
    y = _run(d, x, [(c, s, z)], _offsets(bounds), None, dtype)
    ref, bound = R.w4(x, [(c, s, z)], bounds, None, None, dtype)
    D.assert_close(y, ref, bound, "y")


def test_no_rows():
    d = M.make_w4_desc(64, 16, 1, 64)
    s = M.make_w4(*R.w4_stack(_gen(0), 1, 16, 64, 64, torch.bfloat16))
    x, y = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 16, dtype=torch.bfloat16, device="cuda")
    M.w4_linear(d, x, s, y, D.poisoned(256))
    M.w4_glu(d, x, s, s, y, D.poisoned(256))
