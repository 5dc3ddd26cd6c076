"""Tokens sorted by expert and back, with weights, gradients and dropout,
against their definitions in 64 bits: tables equal, rows within bounds derived
from the types, integer inputs equal."""
import pytest
import torch

import dense_ref as D
import experts_ref as R
import trellis_quantized_moe_exl3_amd as M

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _rng(g):
    return torch.randint(0, 1 << 62, (2,), generator=g, device="cuda")


def _tables(E, n, fill=-77):
    """counts, offsets, sorted_ids, pos inside longer arrays, at odd addresses."""
    whole = [torch.full((m + 8,), fill, dtype=torch.int32, device="cuda") for m in (E, E + 1, n, n)]
    return [t[3:3 + m] for t, m in zip(whole, (E, E + 1, n, n))], whole


def _sort(idx, E, full=True):
    T, k = idx.shape
    d = M.make_tokens_desc(8, E, k)
    (counts, offsets, ids, pos), whole = _tables(E, T * k)
    ws = D.poisoned(M.sort_workspace_size(d, T))
    M.sort(d, idx, counts if full else None, offsets, ids if full else None, pos, ws)
    return counts, offsets, ids, pos, whole, M.status(ws)


def _check_sort(idx, E):
    counts, offsets, ids, pos, whole, _ = _sort(idx, E)
    want = R.sort(idx, E)
    for got, ref, what in zip((counts, offsets, ids, pos), want, ("counts", "offsets", "sorted_ids", "pos")):
        n = ref.numel()
        assert torch.equal(got[:n].cpu().long(), ref.long()), what
        assert (got[n:] == -77).all(), what    # behind the last slot
    for w, m in zip(whole, (E, E + 1, idx.numel(), idx.numel())):
        assert (w[:3] == -77).all() and (w[3 + m:] == -77).all()


# T, k, E: one slot, one expert, the most of them, 4096 slots (what one block
# sorts alone) and one more or less, calls of up to 64 chunks of 2048 slots and of more
SORTS = [(1, 1, 1), (1, 16, 1024), (3, 2, 5), (8, 8, 288), (64, 8, 288), (512, 8, 288), (513, 8, 64), (4095, 1, 7),
         (4096, 1, 1023), (4097, 1, 1024), (1000, 13, 100), (7168, 8, 288), (16384, 8, 1), (16385, 16, 40),
         (32768, 8, 1024), (40000, 15, 1000)]


@pytest.mark.parametrize("T,k,E", SORTS)
def test_sort(T, k, E):
    g = _gen(T + k)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda").to(torch.int32)
    _check_sort(idx, E)
    # crowded experts, and slots without one
    skew = (torch.rand(T, k, generator=g, device="cuda") ** 4 * E).to(torch.int32)
    _check_sort(torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.2, -1, skew), E)


# Whole chunks and one slot more; 64 chunks (each block adds up the counts of all
# others) and the first slot of a 65th (a launch of its own does)
@pytest.mark.parametrize("T,k,E", [(768, 8, 288), (1229, 5, 288), (1229, 5, 1024), (16384, 8, 288), (16384, 8, 1024),
                                   (43691, 3, 288), (43691, 3, 1024)])
def test_sort_at_the_ends_of_chunks(T, k, E):
    assert T * k % 2048 in (0, 1)
    g = _gen(T + E)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda").to(torch.int32)
    _check_sort(idx, E)
    skew = (torch.rand(T, k, generator=g, device="cuda") ** 4 * E).to(torch.int32)
    skew = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.2, -1, skew)
    skew[-1, -1] = E - 1   # the last slot has an expert
    _check_sort(skew, E)
    # an index out of range in the first chunk and in the last
    for t in (0, T - 1):
        wrong = skew.clone()
        wrong[t, k - 1] = E
        assert _sort(wrong, E)[-1] == M.STATUS_BAD_INDEX
        _check_sort(wrong, E)


@pytest.mark.parametrize("value", ["none", "first", "last"])
@pytest.mark.parametrize("T,k,E", [(5, 3, 9), (3000, 4, 300), (40000, 8, 33)])
def test_sort_of_one_kind(T, k, E, value):
    idx = torch.full((T, k), {"none": -1, "first": 0, "last": E - 1}[value], dtype=torch.int32, device="cuda")
    _check_sort(idx, E)


@pytest.mark.parametrize("T,k,E", [(5, 3, 9), (3000, 4, 1024), (40000, 8, 33)])
@pytest.mark.parametrize("bad", [-2, "E", 2 ** 31 - 1, -2 ** 31])
def test_sort_reports_bad_indexes(T, k, E, bad):
    g = _gen(T)
    idx = torch.randint(-1, E, (T, k), generator=g, device="cuda").to(torch.int32)
    assert _sort(idx, E)[-1] == 0
    idx[T - 1, k - 1] = E if bad == "E" else bad
    idx[T // 2, 0] = E if bad == "E" else bad
    assert _sort(idx, E)[-1] == M.STATUS_BAD_INDEX
    _check_sort(idx, E)


def test_sort_without_optional_tables_and_tokens():
    g = _gen(1)
    idx = torch.randint(-1, 20, (300, 5), generator=g, device="cuda").to(torch.int32)
    counts, offsets, ids, pos, _, _ = _sort(idx, 20, full=False)
    _, o, _, p = R.sort(idx, 20)
    assert torch.equal(offsets.cpu().long(), o) and torch.equal(pos.cpu().long(), p)
    assert (counts == -77).all() and (ids == -77).all()
    _check_sort(torch.empty(0, 5, dtype=torch.int32, device="cuda"), 20)


# ---- rows: T, H, E, k
SHAPES = [(1, 8, 1, 1), (1, 4096, 288, 8), (3, 520, 4, 2), (8, 4096, 288, 8), (65, 1032, 30, 3), (100, 72, 16, 16),
          (129, 2056, 12, 9), (300, 16384, 8, 4), (509, 776, 40, 5), (2000, 136, 3, 1)]


class Case:
    """A call's tokens, sorted rows and tables: some slots without expert, the
    last sorted rows cut off where `cut`."""

    def __init__(self, T, H, E, k, dtype, cut=False, ints=False):
        g = self.g = _gen(T * 7 + H + k)
        self.T, self.H, self.k, self.dtype = T, H, k, dtype
        self.d = M.make_tokens_desc(H, E, k, D.DT[dtype])
        idx = torch.argsort(torch.rand(T, E, generator=g, device="cuda"), dim=1)[:, :k].to(torch.int32)
        idx = torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.1, -1, idx)
        self.pos = _sort(idx, E)[3]
        # (one row more than the slots have: named by none)
        self.rows = max(1, (T * k) // 2) if cut else T * k + 1
        if ints:
            row = lambda n: D.inside(D.ints(g, (n, H), 3, dtype))[0]
            self.w = 2.0 ** torch.randint(-2, 2, (T, k), generator=g, device="cuda").float()
        else:
            row = lambda n: D.inside(D.gauss(g, (n, H), 1.0, dtype))[0]
            self.w = torch.randn(T, k, generator=g, device="cuda")
        self.x, self.base, self.dy = row(T), row(T), row(T)
        self.z = row(self.rows)
        self.rng = _rng(g)

    def new(self, rows):
        """Rows to write, inside a larger array of 77s."""
        v, big = D.inside(torch.zeros(rows, self.H, dtype=self.dtype, device="cuda"), 3, 24)
        big.fill_(77.0)
        return v, big

    def around(self, big, rows):
        assert (big[rows:] == 77.0).all() and (big[:, self.H:] == 77.0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,E,k", SHAPES)
def test_dispatch(T, H, E, k, dtype):
    for cut in (False, True):
        c = Case(T, H, E, k, dtype, cut)
        for w in (None, c.w):
            out, big = c.new(c.rows)
            M.dispatch(c.d, c.x, c.pos, out, w=w)
            ref, bound, named = R.spread(c.x.double(), c.pos, w, c.rows, dtype)
            D.assert_close(out[named], ref[named], bound[named], "rows")
            assert (out[~named] == 77.0).all()
            c.around(big, c.rows)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,E,k", SHAPES)
def test_combine(T, H, E, k, dtype):
    for cut in (False, True):
        c = Case(T, H, E, k, dtype, cut)
        for w, base, p in ((None, None, 0.0), (c.w, c.base, 0.0), (c.w, None, 0.3), (None, c.base, 0.7), (c.w, c.base, 1.0)):
            y, big = c.new(T)
            M.combine(c.d, c.z, c.pos, y, w=w, base=base, p=p, rng=c.rng if p else None)
            ref, bound = R.gather(c.z, c.pos, w, T, base, p, c.rng, dtype)
            D.assert_close(y, ref, bound, f"p = {p}")
            c.around(big, T)
            if base is not None:   # in place
                y.copy_(base)
                M.combine(c.d, c.z, c.pos, y, w=w, base=y, p=p, rng=c.rng)
                D.assert_close(y, ref, bound, f"in place, p = {p}")


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,E,k", SHAPES)
def test_dispatch_backward(T, H, E, k, dtype):
    for cut in (False, True):
        c = Case(T, H, E, k, dtype, cut)
        for w, want in ((None, False), (c.w, False), (None, True), (c.w, True)):
            dx, big = c.new(T)
            dw = torch.full((T, k), 77.0, device="cuda")
            M.dispatch_backward(c.d, c.z, c.x if want else None, c.pos, dx, w=w, dw=dw if want else None)
            ref, bound = R.gather(c.z, c.pos, w, T, None, 0, None, dtype)
            D.assert_close(dx, ref, bound, "dx")
            c.around(big, T)
            if want:
                ref, bound = R.products(c.z, c.pos, c.x.double())
                D.assert_close(dw, ref, bound, "dw")
            else:
                assert (dw == 77.0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,E,k", SHAPES)
def test_combine_backward(T, H, E, k, dtype):
    for cut in (False, True):
        c = Case(T, H, E, k, dtype, cut)
        for w, want, p in ((None, False, 0.0), (c.w, True, 0.0), (c.w, True, 0.3), (None, True, 0.7), (c.w, False, 0.5)):
            dz, big = c.new(c.rows)
            dw = torch.full((T, k), 77.0, device="cuda")
            M.combine_backward(c.d, c.dy, c.z if want else None, c.pos, dz, w=w, dw=dw if want else None, p=p, rng=c.rng)
            dy = R.drop(c.dy.double(), p, c.rng)
            ref, bound, named = R.spread(dy, c.pos, w, c.rows, dtype)
            D.assert_close(dz[named], ref[named], bound[named], f"dz, p = {p}")
            assert (dz[~named] == 77.0).all()
            c.around(big, c.rows)
            if want:
                ref, bound = R.products(c.z, c.pos, dy)
                D.assert_close(dw, ref, bound, f"dw, p = {p}")
                again, keep = c.z.clone(), dw.clone()   # dz over z
                M.combine_backward(c.d, c.dy, again, c.pos, again, w=w, dw=dw, p=p, rng=c.rng)
                assert torch.equal(again[named], dz[named]) and torch.equal(again[~named], c.z[~named])
                assert torch.equal(dw, keep)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,E,k", [(5, 264, 7, 3), (200, 1032, 20, 8), (33, 4096, 16, 16)])
def test_gradients_against_differences(T, H, E, k, dtype):
    # dispatch and combine are linear in the rows and in the weights, so a
    # difference of two outputs is the derivative itself; small integers and
    # powers of two make every step exact: y below 2^8 in steps of 1/4 would not
    # be, so the rows are sparse (a token's sums stay below 16)
    c = Case(T, H, E, k, dtype, ints=True)
    g = c.g
    sparse = lambda rows: D.ints(g, (rows, H), 1, dtype, 0.25)
    w, w2 = c.w.clamp(max=0.5), c.w.clamp(max=0.5) * 2
    z, dz, x, dx = sparse(c.rows), sparse(c.rows), sparse(T), sparse(T)
    dy, dxs = sparse(T), sparse(c.rows)

    def combine(z, w):
        y = torch.empty(T, H, dtype=dtype, device="cuda")
        M.combine(c.d, z, c.pos, y, w=w)
        return y.double()

    def dispatch(x, w):
        out = torch.zeros(c.rows, H, dtype=dtype, device="cuda")
        M.dispatch(c.d, x, c.pos, out, w=w)
        return out.double()

    gz, gw = torch.zeros(c.rows, H, dtype=dtype, device="cuda"), torch.empty(T, k, device="cuda")
    M.combine_backward(c.d, dy, z, c.pos, gz, w=w, dw=gw)
    assert ((combine(z + dz, w) - combine(z, w)) * dy.double()).sum() == (gz.double() * dz.double()).sum()
    assert ((combine(z, w2) - combine(z, w)) * dy.double()).sum() == (gw.double() * (w2 - w).double()).sum()
    gx = torch.empty(T, H, dtype=dtype, device="cuda")
    M.dispatch_backward(c.d, dxs, x, c.pos, gx, w=w, dw=gw)
    assert ((dispatch(x + dx, w) - dispatch(x, w)) * dxs.double()).sum() == (gx.double() * dx.double()).sum()
    assert ((dispatch(x, w2) - dispatch(x, w)) * dxs.double()).sum() == (gw.double() * (w2 - w).double()).sum()


@pytest.mark.parametrize("dtype", TYPES)
def test_slots_without_a_row_take_no_part(dtype):
    c = Case(40, 264, 6, 3, dtype)
    c.pos[::4] = -1
    c.pos[1] = 2 ** 31 - 1
    c.pos[2] = c.rows
    c.pos[3] = -2 ** 31
    gone = (c.pos < 0) | (c.pos >= c.rows)
    named = torch.zeros(c.rows, dtype=torch.bool, device="cuda")
    named[c.pos[~gone].long()] = True
    w, z = c.w.clone(), c.z.clone()
    w.view(-1)[gone] = float("nan")
    z[~named] = float("nan")
    y, dx, dw = c.new(40)[0], c.new(40)[0], torch.full((40, 3), 7.0, device="cuda")
    M.combine(c.d, z, c.pos, y, w=w)
    ref, bound = R.gather(c.z, c.pos, torch.where(gone.view(40, 3), 0, w), 40, None, 0, None, dtype)
    D.assert_close(y, ref, bound, "y")
    M.dispatch_backward(c.d, z, c.x, c.pos, dx, w=w, dw=dw)
    D.assert_close(dx, ref, bound, "dx")
    assert (dw.view(-1)[gone] == 0).all() and torch.isfinite(dw).all()
    y[0] = 7.0
    c.pos[:3] = -1   # a token without any row
    M.combine(c.d, z, c.pos, y, w=w, base=c.base)
    assert torch.equal(y[0], c.base[0])
    M.combine(c.d, z, c.pos, y, w=w)
    assert (y[0] == 0).all()


def test_rows_past_four_gib():
    # sorted rows of 5 GiB: offsets beyond 32 bits
    T, H, k = 8, 65536, 1
    rows = 5 * 2 ** 30 // (2 * H)
    d = M.make_tokens_desc(H, 4, k, M.DT_BF16)
    g = _gen(0)
    x = D.gauss(g, (T, H), 1.0, torch.bfloat16)
    out = torch.zeros(rows, H, dtype=torch.bfloat16, device="cuda")
    pos = torch.tensor([rows - 1, 0, rows // 2, 3, rows - 2, 7, 32768, 32767], dtype=torch.int32, device="cuda")
    M.dispatch(d, x, pos, out)
    assert torch.equal(out[pos.long()], x)
    y = torch.empty_like(x)
    M.combine(d, out, pos, y)
    assert torch.equal(y, x)
    out[pos.long()] = 0
    assert not out.any()


def test_more_tokens_than_one_grid_holds():
    # 2^26 tokens and some at 64 threads each are past 2^32 threads
    T, H = 2 ** 26 + 5, 8
    d = M.make_tokens_desc(H, 2, 1, M.DT_BF16)
    x = (torch.arange(T, dtype=torch.int32, device="cuda") % 251).to(torch.bfloat16)[:, None].expand(T, H).contiguous()
    pos = torch.arange(T - 1, -1, -1, dtype=torch.int32, device="cuda")[:, None]
    out, y, dw = torch.zeros_like(x), torch.zeros_like(x), torch.full((T, 1), 7.0, device="cuda")
    M.dispatch(d, x, pos, out)
    assert torch.equal(out, x.flip(0))
    M.combine(d, out, pos, y)
    assert torch.equal(y, x)
    y.zero_()
    M.dispatch_backward(d, out, x, pos, y, dw=dw)
    assert torch.equal(y, x) and torch.equal(dw[:, 0], 8 * x[:, 0].float().square())
    rng = torch.tensor([3, 5], device="cuda")
    M.combine(d, out, pos, y, p=0.5, rng=rng)   # the last rows' counters
    tail = torch.empty_like(x[-9:])
    M.dropout(x[-9:].contiguous(), tail, 0.5, torch.tensor([3, 5 + T - 9], device="cuda"))
    assert torch.equal(y[-9:], tail)


@pytest.mark.parametrize("T", [0, 4])
def test_no_tokens_or_no_rows(T):
    d = M.make_tokens_desc(16, 4, 2)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, z = torch.ones(T, 16, **bf), torch.empty(0, 16, **bf)
    pos, w = torch.zeros(T, 2, dtype=torch.int32, device="cuda"), torch.ones(T, 2, device="cuda")
    y, dw = torch.full((T, 16), 5.0, **bf), torch.full((T, 2), 5.0, device="cuda")
    M.dispatch(d, x, pos, z, w=w)
    M.combine(d, z, pos, y, w=w, base=x)
    assert torch.equal(y, x)
    M.dispatch_backward(d, z, x, pos, y, w=w, dw=dw)
    assert (y == 0).all() and (dw == 0).all()
    dw.fill_(5.0)
    M.combine_backward(d, x, z, pos, z, w=w, dw=dw)
    assert (dw == 0).all()


# ---- dropout


@pytest.mark.parametrize("dtype", TYPES + [torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 8), (3, 7), (5, 9), (17, 4096), (509, 1381), (1000, 64), (2, 40001), (333, 2),
                                       (64, 1024)])
def test_dropout(rows, cols, dtype):
    g = _gen(rows + cols)
    x, r = D.gauss(g, (rows, cols), 1.0, dtype), D.gauss(g, (rows, cols), 1.0, dtype)
    rng = _rng(g)
    for extra in (0, 5, 16):   # strides: contiguous, odd, whole
        xs, _ = D.inside(x, 2, extra)
        rs, _ = D.inside(r, 2, extra)
        for p in (0.0, 0.1, 0.5, 0.93, 1.0):
            for res in (None, rs):
                y, big = D.inside(torch.zeros_like(x), 3, extra)
                big.fill_(77.0)
                M.dropout(xs, y, p, rng, residual=res)
                ref = R.drop(x.double(), p, rng) + (0 if res is None else r.double())
                err = 2 * R.STEP * ref.abs() + R.STEP * r.double().abs()
                bound = err + R.half_step(dtype) * (ref.abs() + err) + R.least(dtype)
                D.assert_close(y, ref, bound, f"p = {p}, stride {xs.stride(0)}")
                assert (big[rows:] == 77.0).all() and (big[:, cols:] == 77.0).all()
                keep = y.clone()
                for over in (xs, res):   # in place
                    if over is not None:
                        mine = D.inside(over, 1, extra)[0]
                        M.dropout(mine if over is xs else xs, mine, p, rng, residual=mine if over is res else res)
                        assert torch.equal(mine, keep)


@pytest.mark.parametrize("dtype", TYPES + [torch.float32])
@pytest.mark.parametrize("cols", [1, 1381])
def test_dropout_of_the_last_rows(cols, dtype):
    # a part of each matrix, from a row that is at 16 bytes although those beside
    # it are not: the same numbers as in a call on all rows, from the counters of
    # the row it begins with; rows before and behind it stay
    first, rows = 16 // dtype.itemsize, 41
    g = _gen(cols)
    x, r = D.gauss(g, (rows, cols), 1.0, dtype), D.gauss(g, (rows, cols), 1.0, dtype)
    rng = _rng(g)
    whole = torch.empty_like(x)
    M.dropout(x, whole, 0.4, rng, residual=r)
    y = torch.full_like(x, 77.0)
    later = rng + torch.tensor([0, first * -(-cols // 8)], device="cuda")
    M.dropout(x[first:-3], y[first:-3], 0.4, later, residual=r[first:-3])
    assert torch.equal(y[first:-3], whole[first:-3])
    assert (y[:first] == 77.0).all() and (y[-3:] == 77.0).all()
    with pytest.raises(M.MoeError) as e:
        M.dropout(x[1:], y[1:], 0.4, rng)
    assert e.value.code == M.ERR_MISALIGNED


def test_dropout_of_a_transposed_row():
    row, rng = D.gauss(_gen(5), (1, 300), 1.0, torch.float32), torch.tensor([8, 9], device="cuda")
    y = torch.zeros(300, 1, device="cuda")
    M.dropout(row.t(), y, 0.5, rng)
    assert torch.equal(y.double(), R.drop(row.t().double(), 0.5, rng))


@pytest.mark.parametrize("seed,offset", [(0, 0), (-1, -1), (-1, -3), (1 << 40, (1 << 32) - 2), (7, -(1 << 63))])
def test_dropout_counters_wrap(seed, offset):
    rng = torch.tensor([seed, offset], dtype=torch.int64, device="cuda")
    x = torch.ones(6, 24, device="cuda")
    y = torch.empty_like(x)
    M.dropout(x, y, 0.5, rng)
    assert torch.equal(y.double(), R.drop(x.double(), 0.5, rng))
    assert rng.tolist() == [seed, offset]   # read, never written


@pytest.mark.parametrize("p,n", [(2.0 ** -17, 1), (2.0 ** -17 - 1e-9, 0), (1 - 2.0 ** -17, 65536), (1 - 1.5 * 2.0 ** -16, 65535)])
def test_dropout_rounds_p(p, n):
    rng = torch.tensor([3, 4], dtype=torch.int64, device="cuda")
    x = torch.ones(2048, 512, device="cuda")
    y = torch.empty_like(x)
    M.dropout(x, y, p, rng)
    kept, f = R.keep(2048, 512, n / 65536, 3, 4)
    assert torch.equal(y != 0, kept.cuda() if f else torch.zeros_like(x, dtype=torch.bool))
    assert (y[y != 0] == torch.tensor(f)).all()   # 65536 / 1 and 65536 / 65535 rounded


def test_dropped_elements_are_zero_whatever_they_were():
    rng = torch.tensor([5, 6], dtype=torch.int64, device="cuda")
    kept = R.keep(64, 40, 0.5, 5, 6)[0].cuda()
    for dtype in TYPES + [torch.float32]:
        x = torch.ones(64, 40, dtype=dtype, device="cuda")
        x[~kept] = float("nan")
        x[0][~kept[0]] = float("inf")
        y = torch.empty_like(x)
        M.dropout(x, y, 0.5, rng)
        assert torch.equal(y, torch.where(kept, 2.0, 0.0).to(dtype))
        M.dropout(x, y, 1.0, rng)
        assert (y == 0).all()
    # and in combine: a row of infinities
    d = M.make_tokens_desc(40, 2, 1, M.DT_BF16)
    z = torch.full((64, 40), float("inf"), dtype=torch.bfloat16, device="cuda")
    y = torch.empty_like(z)
    M.combine(d, z, torch.arange(64, dtype=torch.int32, device="cuda"), y, p=0.5, rng=rng)
    assert torch.equal(y, torch.where(kept, float("inf"), 0.0).bfloat16())


def test_dropout_keeps_its_share():
    # 2^22 elements: the kept share within 5 standard deviations of 1 - p
    rng = torch.tensor([11, 0], dtype=torch.int64, device="cuda")
    x = torch.ones(1024, 4096, device="cuda")
    y = torch.empty_like(x)
    for p in (0.1, 0.25, 0.5):
        M.dropout(x, y, p, rng)
        share = (y != 0).double().mean().item()
        assert abs(share - (1 - p)) < 5 * (p * (1 - p) / x.numel()) ** 0.5 + 2.0 ** -17


@pytest.mark.parametrize("rows,cols,p", [(0, 8, 0.5), (8, 0, 0.5)])
def test_dropout_of_nothing(rows, cols, p):
    x = torch.empty(rows, cols, device="cuda")
    M.dropout(x, torch.empty_like(x), p, torch.zeros(2, dtype=torch.int64, device="cuda"))
