"""The projection with the adapters of many requests against its definition in
64 bits: values within bounds derived from the types, and integer inputs for
which the result has to be equal."""
import pytest
import torch

import dense_ref as R
import trellis_quantized_moe_exl3_amd as M

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]
# T, K, N, adapters, rank
SHAPES = [(1, 256, 128, 1, 8), (1, 2048, 4096, 8, 16), (2, 8, 8, 3, 8), (7, 520, 136, 4, 24), (16, 1032, 200, 16, 32),
          (17, 264, 72, 5, 40), (33, 1032, 1384, 40, 16), (64, 2048, 512, 64, 64), (65, 136, 128, 3, 128),
          (100, 512, 1000, 7, 256), (128, 776, 264, 33, 16), (129, 512, 256, 2, 8), (257, 1000, 328, 300, 16),
          (300, 40, 520, 9, 72), (515, 1384, 1032, 12, 32), (1100, 264, 2056, 6, 136),
          # 64-row tiles of two wavefronts, k cut over blocks, 256-row tiles and
          # 16 tokens a shrink block, one token of rank 32 and of more than that
          (333, 1384, 4096, 5, 24), (70, 16384, 128, 30, 64), (3900, 264, 4096, 6, 24), (1, 4096, 2048, 4, 32),
          (1, 1032, 136, 4, 40),
          # 128-row tiles, two on a CU; adapters dealt to the k splits; many of them
          # in a tile without much of a projection
          (1300, 264, 4096, 6, 104), (89, 5008, 1008, 12, 96), (116, 40, 1984, 62, 32),
          # 8 tokens a shrink block
          (300, 4104, 264, 3, 128)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _ids(g, T, n, pattern):
    if pattern == "runs":      # the tokens of a request stand together
        per = max(1, T // 5)
        i = torch.randint(-1, n, (T // per + 1,), generator=g, device="cuda").repeat_interleave(per)[:T]
    elif pattern == "one":     # all tokens share the last adapter
        i = torch.full((T,), n - 1, device="cuda")
    elif pattern == "none":
        i = torch.full((T,), -1, device="cuda")
    else:
        i = torch.randint(-1, n, (T,), generator=g, device="cuda")
    return i.to(torch.int32)


def _run(d, x, w, a, b, ids, base, scales, ranks, dtype):
    T, N = x.shape[0], d.n_out
    y, big = R.inside(torch.zeros(T, N, dtype=dtype, device="cuda"), 3, 24)
    big.fill_(77.0)
    ws = R.poisoned(M.lora_workspace_size(d, T))
    M.lora_linear(d, x, w, a, b, ids, y, ws, base=base, scales=scales, ranks=ranks)
    assert M.status(ws) == 0
    assert (big[T:] == 77.0).all() and (big[:, N:] == 77.0).all()
    return y


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,N,n,r", SHAPES)
def test_values(T, K, N, n, r, dtype):
    g = _gen(T + K)
    d = M.make_lora_desc(K, N, n, r, R.DT[dtype])
    x, _ = R.inside(R.gauss(g, (T, K), 1.0, dtype))
    w = R.followed(R.gauss(g, (N, K), K ** -0.5, dtype))
    a, b = R.followed(R.gauss(g, (n, r, K), K ** -0.5, dtype)), R.followed(R.gauss(g, (n, N, r), 0.3, dtype))
    base, _ = R.inside(R.gauss(g, (T, N), 1.0, dtype))
    scales = torch.rand(n, generator=g, device="cuda") * 2 - 0.5
    ranks = torch.randint(0, r + 1, (n,), generator=g, device="cuda").to(torch.int32)
    for pattern, w_, base_, s_, r_ in (("mixed", w, None, scales, None), ("runs", w, base, scales, ranks),
                                       ("mixed", None, base, None, ranks), ("one", None, None, scales, None),
                                       ("none", w, None, None, None)):
        ids = _ids(g, T, n, pattern)
        if r_ is not None:   # what lies behind an adapter's own rank takes no part
            av, bv = a.clone(), b.clone()
            for e in range(n):
                av[e, int(r_[e]):] = float("nan")
                bv[e, :, int(r_[e]):] = float("nan")
        else:
            av, bv = a, b
        y = _run(d, x, w_, av, bv, ids, base_, s_, r_, dtype)
        ref, bound = R.lora(x, w_, a, b, ids, base_, s_, r_, dtype)
        R.assert_close(y, ref, bound, pattern, 2 * R.half_step(dtype))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,N,n,r", SHAPES)
def test_integers_are_exact(T, K, N, n, r, dtype):
    # |x A^T| stays below 256 (32 terms of at most 2 a row, seeds checked
    # here), so its 16-bit rounding is exact, and so is every sum
    g = _gen(T * 3 + N)
    d = M.make_lora_desc(K, N, n, r, R.DT[dtype])
    x, _ = R.inside(R.ints(g, (T, K), 2, dtype))
    w = R.followed(R.ints(g, (N, K), 2, dtype))
    a = R.followed(R.ints(g, (n, r, K), 1, dtype, min(1.0, 32.0 / K)))
    b = R.followed(R.ints(g, (n, N, r), 2, dtype))
    base, _ = R.inside(R.ints(g, (T, N), 3, dtype))
    scales = 2.0 ** torch.randint(-1, 2, (n,), generator=g, device="cuda").float()
    ranks = torch.randint(0, r + 1, (n,), generator=g, device="cuda").to(torch.int32)
    mid = x.double() @ a.double().reshape(n * r, K).t()
    assert mid.abs().max() <= 128
    for pattern in ("mixed", "runs"):
        ids = _ids(g, T, n, pattern)
        y = _run(d, x, w, a, b, ids, base, scales, ranks, dtype)
        ref, _ = R.lora(x, w, a, b, ids, base, scales, ranks, dtype)
        assert torch.equal(y, ref.to(dtype)), pattern


@pytest.mark.parametrize("T", [3, 64, 200, 700])
def test_an_adapters_infinities_stay_with_its_tokens(T):
    g = _gen(T)
    dtype = torch.float16
    K, N, n, r = 264, 136, 6, 16
    d = M.make_lora_desc(K, N, n, r, M.DT_F16)
    x, w = R.gauss(g, (T, K), 1.0, dtype), R.gauss(g, (N, K), 0.06, dtype)
    a, b = R.gauss(g, (n, r, K), 0.06, dtype), R.gauss(g, (n, N, r), 0.3, dtype)
    ids = _ids(g, T, n, "mixed")
    ids[0], ids[1] = 2, 3
    clean = _run(d, x, w, a, b, ids, None, None, None, dtype)
    a[2, 3, 7] = float("inf")
    b[2, 5, 1] = float("nan")
    b[4] = float("inf")
    y = _run(d, x, w, a, b, ids, None, None, None, dtype)
    others = (ids != 2) & (ids != 4)
    assert torch.equal(y[others], clean[others])
    assert not torch.isfinite(y[ids == 2]).all(1).any()
    # a token's own NaN stays in its row as well
    x[1, 9] = float("nan")
    z = _run(d, x, w, a, b, ids, None, None, None, dtype)
    others[1] = False
    assert torch.equal(z[others], clean[others]) and torch.isnan(z[1]).all()


@pytest.mark.parametrize("T", [5, 130, 600])
def test_base_in_place_and_rows_without_an_adapter(T):
    g = _gen(T + 1)
    dtype = torch.bfloat16
    K, N, n, r = 520, 264, 4, 32
    d = M.make_lora_desc(K, N, n, r, M.DT_BF16)
    x, a, b = R.gauss(g, (T, K), 1.0, dtype), R.gauss(g, (n, r, K), 0.04, dtype), R.gauss(g, (n, N, r), 0.3, dtype)
    ids = _ids(g, T, n, "mixed")
    ids[0] = -1
    base = R.gauss(g, (T, N), 1.0, dtype)
    want = _run(d, x, None, a, b, ids, base, None, None, dtype)
    y = base.clone()
    M.lora_linear(d, x, None, a, b, ids, y, R.poisoned(M.lora_workspace_size(d, T)), base=y)
    assert torch.equal(y, want)
    assert torch.equal(y[ids < 0], base[ids < 0])


@pytest.mark.parametrize("T", [4, 70, 300])
def test_bad_ids_and_ranks_are_reported_and_left_out(T):
    g = _gen(T + 2)
    dtype = torch.bfloat16
    K, N, n, r = 264, 128, 4, 16
    d = M.make_lora_desc(K, N, n, r, M.DT_BF16)
    x, w = R.gauss(g, (T, K), 1.0, dtype), R.gauss(g, (N, K), 0.06, dtype)
    a, b = R.gauss(g, (n, r, K), 0.06, dtype), R.gauss(g, (n, N, r), 0.3, dtype)
    ids = _ids(g, T, n, "mixed")
    y = torch.empty(T, N, dtype=dtype, device="cuda")
    ws = R.poisoned(M.lora_workspace_size(d, T))
    bad = ids.clone()
    bad[0], bad[1], bad[-1] = n, -2, 2 ** 31 - 1
    M.lora_linear(d, x, w, a, b, bad, y, ws)
    assert M.status(ws) == M.STATUS_BAD_INDEX
    none = torch.where((bad < 0) | (bad >= n), -1, bad).to(torch.int32)
    assert torch.equal(y, _run(d, x, w, a, b, none, None, None, None, dtype))
    ranks = torch.tensor([3, -1, 17, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    M.lora_linear(d, x, w, a, b, ids, y, ws, ranks=ranks)
    assert M.status(ws) == M.STATUS_BAD_WIDTH
    held = ranks.clamp(0, r)
    assert torch.equal(y, _run(d, x, w, a, b, ids, None, None, held, dtype))


@pytest.mark.parametrize("T", [1, 3, 70, 300, 5000])
def test_ranks_of_adapters_without_tokens_are_not_read(T):
    # a stack of many adapters costs what its named ones cost: a rank that no
    # token asks for is no fault, the last token's is
    g = _gen(T + 7)
    K, N, n, r = 72, 64, 3000, 8
    d = M.make_lora_desc(K, N, n, r, M.DT_F16)
    half = torch.float16
    x, w = R.gauss(g, (T, K), 1.0, half), R.gauss(g, (N, K), 0.1, half)
    a, b = R.gauss(g, (n, r, K), 0.1, half), R.gauss(g, (n, N, r), 0.3, half)
    ids = torch.randint(0, 50, (T,), generator=g, device="cuda").to(torch.int32)
    ids[-1] = n - 1
    ranks = torch.full((n,), -5, dtype=torch.int32, device="cuda")
    ranks[:50], ranks[n - 1] = 5, 8
    y, ws = torch.empty(T, N, dtype=half, device="cuda"), R.poisoned(M.lora_workspace_size(d, T))
    M.lora_linear(d, x, w, a, b, ids, y, ws, ranks=ranks)
    assert M.status(ws) == 0
    ranks[n - 1] = 9
    z = torch.empty_like(y)
    M.lora_linear(d, x, w, a, b, ids, z, ws, ranks=ranks)
    assert M.status(ws) == M.STATUS_BAD_WIDTH and torch.equal(y, z)


@pytest.mark.parametrize("T,K,N", [(1, 1032, 264), (48, 1032, 264), (200, 1032, 264), (900, 1032, 264), (100, 8200, 264)])
def test_a_tokens_row_does_not_depend_on_its_neighbours(T, K, N):
    # the same token and adapter among other tokens and ids: the same bits
    # (the calls take the same number of tokens, hence the same kernels)
    g = _gen(T + 3)
    dtype = torch.bfloat16
    n, r = 9, 24
    d = M.make_lora_desc(K, N, n, r, M.DT_BF16)
    x, w = R.gauss(g, (T, K), 1.0, dtype), R.gauss(g, (N, K), 0.03, dtype)
    a, b = R.gauss(g, (n, r, K), 0.03, dtype), R.gauss(g, (n, N, r), 0.3, dtype)
    ids = _ids(g, T, n, "mixed")
    first = _run(d, x, w, a, b, ids, None, None, None, dtype)
    perm = torch.randperm(T, generator=g, device="cuda")
    second = _run(d, x[perm].contiguous(), w, a, b, ids[perm].contiguous(), None, None, None, dtype)
    assert torch.equal(second, first[perm])


@pytest.mark.parametrize("T", [1, 50, 333, 3000])
def test_ids_scales_and_ranks_inside_longer_arrays(T):
    # a chunk of a batch, one layer's rows of a table: any 4-byte alignment, and
    # what stands around them takes no part
    g = _gen(T + 11)
    half = torch.float16
    K, N, n, r = 72, 64, 5, 16
    d = M.make_lora_desc(K, N, n, r, M.DT_F16)
    x, w = R.gauss(g, (T, K), 1.0, half), R.gauss(g, (N, K), 0.1, half)
    a, b = R.gauss(g, (n, r, K), 0.1, half), R.gauss(g, (n, N, r), 0.3, half)
    ids, scales = _ids(g, T, n, "mixed"), torch.rand(n, generator=g, device="cuda") + 0.5
    ranks = torch.randint(1, r + 1, (n,), generator=g, device="cuda").to(torch.int32)
    want = _run(d, x, w, a, b, ids, None, scales, ranks, half)
    for shift in (1, 2, 3):
        inner = [torch.full((t.numel() + 8,), 2 ** 30, dtype=t.dtype, device="cuda")[shift:shift + t.numel()].copy_(t)
                 for t in (ids, scales, ranks)]
        assert torch.equal(_run(d, x, w, a, b, inner[0], None, inner[1], inner[2], half), want)


@pytest.mark.parametrize("T", [1, 40, 300])
def test_stacks_of_more_than_4_gib(T):
    # the last adapters of a long stack, against the same two in a short one
    g = _gen(T + 13)
    half = torch.float16
    K, N, r, n = 8192, 136, 256, 1100
    x, w = R.gauss(g, (T, K), 1.0, half), R.gauss(g, (N, K), 0.01, half)
    a, b = R.gauss(g, (2, r, K), 0.01, half), R.gauss(g, (2, N, r), 0.1, half)
    ids = torch.randint(0, 2, (T,), generator=g, device="cuda").to(torch.int32)
    want = _run(M.make_lora_desc(K, N, 2, r, M.DT_F16), x, w, a, b, ids, None, None, None, half)
    long_a, long_b = torch.empty(n, r, K, dtype=half, device="cuda"), torch.empty(n, N, r, dtype=half, device="cuda")
    long_a[-2:], long_b[-2:] = a, b
    got = _run(M.make_lora_desc(K, N, n, r, M.DT_F16), x, w, long_a, long_b, ids + (n - 2), None, None, None, half)
    # (the stack's length has a part in the choice of tiles: not the same bits)
    ref, bound = R.lora(x, w, a, b, ids, None, None, None, half)
    R.assert_close(got, ref, bound, "long")
    R.assert_close(want, ref, bound, "short")


def test_zero_tokens_and_workspace_reuse():
    g = _gen(5)
    dtype = torch.float16
    K, N, n, r = 520, 200, 5, 16
    d = M.make_lora_desc(K, N, n, r, M.DT_F16)
    w, a, b = R.gauss(g, (N, K), 0.04, dtype), R.gauss(g, (n, r, K), 0.04, dtype), R.gauss(g, (n, N, r), 0.3, dtype)
    ws = R.poisoned(M.lora_workspace_size(d, 900))
    for T in (900, 200, 64, 3, 0):
        x, ids = R.gauss(g, (T, K), 1.0, dtype), _ids(g, T, n, "mixed")
        y = torch.empty(T, N, dtype=dtype, device="cuda")
        M.lora_linear(d, x, w, a, b, ids, y, ws)
        if T:
            assert torch.equal(y, _run(d, x, w, a, b, ids, None, None, None, dtype))


def test_binding_refuses():
    d = M.make_lora_desc(256, 128, 3, 16, M.DT_BF16)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, w, y = torch.zeros(4, 256, **bf), torch.zeros(128, 256, **bf), torch.zeros(4, 128, **bf)
    a, b = torch.zeros(3, 16, 256, **bf), torch.zeros(3, 128, 16, **bf)
    ids = torch.zeros(4, dtype=torch.int32, device="cuda")
    ws = R.poisoned(M.lora_workspace_size(d, 4))
    good = dict(x=x, w=w, a=a, b=b, ids=ids, y=y, ws=ws, base=None, scales=None, ranks=None)
    for kw in (dict(x=x.half()), dict(w=w[:64]), dict(a=a[:2]), dict(a=a.transpose(1, 2)), dict(b=b.transpose(1, 2)),
               dict(ids=ids.long()), dict(ids=ids[:3]), dict(ids=ids.cpu()), dict(y=y[:, :120]), dict(base=y.float()),
               dict(base=y[:1].expand(4, 128)), dict(scales=torch.ones(3, **bf)), dict(scales=torch.ones(2, device="cuda")),
               dict(ranks=ids[:2]), dict(ws=None)):
        c = dict(good)
        c.update(kw)
        with pytest.raises(ValueError):
            M.lora_linear(d, c["x"], c["w"], c["a"], c["b"], c["ids"], c["y"], c["ws"], base=c["base"],
                          scales=c["scales"], ranks=c["ranks"])
