"""The dense operators at their edges: products between the two adapter
matrices that 16 bits do not hold, infinities, calls without tokens, one token's
kernel, and the tile variants that need long sums."""
import pytest
import torch

import dense_ref as R
import test_gpu_glu as G
import test_gpu_lora as L
import trellis_quantized_moe_exl3_amd as M

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]
FEW = [1, 2, 8, 17, 33, 64]   # tokens of the few-token kernel, in all its sizes


def _one_rank(T, n, r, dtype, value, times, b):
    """Adapters whose rank 0 gives times * value for a token of ones and adds b
    times that to every column; the other ranks are zero."""
    K, N = 1032, 72
    bf = dict(dtype=dtype, device="cuda")
    x, a, bm = torch.ones(T, K, **bf), torch.zeros(n, r, K, **bf), torch.zeros(n, N, r, **bf)
    a[:, 0, :times] = value
    bm[:, :, 0] = b
    ids = (torch.arange(T, device="cuda") % n).to(torch.int32)
    return M.make_lora_desc(K, N, n, r, R.DT[dtype]), x, a, bm, ids


# Sums that need one bit more than the type has: 257 = 2^8 + 1 (bf16), 2049 = 3 x 683
# (fp16).  Times 1, next to a base of -256 or -2048, 1 is left of them.
ODD = {torch.bfloat16: (1.0, 257, -256.0), torch.float16: (3.0, 683, -2048.0)}


@pytest.mark.parametrize("r", [8, 40])
@pytest.mark.parametrize("T", FEW)
@pytest.mark.parametrize("dtype", TYPES)
def test_few_tokens_keep_the_product_between_in_fp32(T, r, dtype):
    value, times, base = ODD[dtype]
    d, x, a, b, ids = _one_rank(T, 3, r, dtype, value, times, 1.0)
    base = torch.full((T, d.n_out), base, dtype=dtype, device="cuda")
    y = L._run(d, x, None, a, b, ids, base, None, None, dtype)
    assert (y == 1.0).all()
    assert torch.equal(L._run(d, x, torch.zeros(d.n_out, d.n_in, dtype=dtype, device="cuda"), a, b, ids, base, None,
                              None, dtype), y)


@pytest.mark.parametrize("r", [8, 40])
@pytest.mark.parametrize("T", [65, 300, 1100])
@pytest.mark.parametrize("dtype", TYPES)
def test_more_tokens_round_it_once(T, r, dtype):
    # to even: 256 and 2048
    value, times, base = ODD[dtype]
    d, x, a, b, ids = _one_rank(T, 3, r, dtype, value, times, 1.0)
    base = torch.full((T, d.n_out), base, dtype=dtype, device="cuda")
    assert (L._run(d, x, None, a, b, ids, base, None, None, dtype) == 0.0).all()


@pytest.mark.parametrize("r", [8, 40])
@pytest.mark.parametrize("T", FEW + [65, 300])
def test_products_beyond_fp16(T, r):
    # 70000 = 100 x 700 times 2^-4, and 2^-26 times 2^10 (a scale of 2^-26 on a sum
    # of 1): finite and not zero for few tokens, infinite and zero where the
    # product between is rounded
    d, x, a, b, ids = _one_rank(T, 3, r, torch.float16, 100.0, 700, 2.0 ** -4)
    y = L._run(d, x, None, a, b, ids, None, None, None, torch.float16)
    assert (y == (4376.0 if T <= 64 else float("inf"))).all()   # 4375 to a step of 4
    d, x, a, b, ids = _one_rank(T, 3, r, torch.float16, 1.0, 1, 1024.0)
    scales = torch.full((3,), 2.0 ** -26, device="cuda")
    y = L._run(d, x, None, a, b, ids, None, scales, None, torch.float16)
    assert (y == (2.0 ** -16 if T <= 64 else 0.0)).all()


@pytest.mark.parametrize("rank", [1, 4, 8, 13])
@pytest.mark.parametrize("T", [1, 8, 64, 65, 200, 700, 3900])
def test_an_infinite_token_with_ranks_below_the_stacks(T, rank):
    # positive matrices and an infinity in x: the row is infinite; ranks that
    # take no part must not make a NaN of it (infinity times nothing)
    g = L._gen(T + rank)
    dtype = torch.bfloat16
    K, N, n, r = 264, 4096 if T == 3900 else 136, 3, 24
    d = M.make_lora_desc(K, N, n, r, M.DT_BF16)
    x, w = R.gauss(g, (T, K), 1.0, dtype), R.gauss(g, (N, K), 0.06, dtype).abs() + 0.01
    a, b = R.gauss(g, (n, r, K), 0.06, dtype).abs() + 0.01, R.gauss(g, (n, N, r), 0.3, dtype).abs() + 0.01
    ids = L._ids(g, T, n, "mixed")
    ids[0] = 1
    ranks = torch.full((n,), rank, dtype=torch.int32, device="cuda")
    clean = [L._run(d, x, w_, a, b, ids, None, None, ranks, dtype) for w_ in (w, None)]
    x[0, 5] = float("inf")
    for w_, before in zip((w, None), clean):
        y = L._run(d, x, w_, a, b, ids, None, None, ranks, dtype)
        assert (y[0] == float("inf")).all()
        assert torch.equal(y[1:], before[1:])


@pytest.mark.parametrize("T", [1, 2, 40, 70, 116, 300, 1024, 4000])
@pytest.mark.parametrize("K,N,r", [(840, 1984, 32), (264, 4096, 72)])
def test_adapters_appended_to_a_long_stack_change_no_bits(T, K, N, r):
    g = L._gen(T + N)
    dtype = torch.bfloat16
    n, more = 64, 700   # a call is planned for 64 at most
    x, w = R.gauss(g, (T, K), 1.0, dtype), R.gauss(g, (N, K), K ** -0.5, dtype)
    a, b = R.gauss(g, (n, r, K), K ** -0.5, dtype), R.gauss(g, (n, N, r), 0.3, dtype)
    av, bv = (torch.full((more,) + t.shape[1:], float("nan"), dtype=dtype, device="cuda") for t in (a, b))
    av[:n], bv[:n] = a, b
    for w_ in (w, None):
        ids = L._ids(g, T, n, "mixed")
        want = L._run(M.make_lora_desc(K, N, n, r, M.DT_BF16), x, w_, a, b, ids, None, None, None, dtype)
        assert torch.equal(L._run(M.make_lora_desc(K, N, more, r, M.DT_BF16), x, w_, av, bv, ids, None, None, None, dtype), want)


@pytest.mark.parametrize("want_dx,want_dw", [(True, False), (False, True), (True, True)])
def test_no_tokens(want_dx, want_dw):
    # torch gives a tensor without elements no address
    H, I = 264, 136
    bf = dict(dtype=torch.bfloat16, device="cuda")
    d = M.make_glu_desc(H, I, M.DT_BF16)
    x, dh, w = torch.empty(0, H, **bf), torch.empty(0, I, **bf), torch.zeros(I, H, **bf)
    dw = [torch.full_like(w, 3.0) for _ in range(2)] if want_dw else [None, None]
    M.glu_backward(d, x, w, w, torch.empty(2, 0, I, device="cuda"), dh, R.poisoned(M.glu_backward_workspace_size(d, 0)),
                   dx=torch.empty_like(x) if want_dx else None, dw_gate=dw[0], dw_up=dw[1])
    assert not want_dw or all((t == 0).all() for t in dw)


@pytest.mark.parametrize("bad", [4, -2, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("K,N,r", [(2048, 4096, 16), (264, 72, 32), (1032, 136, 40)])
def test_one_token_with_a_bad_id(K, N, r, bad):
    g = L._gen(K + r)
    dtype = torch.bfloat16
    n = 4
    d = M.make_lora_desc(K, N, n, r, M.DT_BF16)
    x, w = R.gauss(g, (1, K), 1.0, dtype), R.gauss(g, (N, K), K ** -0.5, dtype)
    a, b = R.gauss(g, (n, r, K), K ** -0.5, dtype), R.gauss(g, (n, N, r), 0.3, dtype)
    y, ws = torch.empty(1, N, dtype=dtype, device="cuda"), R.poisoned(M.lora_workspace_size(d, 1))
    ranks = torch.full((n,), r + 1, dtype=torch.int32, device="cuda")   # not this token's: no fault of theirs
    M.lora_linear(d, x, w, a, b, torch.tensor([bad], device="cuda").to(torch.int32), y, ws, ranks=ranks)
    assert M.status(ws) == M.STATUS_BAD_INDEX
    none = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    assert torch.equal(y, L._run(d, x, w, a, b, none, None, None, None, dtype))


@pytest.mark.parametrize("K,N,r", [(2048, 4096, 16), (264, 72, 32), (1032, 136, 40)])
def test_one_token_and_another_adapters_infinities(K, N, r):
    g = L._gen(K + N)
    dtype = torch.float16
    n = 5
    d = M.make_lora_desc(K, N, n, r, M.DT_F16)
    x, w = R.gauss(g, (1, K), 1.0, dtype), R.gauss(g, (N, K), K ** -0.5, dtype)
    a, b = R.gauss(g, (n, r, K), K ** -0.5, dtype), R.gauss(g, (n, N, r), 0.3, dtype)
    base = R.gauss(g, (1, N), 1.0, dtype)
    ranks = torch.tensor([r, r - 3, 5, 8, 0], dtype=torch.int32, device="cuda")
    for e in range(n):
        ids = torch.full((1,), e, dtype=torch.int32, device="cuda")
        av, bv = torch.full_like(a, float("nan")), torch.full_like(b, float("inf"))
        av[e], bv[e] = a[e], b[e]
        y = L._run(d, x, w, av, bv, ids, base, None, ranks, dtype)
        ref, bound = R.lora(x, w, a, b, ids, base, None, ranks, dtype)
        R.assert_close(y, ref, bound, f"adapter {e}")
        y = L._run(d, x, w, av, bv, torch.full_like(ids, -1), base, None, ranks, dtype)
        ref, bound = R.lora(x, w, a, b, torch.full_like(ids, -1), base, None, ranks, dtype)
        R.assert_close(y, ref, bound, "none")


# The weights' gradients in 256 x 256 tiles of many stages: 400 tokens (12 full
# stages of 32 and half of one) and 520 (16 and a quarter); both gradients in
# 64 x 64 tiles of one launch, dx's blocks first; the weights' in eight splits
GRADIENTS = [(400, 16384, 264), (520, 520, 8192), (500, 256, 1032), (4100, 488, 120)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,I", GRADIENTS)
def test_gradients_in_long_tiles(T, H, I, dtype):
    G.test_backward(T, H, I, dtype)
    G.test_gradients_of_integers_are_exact(T, H, I, dtype)


# 256 x 256 tiles whose adapters take several stages of 32 ranks, the last of them
# partly; long k in those and in 128 x 128 tiles, alone on a CU and two on one
PROJECTIONS = [(3900, 264, 4096, 6, 72), (3900, 264, 4096, 3, 256), (3900, 1288, 4096, 3, 72), (1024, 2056, 4096, 6, 40),
               (2500, 1288, 2056, 4, 40)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,K,N,n,r", PROJECTIONS)
def test_projection_in_long_tiles(T, K, N, n, r, dtype):
    L.test_values(T, K, N, n, r, dtype)
    L.test_integers_are_exact(T, K, N, n, r, dtype)
