"""The dense operators at their edges: products between the two adapter
matrices that 16 bits do not hold, infinities, calls without tokens, one token's
kernel, and the tile variants that need long sums."""
import pytest
import torch

import dense_ref as R
import test_gpu_lora as L
import trellis_quantized_moe_exl3_amd as M

pytestmark = pytest.mark.gpu


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
