"""The dense operators at their edges: products between the two adapter
matrices that 16 bits do not hold, infinities, calls without tokens, one token's
kernel, and the tile variants that need long sums."""
import pytest
import torch

import dense_ref as R
import trellis_quantized_moe_exl3_amd as M

pytestmark = pytest.mark.gpu


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
