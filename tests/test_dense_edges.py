"""The dense operators' C entries at their edges: calls that return from the
host's checks, no GPU is needed."""
import trellis_quantized_moe_exl3_amd as M
from test_dense_abi import _bwd, _glu_desc


def test_gradient_of_no_tokens_alone():
    # dx of no tokens has no elements and, from torch, no address; no gradient at
    # all of some tokens is a mistake
    none = dict(dx=None, dwg=None, dwu=None)
    assert _bwd(_glu_desc(), T=0, x=None, pre=None, dh=None, **none) == M.OK
    assert _bwd(_glu_desc(), T=1, **none) == M.ERR_INVALID_ARG
    assert _bwd(_glu_desc(), T=0, dx=None, dwg=None) == M.ERR_INVALID_ARG
