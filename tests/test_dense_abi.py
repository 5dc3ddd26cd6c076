"""Refusals of the dense operators' C entries (the gated feed-forward block and
the projection with adapters): every call here returns from the argument
checks, no GPU is needed."""
import ctypes as C

import pytest

import trellis_quantized_moe_exl3_amd as M

BIG = 1 << 44   # a workspace size that is always enough


def _glu_desc(hidden=512, inter=256, act_dtype=M.DT_BF16, act=M.ACT_SILU):
    return M.make_glu_desc(hidden, inter, act_dtype, act)


def _lora_desc(n_in=512, n_out=256, n_adapters=4, rank=16, act_dtype=M.DT_BF16):
    return M.make_lora_desc(n_in, n_out, n_adapters, rank, act_dtype)


@pytest.mark.parametrize("kw,code", [
    (dict(hidden=0), M.ERR_INVALID_ARG), (dict(hidden=-8), M.ERR_INVALID_ARG), (dict(hidden=100), M.ERR_INVALID_ARG),
    (dict(inter=4), M.ERR_INVALID_ARG), (dict(hidden=65544), M.ERR_UNSUPPORTED),
    (dict(inter=131072), M.ERR_UNSUPPORTED), (dict(act_dtype=M.DT_F32), M.ERR_UNSUPPORTED),
    (dict(act_dtype=M.DT_FP8), M.ERR_UNSUPPORTED), (dict(act=2), M.ERR_UNSUPPORTED), (dict(act=-1), M.ERR_UNSUPPORTED),
    (dict(hidden=65536, inter=65536), M.ERR_UNSUPPORTED),
])
def test_glu_desc_refused(kw, code):
    n = C.c_size_t(0)
    d = _glu_desc(**kw)
    assert M.lib().moe_exl3_glu_workspace_size(C.byref(d), 8, C.byref(n)) == code
    assert M.lib().moe_exl3_glu_backward_workspace_size(C.byref(d), 8, C.byref(n)) == code
    assert _glu(d) == code and _bwd(d) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n_in=4), M.ERR_INVALID_ARG), (dict(n_out=0), M.ERR_INVALID_ARG), (dict(n_adapters=0), M.ERR_INVALID_ARG),
    (dict(rank=4), M.ERR_INVALID_ARG), (dict(rank=264), M.ERR_UNSUPPORTED), (dict(n_adapters=65537), M.ERR_UNSUPPORTED),
    (dict(act_dtype=0), M.ERR_UNSUPPORTED), (dict(n_in=65536, n_out=65536), M.ERR_UNSUPPORTED),
])
def test_lora_desc_refused(kw, code):
    n = C.c_size_t(0)
    d = _lora_desc(**kw)
    assert M.lib().moe_exl3_lora_workspace_size(C.byref(d), 8, C.byref(n)) == code
    assert _lora(d) == code


def test_null_descriptors_and_sizes():
    n = C.c_size_t(0)
    for f in ("moe_exl3_glu_workspace_size", "moe_exl3_glu_backward_workspace_size", "moe_exl3_lora_workspace_size"):
        assert getattr(M.lib(), f)(None, 8, C.byref(n)) == M.ERR_INVALID_ARG
    d, e = _glu_desc(), _lora_desc()
    assert M.lib().moe_exl3_glu_workspace_size(C.byref(d), 8, None) == M.ERR_INVALID_ARG
    assert M.lib().moe_exl3_glu_workspace_size(C.byref(d), -1, C.byref(n)) == M.ERR_INVALID_ARG
    assert M.lib().moe_exl3_lora_workspace_size(C.byref(e), -1, C.byref(n)) == M.ERR_INVALID_ARG
    # 2 GiB of 16-bit rows
    assert M.lib().moe_exl3_glu_workspace_size(C.byref(d), 1 << 21, C.byref(n)) == M.ERR_UNSUPPORTED
    assert M.lib().moe_exl3_glu_workspace_size(C.byref(d), 1 << 62, C.byref(n)) == M.ERR_UNSUPPORTED
    assert M.lib().moe_exl3_lora_workspace_size(C.byref(e), 1 << 40, C.byref(n)) == M.ERR_UNSUPPORTED


@pytest.mark.parametrize("size", ["glu", "backward", "lora"])
@pytest.mark.parametrize("a,b", [(8, 8), (4096, 2048), (1032, 1384), (16384, 256), (256, 16384)])
def test_workspace_never_shrinks_with_tokens(size, a, b):
    fn = {"glu": lambda t: M.glu_workspace_size(_glu_desc(a, b), t),
          "backward": lambda t: M.glu_backward_workspace_size(_glu_desc(a, b), t),
          "lora": lambda t: M.lora_workspace_size(_lora_desc(a, b, 8, 64), t)}[size]
    last = 0
    for t in list(range(0, 300)) + [511, 512, 513, 1000, 2048, 4096, 4097, 7168, 16384]:
        n = fn(t)
        assert n >= last and n >= 256, (t, n, last)
        last = n


# distinct, aligned, far apart addresses; never read
X, WG, WU, OUT, PRE, WS, DH, DX, DWG, DWU = (0x1000_0000_0000 + 0x10_0000_0000 * i for i in range(10))


def _glu(d, x=X, ldx=None, wg=WG, wu=WU, T=8, out=OUT, ldo=None, pre=PRE, ws=WS, n=BIG):
    return M.lib().moe_exl3_glu(C.byref(d), x, d.hidden if ldx is None else ldx, wg, wu, T, out,
                                d.inter if ldo is None else ldo, pre, ws, n, None)


def _bwd(d, x=X, ldx=None, wg=WG, wu=WU, pre=PRE, dh=DH, ldh=None, T=8, dx=DX, lddx=None, dwg=DWG, dwu=DWU, ws=WS, n=BIG):
    return M.lib().moe_exl3_glu_backward(C.byref(d), x, d.hidden if ldx is None else ldx, wg, wu, pre, dh,
                                         d.inter if ldh is None else ldh, T, dx, d.hidden if lddx is None else lddx,
                                         dwg, dwu, ws, n, None)


def _lora(d, x=X, ldx=None, w=WG, a=WU, b=DWG, scales=None, ranks=None, ids=PRE, base=None, ldb=None, T=8, y=OUT,
          ldy=None, ws=WS, n=BIG, null=False):
    ad = M.LoraAdapters(a, b, scales, ranks)
    return M.lib().moe_exl3_lora_linear(C.byref(d), x, d.n_in if ldx is None else ldx, w, None if null else C.byref(ad),
                                        ids, base, d.n_out if ldb is None else ldb, T, y,
                                        d.n_out if ldy is None else ldy, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), M.ERR_INVALID_ARG), (dict(wg=None), M.ERR_INVALID_ARG), (dict(wu=None), M.ERR_INVALID_ARG),
    (dict(out=None), M.ERR_INVALID_ARG), (dict(ws=None), M.ERR_INVALID_ARG), (dict(T=-1), M.ERR_INVALID_ARG),
    (dict(ldx=504), M.ERR_INVALID_ARG), (dict(ldo=0), M.ERR_INVALID_ARG), (dict(ldo=-256), M.ERR_INVALID_ARG),
    (dict(ldx=516), M.ERR_MISALIGNED), (dict(x=X + 8), M.ERR_MISALIGNED), (dict(wg=WG + 2), M.ERR_MISALIGNED),
    (dict(out=OUT + 4), M.ERR_MISALIGNED), (dict(pre=PRE + 4), M.ERR_MISALIGNED), (dict(ws=WS + 16), M.ERR_MISALIGNED),
    (dict(ldx=(1 << 20) + 8), M.ERR_UNSUPPORTED), (dict(T=1 << 22), M.ERR_UNSUPPORTED),
    (dict(T=1 << 62), M.ERR_UNSUPPORTED), (dict(T=3000, ldx=1 << 20), M.ERR_UNSUPPORTED), (dict(n=128), M.ERR_WORKSPACE),
    # outputs over inputs or each other
    (dict(out=X), M.ERR_INVALID_ARG), (dict(out=X + 16), M.ERR_INVALID_ARG), (dict(out=WG), M.ERR_INVALID_ARG),
    (dict(out=WU + 16), M.ERR_INVALID_ARG), (dict(pre=OUT), M.ERR_INVALID_ARG), (dict(pre=X), M.ERR_INVALID_ARG),
    # a column range of x's own rows that meets it, one that does not fit behind it
    (dict(ldx=768, ldo=768, out=X + 2 * 504), M.ERR_INVALID_ARG),
    (dict(ldx=760, ldo=760, out=X + 2 * 512), M.ERR_INVALID_ARG),
    (dict(ldx=768, ldo=776, out=X + 2 * 512), M.ERR_INVALID_ARG),
])
def test_glu_refused(kw, code):
    assert _glu(_glu_desc(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), M.ERR_INVALID_ARG), (dict(pre=None), M.ERR_INVALID_ARG), (dict(dh=None), M.ERR_INVALID_ARG),
    (dict(wg=None), M.ERR_INVALID_ARG), (dict(dwg=None), M.ERR_INVALID_ARG), (dict(dwu=None), M.ERR_INVALID_ARG),
    (dict(dx=None, dwg=None, dwu=None), M.ERR_INVALID_ARG), (dict(T=-5), M.ERR_INVALID_ARG),
    # a broadcast gradient (stride 0) has to be written out first
    (dict(ldh=0), M.ERR_INVALID_ARG),
    (dict(pre=PRE + 8), M.ERR_MISALIGNED), (dict(dh=DH + 2), M.ERR_MISALIGNED), (dict(dwu=DWU + 8), M.ERR_MISALIGNED),
    (dict(lddx=516), M.ERR_MISALIGNED), (dict(n=256), M.ERR_WORKSPACE), (dict(T=1 << 22), M.ERR_UNSUPPORTED),
    (dict(dx=X), M.ERR_INVALID_ARG), (dict(dx=DH), M.ERR_INVALID_ARG), (dict(dx=PRE), M.ERR_INVALID_ARG),
    (dict(dwg=WG), M.ERR_INVALID_ARG), (dict(dwg=DWU), M.ERR_INVALID_ARG), (dict(dx=DWU), M.ERR_INVALID_ARG),
    (dict(T=0, n=0), M.ERR_WORKSPACE),
])
def test_glu_backward_refused(kw, code):
    assert _bwd(_glu_desc(), **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), M.ERR_INVALID_ARG), (dict(a=None), M.ERR_INVALID_ARG), (dict(b=None), M.ERR_INVALID_ARG),
    (dict(ids=None), M.ERR_INVALID_ARG), (dict(y=None), M.ERR_INVALID_ARG), (dict(null=True), M.ERR_INVALID_ARG),
    (dict(T=-1), M.ERR_INVALID_ARG), (dict(ldy=248), M.ERR_INVALID_ARG), (dict(base=DX, ldb=0), M.ERR_INVALID_ARG),
    (dict(ids=PRE + 2), M.ERR_MISALIGNED), (dict(a=WU + 2), M.ERR_MISALIGNED), (dict(scales=DX + 2), M.ERR_MISALIGNED),
    (dict(ranks=DX + 1), M.ERR_MISALIGNED), (dict(w=WG + 8), M.ERR_MISALIGNED), (dict(ldx=514), M.ERR_MISALIGNED),
    (dict(ws=WS + 128), M.ERR_MISALIGNED), (dict(n=256), M.ERR_WORKSPACE), (dict(T=1 << 22), M.ERR_UNSUPPORTED),
    (dict(y=X), M.ERR_INVALID_ARG), (dict(y=WG), M.ERR_INVALID_ARG), (dict(y=WU + 64), M.ERR_INVALID_ARG),
    (dict(y=DWG), M.ERR_INVALID_ARG), (dict(y=PRE), M.ERR_INVALID_ARG),
    # base may be y, but not shifted against it
    (dict(base=OUT + 16), M.ERR_INVALID_ARG), (dict(base=OUT, ldb=512), M.ERR_INVALID_ARG),
])
def test_lora_refused(kw, code):
    assert _lora(_lora_desc(), **kw) == code


def test_zero_tokens_return_before_any_launch():
    assert _glu(_glu_desc(), T=0, x=None, out=None, ws=None) == M.OK
    assert _lora(_lora_desc(), T=0, x=None, y=None, ids=None, ws=None) == M.OK
    # dx alone of no tokens: nothing to write
    assert _bwd(_glu_desc(), T=0, x=None, pre=None, dh=None, dwg=None, dwu=None) == M.OK
