"""Refusals of the C entries around a MoE layer's own experts (sort, dispatch,
combine, dropout, 4-bit products) and of their binding, the counter-based
generator's published answers: no GPU is needed."""
import ctypes as C

import numpy as np
import pytest
import torch

import experts_ref as R
import trellis_quantized_moe_exl3_amd as M

BIG = 1 << 44
# distinct, aligned, far apart addresses; never read
A = [0x1000_0000_0000 + 0x100_0000_0000 * i for i in range(12)]
INV, UNS, MIS, WSP = M.ERR_INVALID_ARG, M.ERR_UNSUPPORTED, M.ERR_MISALIGNED, M.ERR_WORKSPACE


def test_generator_known_answers():
    # the method's published answers (Random123's kat_vectors: philox4x32 10)
    assert [hex(v) for v in R.philox([0], 0)[0]] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]


def _tokens(**kw):
    return M.make_tokens_desc(**{**dict(hidden=512, n_experts=40, top_k=4), **kw})


def _w4d(**kw):
    return M.make_w4_desc(**{**dict(n_in=512, n_out=256, n_experts=4, group=64), **kw})


def _sort(d, idx=A[0], T=8, counts=A[1], offsets=A[2], ids=A[3], pos=A[4], ws=A[5], n=BIG):
    return M.lib().moe_exl3_sort(C.byref(d), idx, T, counts, offsets, ids, pos, ws, n, None)


def _dispatch(d, x=A[0], ldx=512, pos=A[1], w=A[2], T=8, rows=32, out=A[3], ldo=512):
    return M.lib().moe_exl3_dispatch(C.byref(d), x, ldx, pos, w, T, rows, out, ldo, None)


def _dispatch_b(d, g=A[0], ldg=512, x=A[1], ldx=512, pos=A[2], w=A[3], T=8, rows=32, dx=A[4], lddx=512, dw=A[5]):
    return M.lib().moe_exl3_dispatch_backward(C.byref(d), g, ldg, x, ldx, pos, w, T, rows, dx, lddx, dw, None)


def _drop(p, rng):
    return None if p is None else C.byref(M.Drop(p, rng))


def _combine(d, z=A[0], ldz=512, pos=A[1], w=A[2], base=A[3], ldb=512, p=0.5, rng=A[4], T=8, rows=32, y=A[5], ldy=512):
    return M.lib().moe_exl3_combine(C.byref(d), z, ldz, pos, w, base, ldb, _drop(p, rng), T, rows, y, ldy, None)


def _combine_b(d, dy=A[0], lddy=512, z=A[1], ldz=512, pos=A[2], w=A[3], p=0.5, rng=A[4], T=8, rows=32, dz=A[5], lddz=512,
               dw=A[6]):
    return M.lib().moe_exl3_combine_backward(C.byref(d), dy, lddy, z, ldz, pos, w, _drop(p, rng), T, rows, dz, lddz, dw,
                                             None)


def _dropout(dt=M.DT_BF16, x=A[0], ldx=100, res=A[1], ldr=100, p=0.5, rng=A[2], rows=8, cols=100, y=A[3], ldy=100):
    return M.lib().moe_exl3_dropout(dt, x, ldx, res, ldr, _drop(p, rng), rows, cols, y, ldy, None)


def _w4(d, x=A[0], ldx=512, codes=A[1], scales=A[2], zeros=A[3], offsets=A[4], base=A[5], ldb=256, rows=8, y=A[6], ldy=256,
        ws=A[7], n=BIG, null=False, glu=False, codes2=A[8], null2=False):
    w, u = M.W4Weights(codes, scales, zeros), M.W4Weights(codes2, scales, zeros)
    if glu:
        return M.lib().moe_exl3_w4_glu(C.byref(d), x, ldx, None if null else C.byref(w), None if null2 else C.byref(u),
                                       offsets, rows, y, ldy, ws, n, None)
    return M.lib().moe_exl3_w4_linear(C.byref(d), x, ldx, None if null else C.byref(w), offsets, base, ldb, rows, y, ldy,
                                      ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(hidden=0), INV), (dict(hidden=-8), INV), (dict(hidden=100), INV), (dict(hidden=65544), UNS),
    (dict(n_experts=0), INV), (dict(n_experts=-1), INV), (dict(n_experts=1025), UNS), (dict(top_k=0), INV),
    (dict(top_k=17), UNS), (dict(act_dtype=M.DT_F32), UNS), (dict(act_dtype=M.DT_FP8), UNS),
])
def test_tokens_desc_refused(kw, code):
    n = C.c_size_t(0)
    d = _tokens(**kw)
    assert M.lib().moe_exl3_sort_workspace_size(C.byref(d), 8, C.byref(n)) == code
    for f in (_sort, _dispatch, _dispatch_b, _combine, _combine_b):
        assert f(d) == code


@pytest.mark.parametrize("kw,code", [
    (dict(n_in=0), INV), (dict(n_in=100), INV), (dict(n_in=96), INV), (dict(n_out=4), INV), (dict(n_out=0), INV),
    (dict(n_in=65600), UNS), (dict(n_out=65544), UNS), (dict(group=16), UNS), (dict(group=0), UNS), (dict(group=256), UNS),
    (dict(n_experts=0), INV), (dict(n_experts=1025), UNS), (dict(act_dtype=M.DT_F32), UNS), (dict(act=2), UNS),
    (dict(act=-1), UNS), (dict(n_in=65536, n_out=65536), UNS),
])
def test_w4_desc_refused(kw, code):
    n = C.c_size_t(0)
    d = _w4d(**kw)
    assert M.lib().moe_exl3_w4_workspace_size(C.byref(d), 8, C.byref(n)) == code
    assert _w4(d) == code and _w4(d, glu=True) == code


def test_null_descriptors_and_sizes():
    n = C.c_size_t(0)
    l = M.lib()
    assert l.moe_exl3_sort_workspace_size(None, 8, C.byref(n)) == INV
    assert l.moe_exl3_w4_workspace_size(None, 8, C.byref(n)) == INV
    assert l.moe_exl3_sort_workspace_size(C.byref(_tokens()), 8, None) == INV
    assert l.moe_exl3_sort_workspace_size(C.byref(_tokens()), -1, C.byref(n)) == INV
    assert l.moe_exl3_sort_workspace_size(C.byref(_tokens()), 1 << 29, C.byref(n)) == UNS   # 2^31 slots
    assert l.moe_exl3_w4_workspace_size(C.byref(_w4d()), 8, None) == INV
    assert l.moe_exl3_w4_workspace_size(C.byref(_w4d()), -1, C.byref(n)) == INV
    assert l.moe_exl3_w4_workspace_size(C.byref(_w4d()), 1 << 21, C.byref(n)) == UNS        # 2 GiB of rows
    assert l.moe_exl3_w4_workspace_size(C.byref(_w4d()), 1 << 62, C.byref(n)) == UNS


@pytest.mark.parametrize("E,k", [(1, 1), (40, 4), (1024, 16)])
def test_workspaces_never_shrink(E, k):
    last = 0
    for t in (0, 1, 2, 255, 256, 257, 4096, 4097, 16384, 20000, 100000, 1 << 24):
        n = M.sort_workspace_size(_tokens(n_experts=E, top_k=k), t)
        assert n >= last and n >= 256 and n % 256 == 0
        last = n
    last = 0
    for t in (0, 1, 16, 17, 64, 65, 1000, 4096, 50000, 1000000):
        n = M.w4_workspace_size(_w4d(n_experts=E), t)
        assert n >= last and n >= 256
        last = n


@pytest.mark.parametrize("kw,code", [
    (dict(idx=None), INV), (dict(offsets=None), INV), (dict(pos=None), INV), (dict(ws=None), INV), (dict(T=-1), INV),
    (dict(T=1 << 29), UNS), (dict(T=1 << 62), UNS), (dict(idx=A[0] + 2), MIS), (dict(counts=A[1] + 1), MIS),
    (dict(offsets=A[2] + 2), MIS), (dict(ids=A[3] + 3), MIS), (dict(pos=A[4] + 2), MIS), (dict(ws=A[5] + 16), MIS),
    (dict(n=128), WSP), (dict(T=2000, n=256), WSP), (dict(pos=A[0]), INV), (dict(ids=A[0] + 64), INV),
    (dict(pos=A[3]), INV), (dict(counts=A[2] + 4), INV), (dict(T=0, ws=None), INV), (dict(T=0, offsets=None), INV),
])
def test_sort_refused(kw, code):
    assert _sort(_tokens(), **kw) == code


ROWS = [
    (dict(pos=None), INV), (dict(T=-1), INV), (dict(rows=-1), INV), (dict(T=1 << 29), UNS), (dict(rows=1 << 31), UNS),
    (dict(T=1 << 62), UNS), (dict(w=A[10] + 2), MIS), (dict(pos=A[10] + 1), MIS),
]


@pytest.mark.parametrize("kw,code", ROWS + [
    (dict(x=None), INV), (dict(out=None), INV), (dict(ldx=504), INV), (dict(ldo=0), INV), (dict(ldx=516), MIS),
    (dict(ldo=514), MIS), (dict(x=A[0] + 8), MIS), (dict(out=A[3] + 2), MIS), (dict(ldx=(1 << 20) + 8), UNS),
    (dict(out=A[0]), INV), (dict(out=A[0] + 1024), INV), (dict(out=A[1]), INV), (dict(out=A[2]), INV),
])
def test_dispatch_refused(kw, code):
    assert _dispatch(_tokens(), **kw) == code


@pytest.mark.parametrize("kw,code", ROWS + [
    (dict(g=None), INV), (dict(x=None), INV), (dict(dx=None), INV), (dict(ldg=8), INV), (dict(ldx=0), INV),
    (dict(lddx=508), INV), (dict(lddx=516), MIS), (dict(g=A[0] + 4), MIS), (dict(dw=A[5] + 2), MIS),
    (dict(dx=A[0]), INV), (dict(dx=A[1]), INV), (dict(dx=A[2]), INV), (dict(dx=A[3]), INV), (dict(dx=A[5]), INV),
    (dict(dw=A[0]), INV), (dict(dw=A[1]), INV), (dict(dw=A[2]), INV), (dict(dw=A[3]), INV), (dict(dw=A[4] + 64), INV),
])
def test_dispatch_backward_refused(kw, code):
    assert _dispatch_b(_tokens(), **kw) == code


DROPS = [
    (dict(p=-0.1), INV), (dict(p=1.01), INV), (dict(p=float("nan")), INV), (dict(p=float("inf")), INV), (dict(rng=None), INV),
    (dict(rng=A[10] + 4), MIS),
]


@pytest.mark.parametrize("kw,code", ROWS + DROPS + [
    (dict(z=None), INV), (dict(y=None), INV), (dict(ldz=0), INV), (dict(ldb=8), INV), (dict(ldy=516), MIS),
    (dict(base=A[3] + 2), MIS), (dict(y=A[0]), INV), (dict(y=A[1]), INV), (dict(y=A[2]), INV), (dict(y=A[4]), INV),
    # base may be y, but not shifted against it
    (dict(y=A[3] + 16), INV), (dict(y=A[3], ldy=520), INV),
])
def test_combine_refused(kw, code):
    assert _combine(_tokens(), **kw) == code


@pytest.mark.parametrize("kw,code", ROWS + DROPS + [
    (dict(dy=None), INV), (dict(z=None), INV), (dict(dz=None), INV), (dict(lddy=0), INV), (dict(lddz=516), MIS),
    (dict(dw=A[6] + 1), MIS), (dict(dz=A[0]), INV), (dict(dz=A[2]), INV), (dict(dz=A[3]), INV), (dict(dz=A[4]), INV),
    (dict(dz=A[6]), INV), (dict(dw=A[0]), INV), (dict(dw=A[1]), INV), (dict(dw=A[2]), INV), (dict(dw=A[3]), INV),
    (dict(dw=A[4]), INV), (dict(dz=A[1] + 16), INV), (dict(dz=A[1], lddz=520), INV),
])
def test_combine_backward_refused(kw, code):
    assert _combine_b(_tokens(), **kw) == code


@pytest.mark.parametrize("kw,code", DROPS + [
    (dict(dt=M.DT_FP8), UNS), (dict(dt=9), UNS), (dict(rows=-1), INV), (dict(cols=-1), INV), (dict(p=None), INV),
    (dict(x=None), INV), (dict(y=None), INV), (dict(ldx=99), INV), (dict(ldr=0), INV), (dict(ldy=-100), INV),
    (dict(cols=(1 << 20) + 1), UNS), (dict(ldx=(1 << 20) + 1), UNS), (dict(x=A[0] + 2), MIS), (dict(res=A[1] + 8), MIS),
    (dict(y=A[3] + 4), MIS), (dict(y=A[0] + 16), INV), (dict(y=A[0], ldy=104), INV), (dict(y=A[1], ldy=101), INV),
    (dict(y=A[2]), INV), (dict(rows=1 << 32), UNS), (dict(rows=1 << 62), UNS),
])
def test_dropout_refused(kw, code):
    assert _dropout(**kw) == code


@pytest.mark.parametrize("dt,size", [(M.DT_BF16, 2), (M.DT_F16, 2), (M.DT_F32, 4)])
def test_dropout_of_a_part_begins_at_16_bytes(dt, size):
    # rows of 1381: from row 16 / size on each 16th byte, not from those between.
    # (What passes the checks of addresses is refused for the generator inside y.)
    for row in range(1, 16 // size + 1):
        for name, base in (("x", A[0]), ("res", A[1]), ("y", A[3])):
            at = base + row * 1381 * size
            kw = {"rng": (at if name == "y" else A[3]) // 8 * 8 + 64, name: at}
            assert _dropout(dt=dt, ldx=1381, ldr=1381, ldy=1381, cols=1381, **kw) == (INV if row == 16 // size else MIS)


W4S = [
    (dict(x=None), INV), (dict(codes=None), INV), (dict(scales=None), INV), (dict(null=True), INV), (dict(y=None), INV),
    (dict(ws=None), INV), (dict(offsets=None), INV), (dict(rows=-1), INV), (dict(ldx=504), INV), (dict(ldy=0), INV),
    (dict(ldx=516), MIS), (dict(x=A[0] + 8), MIS), (dict(codes=A[1] + 4), MIS), (dict(scales=A[2] + 2), MIS),
    (dict(zeros=A[3] + 1), MIS), (dict(offsets=A[4] + 2), MIS), (dict(y=A[6] + 8), MIS), (dict(ws=A[7] + 16), MIS),
    (dict(n=128), WSP), (dict(rows=1 << 21), UNS), (dict(rows=1 << 62), UNS), (dict(ldx=(1 << 20) + 8), UNS),
    (dict(y=A[0]), INV), (dict(y=A[1] + 65536), INV), (dict(y=A[2]), INV), (dict(y=A[3]), INV), (dict(y=A[4]), INV),
]


@pytest.mark.parametrize("kw,code", W4S + [
    (dict(ldb=0), INV), (dict(base=A[5] + 2), MIS), (dict(y=A[5] + 16), INV), (dict(y=A[5], ldy=264), INV),
])
def test_w4_linear_refused(kw, code):
    assert _w4(_w4d(), **kw) == code


@pytest.mark.parametrize("kw,code", W4S + [(dict(codes2=None), INV), (dict(null2=True), INV), (dict(codes2=A[8] + 8), MIS),
                                           (dict(y=A[8]), INV)])
def test_w4_glu_refused(kw, code):
    assert _w4(_w4d(), glu=True, **kw) == code


@pytest.mark.parametrize("glu", [False, True])
def test_w4_takes_the_zeros_of_one_expert(glu):
    # N K / group is a multiple of 8, of 16 not always (1032 x 1376 in groups of
    # 32): where the next expert's zeros begin.  (128 bytes are too few: the
    # workspace is what is refused last)
    assert _w4(_w4d(), zeros=A[3] + 8, n=128, glu=glu) == WSP
    for off in (1, 2, 4, 12):
        assert _w4(_w4d(), zeros=A[3] + off, n=128, glu=glu) == MIS


def test_calls_without_work_return_before_any_launch():
    d = _tokens()
    assert _dispatch(d, T=0, x=None, pos=None, out=None) == M.OK
    assert _dispatch(d, rows=0, out=None) == M.OK
    assert _dispatch_b(d, T=0, g=None, x=None, pos=None, dx=None) == M.OK
    assert _combine(d, T=0, z=None, pos=None, y=None) == M.OK
    assert _combine_b(d, T=0, dy=None, pos=None, dz=None) == M.OK
    assert _combine_b(d, rows=0, dz=None, z=None, dw=None) == M.OK
    assert _dropout(rows=0, x=None, y=None, res=None) == M.OK and _dropout(cols=0) == M.OK
    assert _w4(_w4d(), rows=0, x=None, y=None, ws=None) == M.OK


def test_binding_refuses_what_the_kernels_could_not_read():
    # tensors on the CPU, of other types, shapes or strides: all before any call
    d = _tokens(hidden=16, n_experts=4, top_k=2)
    x, z = torch.zeros(3, 16, dtype=torch.bfloat16), torch.zeros(6, 16, dtype=torch.bfloat16)
    pos = torch.zeros(3, 2, dtype=torch.int32)
    rng = torch.zeros(2, dtype=torch.int64)
    calls = [lambda: M.dispatch(d, x, pos, z), lambda: M.combine(d, z, pos, x), lambda: M.dropout(x, x, 0.5, rng),
             lambda: M.dispatch_backward(d, z, x, pos, x), lambda: M.combine_backward(d, x, z, pos, z),
             lambda: M.sort(d, pos, None, pos, None, pos, rng)]
    for call in calls:
        with pytest.raises((ValueError, RuntimeError, AssertionError)):
            call()


def test_a_single_column_has_no_stride():
    # a row transposed is contiguous rows of one element, whatever the stride that
    # a tensor names for its columns
    f32 = (torch.float32,)
    row = torch.zeros(1, 5)
    assert row.t().stride() == (1, 5) and row.t().is_contiguous()
    assert M._rows(row.t(), 5, 1, f32, -1, "x") == 1
    assert M._rows(torch.zeros(5, 7)[:, 3:4], 5, 1, f32, -1, "x") == 7
    for t in (torch.zeros(2, 5).t(), torch.zeros(5, 4)[:, ::2]):
        with pytest.raises(ValueError):
            M._rows(t, 5, 2, f32, -1, "x")
    with pytest.raises(ValueError):
        M._rows(torch.zeros(1, 1).expand(5, 1), 5, 1, f32, -1, "x")


def test_weights_hold_the_memory_they_were_made_with():
    codes, scales = torch.zeros(2, 8, 16, dtype=torch.uint8), torch.ones(2, 8, 1, dtype=torch.bfloat16)
    w = M.make_w4(codes, scales)
    at = codes.data_ptr()
    codes.data = torch.ones(2, 8, 64, dtype=torch.uint8)   # other memory for the caller's tensor
    assert w.weights.codes == w.codes.data_ptr() == at and w.codes.shape == (2, 8, 16) and w.zeros is None
    with pytest.raises(AttributeError):
        w.codes = codes
    one = M.make_w4(codes[0], scales[0], torch.zeros(8, 1, dtype=torch.uint8))
    assert one.codes.shape == (1, 8, 64) and one.zeros.shape == (1, 8, 1)


def test_keep_matches_a_plain_loop():
    # the vectorised mask against single counters
    kept, f = R.keep(3, 11, 0.25, 9, 2 ** 64 - 2)
    assert f == 65536 / (65536 - 16384)
    for r in range(3):
        for c in range(11):
            words = R.philox([(2 ** 64 - 2 + 2 * r + c // 8) % 2 ** 64], 9)[0]
            half = int(words[c % 8 // 2]) >> 16 * (c % 2) & 0xFFFF
            assert bool(kept[r, c]) == (half >= 16384)
    assert np.uint32(1).nbytes == 4
