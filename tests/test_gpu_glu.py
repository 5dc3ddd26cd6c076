"""The gated feed-forward block and its backward pass against their definition
in 64 bits: values within bounds derived from the types, and integer inputs
for which every product and sum is exact and the result has to be equal."""
import pytest
import torch

import dense_ref as R
import trellis_quantized_moe_exl3_amd as M

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16]
ACTS = [M.ACT_SILU, M.ACT_GELU_TANH]
# tokens around the tile and fragment edges; sizes that end inside a stage of
# 32, a tile of 64 or 128 columns and a 16-row block
SHAPES = [(1, 256, 128), (1, 8, 8), (2, 264, 40), (7, 520, 136), (8, 4096, 2048), (15, 40, 72), (16, 1032, 200),
          (17, 256, 264), (31, 72, 1000), (33, 1032, 1384), (63, 512, 64), (64, 2048, 512), (65, 136, 128),
          (127, 776, 1304), (128, 512, 256), (129, 24, 520), (257, 1000, 328), (300, 4096, 136), (515, 640, 1032),
          (1100, 264, 2056),
          # 32 weight rows a block, the 64-row tiles of two wavefronts, k cut over
          # blocks (forward, dx, dw), the 256-row tiles (forward, dx, dw)
          (40, 136, 2056), (64, 264, 2048), (333, 1032, 1384), (70, 16384, 128), (70, 128, 8192), (20000, 128, 64),
          (4000, 264, 2040), (3990, 4088, 264), (260, 2056, 2040),
          # dw and dx in 64-row tiles of their own launch
          (1000, 4096, 64), (1000, 4096, 136), (320, 4096, 1024),
          # dx in 64-row tiles of four and of two wavefronts with dw in 128- and
          # 256-row ones, both in 64-row tiles of one launch, the longer dw first
          (2000, 512, 1024), (333, 4096, 2048), (1000, 256, 256), (3000, 264, 136),
          # launches of their own: 128-row tiles of dx and dw, two on a CU; 64-row ones
          # of dx with 256-row ones of dw
          (2600, 2056, 1032), (100, 16384, 2048)]


def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _forward(d, x, wg, wu, with_pre=True, dtype=None):
    T, I = x.shape[0], d.inter
    out, big = R.inside(torch.zeros(T, I, dtype=x.dtype, device="cuda"), 3, 24, 77.0)
    big.fill_(77.0)
    pre = torch.full((2, T, I), float("nan"), device="cuda") if with_pre else None
    ws = R.poisoned(M.glu_workspace_size(d, T))
    M.glu(d, x, wg, wu, out, ws, pre=pre)
    torch.cuda.synchronize()
    # nothing behind the rows or the columns is written
    assert (big[T:] == 77.0).all() and (big[:, I:] == 77.0).all()
    return out, pre


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,I", SHAPES)
def test_forward(T, H, I, dtype):
    g = _gen(T * 7 + H)
    for a in ACTS:
        d = M.make_glu_desc(H, I, R.DT[dtype], a)
        x, _ = R.inside(R.gauss(g, (T, H), 1.0, dtype))
        wg, wu = (R.followed(R.gauss(g, (I, H), H ** -0.5, dtype)) for _ in range(2))
        out, pre = _forward(d, x, wg, wu)
        h, p, bound, pbound = R.glu(x, wg, wu, a, dtype)
        R.assert_close(pre, p, pbound + 1e-30, "pre")
        R.assert_close(out, h, bound, "h", 1.01 * R.half_step(dtype))
        bare, _ = _forward(d, x, wg, wu, with_pre=False)
        assert torch.equal(bare, out)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,I", SHAPES)
def test_products_of_integers_are_exact(T, H, I, dtype):
    g = _gen(T + 3 * H)
    d = M.make_glu_desc(H, I, R.DT[dtype])
    x, _ = R.inside(R.ints(g, (T, H), 4, dtype))
    wg, wu = (R.followed(R.ints(g, (I, H), 4, dtype)) for _ in range(2))
    _, pre = _forward(d, x, wg, wu)
    assert torch.equal(pre[0].double(), x.double() @ wg.double().t())
    assert torch.equal(pre[1].double(), x.double() @ wu.double().t())


def _backward(d, x, wg, wu, pre, dh, want_dx=True, want_dw=True):
    T, H, I = x.shape[0], d.hidden, d.inter
    dx, big = R.inside(torch.zeros(T, H, dtype=x.dtype, device="cuda"), 3, 24)
    big.fill_(55.0)
    dwg, dwu = (torch.full((I, H), float("nan"), dtype=x.dtype, device="cuda") for _ in range(2))
    ws = R.poisoned(M.glu_backward_workspace_size(d, T))
    M.glu_backward(d, x, wg, wu, pre, dh, ws, dx=dx if want_dx else None, dw_gate=dwg if want_dw else None,
                   dw_up=dwu if want_dw else None)
    torch.cuda.synchronize()
    assert (big[T:] == 55.0).all() and (big[:, H:] == 55.0).all()
    assert want_dx or (big == 55.0).all()
    assert want_dw or (torch.isnan(dwg).all() and torch.isnan(dwu).all())
    return dx, dwg, dwu


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,I", SHAPES)
def test_backward(T, H, I, dtype):
    g = _gen(T * 5 + I)
    for a in ACTS:
        d = M.make_glu_desc(H, I, R.DT[dtype], a)
        x, _ = R.inside(R.gauss(g, (T, H), 1.0, dtype))
        wg, wu = (R.followed(R.gauss(g, (I, H), H ** -0.5, dtype)) for _ in range(2))
        dh, _ = R.inside(R.gauss(g, (T, I), 0.5, dtype))
        _, pre = _forward(d, x, wg, wu)
        got = _backward(d, x, wg, wu, pre, dh)
        for name, y, (ref, bound) in zip(("dx", "dwg", "dwu"), got, R.glu_backward(x, wg, wu, pre, dh, a, dtype)):
            R.assert_close(y, ref, bound, name, 2 * R.half_step(dtype))
        # each alone gives the same bits
        alone = _backward(d, x, wg, wu, pre, dh, want_dw=False)
        assert torch.equal(alone[0], got[0])
        alone = _backward(d, x, wg, wu, pre, dh, want_dx=False)
        assert torch.equal(alone[1], got[1]) and torch.equal(alone[2], got[2])


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,H,I", SHAPES)
def test_gradients_of_integers_are_exact(T, H, I, dtype):
    # gate 0: act = 0, act' = 1/2; gate 32: act = 32, act' = 1 (in fp32 the
    # logistic of 32 is 1), so dg and du are small integers
    g = _gen(T + H + I)
    d = M.make_glu_desc(H, I, R.DT[dtype])
    x, _ = R.inside(R.ints(g, (T, H), 2, dtype))
    wg, wu = (R.followed(R.ints(g, (I, H), 2, dtype)) for _ in range(2))
    pre = torch.stack((32.0 * torch.randint(0, 2, (T, I), generator=g, device="cuda"),
                       R.ints(g, (T, I), 2, torch.float32)))
    dh, _ = R.inside(2 * R.ints(g, (T, I), 1, dtype, 0.5))
    dx, dwg, dwu = _backward(d, x, wg, wu, pre, dh)
    gate, up = pre.double()
    dg = dh.double() * up * torch.where(gate > 0, 1.0, 0.5)
    du = dh.double() * gate
    assert torch.equal(dx, (dg @ wg.double() + du @ wu.double()).to(dtype))
    assert torch.equal(dwg, (dg.t() @ x.double()).to(dtype))
    assert torch.equal(dwu, (du.t() @ x.double()).to(dtype))


def test_backward_of_no_tokens_zeroes_the_weights_gradients():
    d = M.make_glu_desc(264, 136, M.DT_BF16)
    x = torch.empty(0, 264, dtype=torch.bfloat16, device="cuda")
    dh = torch.empty(0, 136, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(136, 264, dtype=torch.bfloat16, device="cuda")
    dwg, dwu = torch.full_like(w, 3.0), torch.full_like(w, 4.0)
    ws = R.poisoned(M.glu_backward_workspace_size(d, 0))
    M.glu_backward(d, x, w, w, torch.empty(2, 0, 136, device="cuda"), dh, ws, dx=torch.empty_like(x), dw_gate=dwg,
                   dw_up=dwu)
    assert (dwg == 0).all() and (dwu == 0).all()
    out = torch.empty_like(dh)
    M.glu(d, x, w, w, out, R.poisoned(M.glu_workspace_size(d, 0)))


@pytest.mark.parametrize("T", [9, 400])
def test_weights_gradients_need_no_weights(T):
    g = _gen(T)
    d = M.make_glu_desc(264, 136, M.DT_BF16)
    x, dh = R.gauss(g, (T, 264), 1.0, torch.bfloat16), R.gauss(g, (T, 136), 0.5, torch.bfloat16)
    wg, wu = (R.gauss(g, (136, 264), 0.06, torch.bfloat16) for _ in range(2))
    _, pre = _forward(d, x, wg, wu)
    _, dwg, dwu = _backward(d, x, wg, wu, pre, dh, want_dx=False)
    got = _backward(d, x, None, None, pre, dh, want_dx=False)
    assert torch.equal(got[1], dwg) and torch.equal(got[2], dwu)


@pytest.mark.parametrize("a", ACTS)
def test_gradients_against_differences(a):
    # <grad, v> against the central difference of <dh, h> along v, the 64-bit
    # forward evaluated on both sides; its own error is O(eps^2)
    T, H, I, dtype = 37, 264, 200, torch.float16
    g = _gen(11)
    d = M.make_glu_desc(H, I, R.DT[dtype], a)
    x, wg, wu = R.gauss(g, (T, H), 1.0, dtype), R.gauss(g, (I, H), 0.06, dtype), R.gauss(g, (I, H), 0.06, dtype)
    dh = R.gauss(g, (T, I), 0.5, dtype)
    _, pre = _forward(d, x, wg, wu)
    grads = _backward(d, x, wg, wu, pre, dh)
    bounds = [b for _, b in R.glu_backward(x, wg, wu, pre, dh, a, dtype)]
    args = [x.double(), wg.double(), wu.double()]
    for k in range(3):
        v = torch.randn(args[k].shape, generator=g, device="cuda", dtype=torch.float64)
        e = 1e-4

        def value(s):
            p = list(args)
            p[k] = p[k] + s * e * v
            return (dh.double() * R.act(a, p[0] @ p[1].t())[0] * (p[0] @ p[2].t())).sum()

        diff = (value(1) - value(-1)) / (2 * e)
        tol = (bounds[k] * v.abs()).sum() + 1e-5 * diff.abs() + 1e-4
        assert ((grads[k].double() * v).sum() - diff).abs() <= tol


@pytest.mark.parametrize("T", [5, 70, 200])
def test_extreme_values(T):
    # a token of zeros, one of huge values (overflow to infinity in fp16), one
    # with a NaN and one with an infinity: each stays in its own row, and gates
    # far from zero give the activations' limits
    H, I, dtype = 264, 136, torch.float16
    g = _gen(T)
    d = M.make_glu_desc(H, I, M.DT_F16)
    x = R.gauss(g, (T, H), 1.0, dtype)
    x[0] = 0
    x[1] = 30000.0
    x[2, 5] = float("nan")
    x[3, 7] = float("inf")
    wg, wu = R.gauss(g, (I, H), 0.06, dtype), R.gauss(g, (I, H), 0.06, dtype)
    out, pre = _forward(d, x, wg, wu)
    assert (out[0] == 0).all()
    p = torch.stack((x[1].double() @ wg.double().t(), x[1].double() @ wu.double().t()))
    h1 = (R.act(M.ACT_SILU, p[0])[0] * p[1])
    ok = (out[1].double() - h1).abs() <= 2e-3 * h1.abs() + 1e-3
    assert (ok | (out[1].isinf() & (h1.abs() > 65000))).all()
    assert torch.isnan(out[2]).all()
    assert torch.isnan(pre[:, 3]).any() or torch.isinf(pre[:, 3]).all()
    h, _, bound, _ = R.glu(x[4:], wg, wu, M.ACT_SILU, dtype)
    R.assert_close(out[4:], h, bound, "clean rows")


@pytest.mark.parametrize("a", ACTS)
def test_slope_of_huge_gates(a):
    # gates far past where the activation is straight: slope 1 or 0, no
    # overflow of their squares; a NaN gate stays one
    H, I = 8, 16
    d = M.make_glu_desc(H, I, M.DT_BF16, a)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    gate = torch.tensor([1e4, 1e13, 1e19, 1e25, 3e38, -1e4, -1e13, -1e19, -1e25, -3e38, 20.0, -200.0, 16.0, 0.0, 90.0,
                         float("nan")], device="cuda")
    pre = torch.stack((gate, torch.ones_like(gate)))[:, None].contiguous()
    x, dout = torch.ones(1, H, **bf), torch.ones(1, I, **bf)
    dwg, dwu = torch.empty(I, H, **bf), torch.empty(I, H, **bf)
    M.glu_backward(d, x, None, None, pre, dout, R.poisoned(M.glu_backward_workspace_size(d, 1)), dw_gate=dwg, dw_up=dwu)
    slope = (gate > 0).float()
    slope[13] = 0.5
    assert torch.equal(dwg[:15].float(), slope[:15, None].expand(15, H))
    assert torch.equal(dwu[:15].float(), gate[:15].clamp(min=0).bfloat16().float()[:, None].expand(15, H))
    assert torch.isnan(dwg[15]).all() and torch.isnan(dwu[15]).all()


@pytest.mark.parametrize("T,H,I", [(1, 4096, 2048), (40, 512, 256), (300, 1032, 1384), (2100, 520, 512)])
def test_same_bits_every_time(T, H, I):
    g = _gen(1)
    dtype = torch.bfloat16
    d = M.make_glu_desc(H, I, R.DT[dtype])
    x, dh = R.gauss(g, (T, H), 1.0, dtype), R.gauss(g, (T, I), 0.5, dtype)
    wg, wu = (R.gauss(g, (I, H), H ** -0.5, dtype) for _ in range(2))
    first = None
    for _ in range(3):
        out, pre = _forward(d, x, wg, wu)
        now = (out.clone(), pre) + tuple(t.clone() for t in _backward(d, x, wg, wu, pre, dh))
        if first is not None:
            assert all(torch.equal(p, q) for p, q in zip(first, now))
        first = now


def test_workspace_of_more_tokens_serves_fewer():
    g = _gen(2)
    dtype = torch.bfloat16
    H, I = 1032, 520
    d = M.make_glu_desc(H, I, R.DT[dtype])
    wg, wu = (R.gauss(g, (I, H), H ** -0.5, dtype) for _ in range(2))
    ws = R.poisoned(M.glu_workspace_size(d, 1000))
    for T in (1000, 300, 65, 64, 17, 1):
        x = R.gauss(g, (T, H), 1.0, dtype)
        out = torch.empty(T, I, dtype=dtype, device="cuda")
        M.glu(d, x, wg, wu, out, ws)
        want, _ = _forward(d, x, wg, wu)
        assert torch.equal(out, want)


def test_columns_of_one_buffer():
    # x and the result as column ranges of one buffer
    g = _gen(3)
    dtype = torch.float16
    T, H, I = 50, 256, 128
    d = M.make_glu_desc(H, I, R.DT[dtype])
    buf = R.gauss(g, (T, H + I + 8), 1.0, dtype)
    wg, wu = (R.gauss(g, (I, H), H ** -0.5, dtype) for _ in range(2))
    want, _ = _forward(d, buf[:, :H], wg, wu)
    keep = buf.clone()
    M.glu(d, buf[:, :H], wg, wu, buf[:, H:H + I], R.poisoned(M.glu_workspace_size(d, T)))
    assert torch.equal(buf[:, H:H + I], want)
    assert torch.equal(buf[:, :H], keep[:, :H]) and torch.equal(buf[:, H + I:], keep[:, H + I:])


def test_binding_refuses():
    d = M.make_glu_desc(256, 128, M.DT_BF16)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    x, w, out = torch.zeros(4, 256, **bf), torch.zeros(128, 256, **bf), torch.zeros(4, 128, **bf)
    ws = R.poisoned(M.glu_workspace_size(d, 4))
    bad = [dict(x=x[:, :248]), dict(x=x.half()), dict(x=x.cpu()), dict(x=x.t()), dict(x=x[:1].expand(4, 256)),
           dict(w=w.t()), dict(w=w[:120]), dict(out=out[:3]), dict(out=out.float()), dict(ws=ws.cpu()), dict(ws=None),
           dict(pre=torch.zeros(2, 4, 128, **bf)), dict(pre=torch.zeros(4, 2, 128, device="cuda"))]
    for kw in bad:
        a = dict(x=x, w=w, out=out, ws=ws, pre=None)
        a.update(kw)
        with pytest.raises(ValueError):
            M.glu(d, a["x"], a["w"], w, a["out"], a["ws"], pre=a["pre"])
    class Elsewhere:   # a stream of another GPU
        device, cuda_stream = torch.device("cuda", 7), 0
    with pytest.raises(ValueError):
        M.glu(d, x, w, w, out, ws, stream=Elsewhere())
    with pytest.raises(M.MoeError) as e:
        M.glu(d, x, w, w, out, ws[:16])
    assert e.value.code == M.ERR_WORKSPACE
    pre = torch.zeros(2, 4, 128, device="cuda")
    wsb = R.poisoned(M.glu_backward_workspace_size(d, 4))
    with pytest.raises(ValueError):   # a broadcast gradient
        M.glu_backward(d, x, w, w, pre, out[:1].expand(4, 128), wsb, dx=torch.empty_like(x))
    with pytest.raises(M.MoeError) as e:
        M.glu_backward(d, x, w, w, pre, out, wsb)
    assert e.value.code == M.ERR_INVALID_ARG
