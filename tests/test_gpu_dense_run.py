"""The dense operators as a program uses them together: a dense feed-forward
layer (the gated block, then the down projection with each request's adapter)
beside the MoE layer, training steps, captured graphs and streams."""
import pytest
import torch

import dense_ref as R
import trellis_quantized_moe_exl3_amd as M
import workloads as W
from gpu_util import DevLayer

pytestmark = pytest.mark.gpu


class Dense:
    """A dense feed-forward layer with adapters on its down projection."""

    def __init__(self, T, H, I, n, r, dtype, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.g, self.T, self.H, self.I, self.dtype = g, T, H, I, dtype
        self.wg, self.wu = (R.gauss(g, (I, H), H ** -0.5, dtype) for _ in range(2))
        self.wd = R.gauss(g, (H, I), I ** -0.5, dtype)
        self.a, self.b = R.gauss(g, (n, r, I), I ** -0.5, dtype), R.gauss(g, (n, H, r), 0.2, dtype)
        self.scales = torch.rand(n, generator=g, device="cuda") + 0.5
        self.ids = torch.randint(-1, n, (T,), generator=g, device="cuda").to(torch.int32)
        self.gd = M.make_glu_desc(H, I, R.DT[dtype])
        self.ld = M.make_lora_desc(I, H, n, r, R.DT[dtype])
        self.ws = [R.poisoned(M.glu_workspace_size(self.gd, T)), R.poisoned(M.lora_workspace_size(self.ld, T))]
        self.x = R.gauss(g, (T, H), 1.0, dtype)
        self.h = torch.empty(T, I, dtype=dtype, device="cuda")
        self.y = torch.empty(T, H, dtype=dtype, device="cuda")

    def run(self, stream=None, residual=None):
        M.glu(self.gd, self.x, self.wg, self.wu, self.h, self.ws[0], stream=stream)
        M.lora_linear(self.ld, self.h, self.wd, self.a, self.b, self.ids, self.y, self.ws[1], base=residual,
                      scales=self.scales, stream=stream)
        return self.y

    def check(self, residual=None):
        h, _, bound, _ = R.glu(self.x, self.wg, self.wu, M.ACT_SILU, self.dtype)
        R.assert_close(self.h, h, bound, "h")
        ref, bound = R.lora(self.h, self.wd, self.a, self.b, self.ids, residual, self.scales, None, self.dtype)
        R.assert_close(self.y, ref, bound, "y", 2 * R.half_step(self.dtype))


@pytest.mark.parametrize("T", [1, 8, 64, 200, 700])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_dense_layer_with_residual(T, dtype):
    m = Dense(T, 1024, 520, 12, 16, dtype)
    m.run(residual=m.x)
    m.check(m.x)


@pytest.mark.parametrize("T", [8, 100])
def test_beside_the_moe_layer(T):
    # the layer's output takes adapters of the layer's input: a call without a
    # projection of its own, in place on the layer's output
    cfg = W.BY_NAME["tiny"].replace(tokens=T)
    dl = DevLayer(W.gen_layer(cfg))
    x = dl.x.view(torch.float16)
    out = torch.empty_like(dl.x)
    M.layer(dl.desc, dl.weights, dl.x, out, dl.workspace(T))
    y = out.view(torch.float16)
    keep = y.clone()
    g = torch.Generator(device="cuda").manual_seed(T)
    H, n, r = cfg.hidden, 3, 8
    a, b = R.gauss(g, (n, r, H), H ** -0.5, torch.float16), R.gauss(g, (n, H, r), 0.2, torch.float16)
    ids = torch.randint(-1, n, (T,), generator=g, device="cuda").to(torch.int32)
    d = M.make_lora_desc(H, H, n, r, M.DT_F16)
    M.lora_linear(d, x, None, a, b, ids, y, R.poisoned(M.lora_workspace_size(d, T)), base=y)
    ref, bound = R.lora(x, None, a, b, ids, keep, None, None, torch.float16)
    R.assert_close(y, ref, bound, "y")
    # raw 16-bit tensors, as the layer takes them, give the same
    again = out.clone()
    again.view(torch.float16).copy_(keep)
    M.lora_linear(d, dl.x, None, a.view(torch.int16), b.view(torch.int16), ids, again,
                  R.poisoned(M.lora_workspace_size(d, T)), base=again)
    assert torch.equal(again, out)


@pytest.mark.parametrize("T", [1, 8, 64, 300])
def test_graph_replays_match_eager(T):
    m = Dense(T, 1024, 520, 12, 16, torch.bfloat16)
    dh = R.gauss(m.g, (T, m.I), 0.5, m.dtype)
    pre = torch.empty(2, T, m.I, device="cuda")
    dx, dwg, dwu = torch.empty_like(m.x), torch.empty_like(m.wg), torch.empty_like(m.wu)
    wsb = R.poisoned(M.glu_backward_workspace_size(m.gd, T))

    def step():
        m.run()
        M.glu(m.gd, m.x, m.wg, m.wu, m.h, m.ws[0], pre=pre)
        M.glu_backward(m.gd, m.x, m.wg, m.wu, pre, dh, wsb, dx=dx, dw_gate=dwg, dw_up=dwu)

    def eager():
        step()
        torch.cuda.synchronize()
        return [t.clone() for t in (m.y, dx, dwg, dwu)]

    want = eager()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    # two graphs over the same workspaces, replayed in turn
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for gr in graphs:
        with torch.cuda.graph(gr):
            step()
    torch.cuda.synchronize()
    for rep in range(3):
        for gr in graphs:
            for t in (m.y, dx, dwg, dwu, m.h, pre):
                t.fill_(3.0)
            for ws in m.ws + [wsb]:
                ws.fill_(0xFF)
            gr.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip((m.y, dx, dwg, dwu), want)), rep
        eager()
    # new contents of the same buffers
    m.x.copy_(m.x.flip(0).clone())
    m.ids.copy_(m.ids.flip(0).clone())
    graphs[0].replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (m.y, dx, dwg, dwu)]
    want = eager()
    assert all(torch.equal(p, q) for p, q in zip(got, want))


@pytest.mark.parametrize("T", [4, 90])
def test_two_streams_at_once(T):
    # two layers on two streams, each with its own workspaces
    ms = [Dense(T, 1024, 520, 6, 16, torch.bfloat16, seed=s) for s in (1, 2)]
    want = [m.run().clone() for m in ms]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ms]
    for m in ms:
        m.y.fill_(5.0)
    torch.cuda.synchronize()
    for _ in range(5):
        for m, s in zip(ms, streams):
            m.run(stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(m.y, w) for m, w in zip(ms, want))


def test_a_training_step_through_the_block():
    # loss = <c, h Wd^T>: the down projection's gradient by torch in fp32, the
    # block's by glu_backward, against 64-bit autograd of the whole
    m = Dense(150, 264, 136, 2, 8, torch.float16)
    c = R.gauss(m.g, (m.T, m.H), 0.3, m.dtype)
    pre = torch.empty(2, m.T, m.I, device="cuda")
    M.glu(m.gd, m.x, m.wg, m.wu, m.h, m.ws[0], pre=pre)
    dh = (c.float() @ m.wd.float()).to(m.dtype)
    grads = [torch.empty_like(t) for t in (m.x, m.wg, m.wu)]
    M.glu_backward(m.gd, m.x, m.wg, m.wu, pre, dh, R.poisoned(M.glu_backward_workspace_size(m.gd, m.T)), dx=grads[0],
                   dw_gate=grads[1], dw_up=grads[2])
    leaves = [t.double().requires_grad_() for t in (m.x, m.wg, m.wu)]
    gate, up = leaves[0] @ leaves[1].t(), leaves[0] @ leaves[2].t()
    ((torch.nn.functional.silu(gate) * up) @ m.wd.double().t() * c.double()).sum().backward()
    for got, leaf in zip(grads, leaves):
        rel = ((got.double() - leaf.grad).norm() / leaf.grad.norm()).item()
        # dh, then dg and du, then the output: three roundings
        assert rel <= 3 * R.half_step(m.dtype)


def test_rows_up_to_the_2_gib_limit():
    # columns of one buffer whose rows lie 2 MiB apart: byte offsets up to 2^31,
    # and past it for a tile's rows behind the last token
    T, H, I, ld = 1020, 264, 136, 1 << 20
    g = torch.Generator(device="cuda").manual_seed(3)
    dtype = torch.bfloat16
    big = torch.empty(T, ld, dtype=dtype, device="cuda")

    def far(col, cols, fill=None):
        v = big[:, col:col + cols]
        return v if fill is None else v.copy_(fill)

    x, dh, base = (R.gauss(g, (T, n), 1.0, dtype) for n in (H, I, H))
    wg, wu = (R.gauss(g, (I, H), H ** -0.5, dtype) for _ in range(2))
    d = M.make_glu_desc(H, I, M.DT_BF16)
    n = max(M.glu_workspace_size(d, T), M.glu_backward_workspace_size(d, T))
    ids = torch.randint(-1, 3, (T,), generator=g, device="cuda").to(torch.int32)
    w, a, b = R.gauss(g, (H, I), 0.1, dtype), R.gauss(g, (3, 16, I), 0.1, dtype), R.gauss(g, (3, H, 16), 0.3, dtype)
    ld_desc = M.make_lora_desc(I, H, 3, 16, M.DT_BF16)

    def run(x, h, dh, dx, base, y):
        pre = torch.empty(2, T, I, device="cuda")
        dwg, dwu = torch.empty_like(wg), torch.empty_like(wu)
        ws = R.poisoned(n)
        M.glu(d, x, wg, wu, h, ws, pre=pre)
        M.glu_backward(d, x, wg, wu, pre, dh, ws, dx=dx, dw_gate=dwg, dw_up=dwu)
        M.lora_linear(ld_desc, h, w, a, b, ids, y, R.poisoned(M.lora_workspace_size(ld_desc, T)), base=base)
        return h, dx, dwg, dwu, y

    def near(cols):
        return torch.empty(T, cols, dtype=dtype, device="cuda")

    want = run(x, near(I), dh, near(H), base, near(H))
    got = run(far(0, H, x), far(512, I), far(1024, I, dh), far(2048, H), far(ld - 512, H, base), far(4096, H))
    for a_, b_ in zip(got, want):
        assert torch.equal(a_, b_)
    with pytest.raises(M.MoeError) as e:   # one row more no longer spans less than 2 GiB
        more = torch.empty(1025, ld, dtype=dtype, device="cuda")[:, :H]
        M.glu(d, more, wg, wu, torch.empty(1025, I, dtype=dtype, device="cuda"), R.poisoned(M.glu_workspace_size(d, 1025)))
    assert e.value.code == M.ERR_UNSUPPORTED
