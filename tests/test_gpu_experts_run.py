"""The operators around a MoE layer's own experts as a program uses them
together: a layer of 4-bit experts behind this library's router, a training
step of 16-bit experts, captured graphs and streams."""
import pytest
import torch

import dense_ref as D
import experts_ref as R
import trellis_quantized_moe_exl3_amd as M
import workloads as W
from gpu_util import DevLayer

pytestmark = pytest.mark.gpu


class Layer4:
    """Experts of 4-bit weights (gated pair, then down), top-k routed."""

    def __init__(self, T, H, I, E, k, group, dtype, seed=0):
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.E, self.k, self.dtype = T, E, k, dtype
        self.raw = [R.w4_stack(g, E, I, H, group, dtype), R.w4_stack(g, E, I, H, group, dtype, zeros=False),
                    R.w4_stack(g, E, H, I, group, dtype)]
        self.w = [M.make_w4(*r) for r in self.raw]
        dt = D.DT[dtype]
        self.td = M.make_tokens_desc(H, E, k, dt)
        self.gd, self.dd = M.make_w4_desc(H, I, E, group, dt), M.make_w4_desc(I, H, E, group, dt)
        self.x = D.gauss(g, (T, H), 1.0, dtype)
        logits = torch.randn(T, E, generator=g, device="cuda")
        top, idx = torch.topk(logits, k, dim=1)
        self.idx, self.rw = idx.to(torch.int32).contiguous(), torch.softmax(top, 1).contiguous()
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        self.pos = torch.empty(T * k, dtype=torch.int32, device="cuda")
        new = lambda n, c: torch.empty(n, c, dtype=dtype, device="cuda")
        self.xs, self.h, self.z, self.y = new(T * k, H), new(T * k, I), new(T * k, H), new(T, H)
        self.ws = [D.poisoned(M.sort_workspace_size(self.td, T)), D.poisoned(M.w4_workspace_size(self.gd, T * k)),
                   D.poisoned(M.w4_workspace_size(self.dd, T * k))]

    def experts(self, stream=None):
        M.w4_glu(self.gd, self.xs, self.w[0], self.w[1], self.h, self.ws[1], offsets=self.offsets, stream=stream)
        M.w4_linear(self.dd, self.h, self.w[2], self.z, self.ws[2], offsets=self.offsets, stream=stream)

    def run(self, stream=None, **drop):
        M.sort(self.td, self.idx, None, self.offsets, None, self.pos, self.ws[0], stream=stream)
        M.dispatch(self.td, self.x, self.pos, self.xs, stream=stream)
        self.experts(stream)
        M.combine(self.td, self.z, self.pos, self.y, w=self.rw, base=self.x, stream=stream, **drop)
        return self.y

    def check(self, p=0.0, rng=None):
        """Each step against its definition on the kernels' own inputs."""
        _, offsets, order, pos = R.sort(self.idx, self.E)
        assert torch.equal(self.offsets.cpu().long(), offsets) and torch.equal(self.pos.cpu().long(), pos)
        assert torch.equal(self.xs, self.x[(order // self.k).cuda()])
        bounds = offsets.tolist()
        ref, bound = R.w4(self.xs, self.raw[:2], bounds, None, M.ACT_SILU, self.dtype)
        D.assert_close(self.h, ref, bound, "h")
        ref, bound = R.w4(self.h, self.raw[2:], bounds, None, None, self.dtype)
        D.assert_close(self.z, ref, bound, "z")
        ref, bound = R.gather(self.z, self.pos, self.rw, self.T, self.x, p, rng, self.dtype)
        D.assert_close(self.y, ref, bound, "y")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,I,E,k,group", [(1, 512, 256, 8, 2, 64), (8, 1024, 512, 40, 8, 128), (200, 512, 384, 12, 4, 32),
                                             (1500, 256, 512, 6, 3, 128)])
def test_layer_of_4_bit_experts(T, H, I, E, k, group, dtype):
    m = Layer4(T, H, I, E, k, group, dtype)
    m.run()
    m.check()
    rng = torch.tensor([3, 1 << 33], dtype=torch.int64, device="cuda")
    m.run(p=0.2, rng=rng)
    m.check(0.2, rng)


@pytest.mark.parametrize("T", [1, 8, 300])
def test_behind_the_librarys_router(T):
    # moe_exl3_route's own tables feed dispatch, the 4-bit experts and combine,
    # and sort() gives the same tables from its indexes
    cfg = W.BY_NAME["tiny"].replace(tokens=T)
    dl = DevLayer(W.gen_layer(cfg))
    E, k = cfg.n_experts, cfg.top_k
    m = Layer4(T, cfg.hidden, 128, E, k, 64, torch.float16)
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, counts, ids = torch.empty(T * k, **i32), torch.empty(E, **i32), torch.empty(T * k, **i32)
    M.route(dl.desc, dl.weights, dl.x, idx, m.rw, counts, m.offsets, ids, m.pos, dl.workspace(T))
    tables = [torch.empty_like(t) for t in (counts, m.offsets, ids, m.pos)]
    M.sort(m.td, idx.view(T, k), *tables, m.ws[0])
    for got, want in zip(tables, (counts, m.offsets, ids, m.pos)):
        assert torch.equal(got, want)
    m.x, m.idx = dl.x.view(torch.float16), idx.view(T, k)
    M.dispatch(m.td, m.x, m.pos, m.xs)
    m.experts()
    M.combine(m.td, m.z, m.pos, m.y, w=m.rw, base=m.x)
    m.check()


class Training:
    """Experts of one gated block each, trained: rows [T k][H] -> [T k][I]."""

    def __init__(self, T, H, I, E, k, dtype, p, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.H, self.I, self.E, self.k, self.dtype, self.p = T, H, I, E, k, dtype, p
        self.idx = torch.argsort(torch.rand(T, E, generator=g, device="cuda"), dim=1)[:, :k].to(torch.int32).contiguous()
        self.idx[0, 0] = -1
        self.rw = torch.rand(T, k, generator=g, device="cuda")
        self.x, self.base, self.dy = (D.gauss(g, (T, n), 1.0, dtype) for n in (H, I, I))
        self.wg, self.wu = (D.gauss(g, (E, I, H), H ** -0.5, dtype) for _ in range(2))
        self.rng = torch.tensor([seed + 1, 77], dtype=torch.int64, device="cuda")
        dt = D.DT[dtype]
        self.hd, self.id = M.make_tokens_desc(H, E, k, dt), M.make_tokens_desc(I, E, k, dt)
        self.gd = M.make_glu_desc(H, I, dt)
        n = T * k
        new = lambda r, c: torch.zeros(r, c, dtype=dtype, device="cuda")
        self.xs, self.z, self.y = new(n, H), new(n, I), new(T, I)
        self.dz, self.dxs, self.dx = new(n, I), new(n, H), new(T, H)
        self.dwg, self.dwu, self.dw = torch.zeros_like(self.wg), torch.zeros_like(self.wu), torch.empty(T, k, device="cuda")
        self.offsets = torch.empty(E + 1, dtype=torch.int32, device="cuda")
        self.pos = torch.empty(n, dtype=torch.int32, device="cuda")
        self.pre = [torch.empty(0, device="cuda")] * E
        self.ws = D.poisoned(max(M.glu_workspace_size(self.gd, n), M.glu_backward_workspace_size(self.gd, n),
                                 M.sort_workspace_size(self.hd, T)))
        M.sort(self.hd, self.idx, None, self.offsets, None, self.pos, self.ws)
        self.bounds = self.offsets.tolist()
        self.pre = [torch.empty(2, b - a, I, device="cuda") for a, b in zip(self.bounds, self.bounds[1:])]

    def step(self):
        M.sort(self.hd, self.idx, None, self.offsets, None, self.pos, self.ws)
        M.dispatch(self.hd, self.x, self.pos, self.xs)
        each = list(zip(range(self.E), self.bounds, self.bounds[1:]))
        for e, a, b in each:
            M.glu(self.gd, self.xs[a:b], self.wg[e], self.wu[e], self.z[a:b], self.ws, pre=self.pre[e])
        M.combine(self.id, self.z, self.pos, self.y, w=self.rw, base=self.base, p=self.p, rng=self.rng)
        M.combine_backward(self.id, self.dy, self.z, self.pos, self.dz, w=self.rw, dw=self.dw, p=self.p, rng=self.rng)
        for e, a, b in each:
            M.glu_backward(self.gd, self.xs[a:b], self.wg[e], self.wu[e], self.pre[e], self.dz[a:b], self.ws,
                           dx=self.dxs[a:b], dw_gate=self.dwg[e], dw_up=self.dwu[e])
        M.dispatch_backward(self.hd, self.dxs, None, self.pos, self.dx)
        return self.y, self.dx, self.dw, self.dwg, self.dwu

    def autograd(self):
        """The same step in 64 bits, gradients by autograd on the CPU."""
        leaf = lambda t: t.double().cpu().requires_grad_(True)
        x, rw, wg, wu = (leaf(t) for t in (self.x, self.rw, self.wg, self.wu))
        kept, f = R.keep(self.T, self.I, self.p, *self.rng.tolist())
        slots = []
        for t in range(self.T):
            total = torch.zeros(self.I, dtype=torch.float64)
            for j, e in enumerate(self.idx[t].tolist()):
                if e >= 0:
                    g = wg[e] @ x[t]
                    total = total + rw[t, j] * (g * torch.sigmoid(g) * (wu[e] @ x[t]))
            slots.append(total)
        y = self.base.double().cpu() + torch.stack(slots) * kept * f
        y.backward(self.dy.double().cpu())
        return [t.detach() for t in (y, x.grad, rw.grad, wg.grad, wu.grad)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T,H,I,E,k,p", [(1, 264, 136, 3, 2, 0.25), (40, 264, 136, 5, 3, 0.1), (64, 520, 72, 4, 4, 0.0)])
def test_training_step(T, H, I, E, k, p, dtype):
    m = Training(T, H, I, E, k, dtype, p)
    got = m.step()
    # in the 2-norm each of the roundings on a path (y: h and y; dx: dz, the pair
    # dg and du, dxs, dx; the weights': dz, dg or du, the result) costs half a step
    # of its value at most, four on the longest; twice that for what the steps
    # between do to it
    ref = dict(zip(("y", "dx", "dw", "dwg", "dwu"), m.autograd()))
    for v, what in zip(got, ref):
        off = (v.double().cpu() - ref[what]).norm()
        if what != "dw":
            assert off <= 8 * R.half_step(dtype) * ref[what].norm(), (what, off)
    # dw = sum of D(dy) z, each z off by half a step of it: half a step of the
    # sum of magnitudes, however far the sum itself cancels (one token's has one
    # number: 5% off in bf16 at 136 terms); twice that for the sums in fp32
    dy = R.drop(m.dy.double(), p, m.rng)
    terms = (R.slot_rows(m.z, m.pos, T)[0] * dy[:, None]).abs().sum(2).cpu()
    assert ((m.dw.double().cpu() - ref["dw"]).abs() <= 2 * R.half_step(dtype) * terms).all()


@pytest.mark.parametrize("kind", ["layer", "training"])
def test_graph_replays_match_eager(kind):
    if kind == "layer":
        m = Layer4(24, 512, 256, 10, 4, 64, torch.bfloat16)
        rng = torch.tensor([1, 0], dtype=torch.int64, device="cuda")
        step, outs = (lambda: m.run(p=0.3, rng=rng)), (m.y,)
    else:
        m = Training(40, 264, 136, 5, 3, torch.bfloat16, 0.3)
        rng = m.rng
        step, outs = m.step, (m.y, m.dx, m.dw, m.dwg, m.dwu)

    def eager():
        step()
        torch.cuda.synchronize()
        return [t.clone() for t in outs]

    def new_inputs(i):
        rng.copy_(torch.tensor([1, 1000 * i], device="cuda"))
        m.x.copy_(D.gauss(torch.Generator(device="cuda").manual_seed(i), tuple(m.x.shape), 1.0, m.dtype))

    eager()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    # two graphs over the same workspaces, replayed in turn with other numbers
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for gr in graphs:
        with torch.cuda.graph(gr):
            step()
    for i in range(6):
        new_inputs(i)
        want = eager()
        for t in outs:
            t.zero_()
        graphs[i % 2].replay()
        torch.cuda.synchronize()
        for got, ref in zip(outs, want):
            assert torch.equal(got, ref), i
        eager()


def test_on_another_stream():
    m = Layer4(100, 512, 256, 10, 4, 64, torch.float16)
    want = m.run().clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for t in (m.xs, m.h, m.z, m.y):
        t.zero_()
    s.wait_stream(torch.cuda.current_stream())
    m.run(stream=s)
    s.synchronize()
    assert torch.equal(m.y, want)
    x = torch.ones(33, 40, device="cuda")
    y, rng = torch.zeros_like(x), torch.tensor([1, 2], dtype=torch.int64, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    M.dropout(x, y, 0.5, rng, stream=s)
    s.synchronize()
    assert torch.equal(y.double(), R.drop(x.double(), 0.5, rng))


def test_two_calls_at_once():
    # two streams, each call with its own workspace
    ms = [Layer4(150, 512, 256, 10, 4, 64, torch.float16, seed=i) for i in range(2)]
    want = [m.run().clone() for m in ms]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ms]
    for _ in range(5):
        for m, s in zip(ms, streams):
            m.run(stream=s)
    torch.cuda.synchronize()
    for m, w in zip(ms, want):
        assert torch.equal(m.y, w)


def test_binding_refuses_other_tensors():
    m = Layer4(10, 256, 128, 4, 2, 64, torch.float16)
    m.run()
    bad = [lambda: M.dispatch(m.td, m.x.float(), m.pos, m.xs), lambda: M.dispatch(m.td, m.x, m.pos.long(), m.xs),
           lambda: M.dispatch(m.td, m.x, m.pos[:-1], m.xs), lambda: M.dispatch(m.td, m.x, m.pos, m.xs[:, :-8]),
           lambda: M.dispatch(m.td, m.x, m.pos, m.xs, w=m.rw.half()), lambda: M.dispatch(m.td, m.x, m.pos.cpu(), m.xs),
           lambda: M.dispatch(m.td, m.x.t(), m.pos, m.xs), lambda: M.combine(m.td, m.z, m.pos, m.y, p=0.5),
           lambda: M.combine(m.td, m.z, m.pos, m.y, p=0.5, rng=torch.zeros(2, device="cuda")),
           lambda: M.combine(m.td, m.z, m.pos, m.y, p=0.5, rng=torch.zeros(2, dtype=torch.int64)),
           lambda: M.combine(m.td, m.z, m.pos, m.y, base=m.x[:-1]),
           lambda: M.sort(m.td, m.idx, None, m.offsets[:-1], None, m.pos, m.ws[0]),
           lambda: M.sort(m.td, m.idx.t(), None, m.offsets, None, m.pos, m.ws[0]),
           lambda: M.sort(m.td, m.idx, None, m.offsets, None, m.pos, None),
           lambda: M.dropout(m.x, m.y.float(), 0.5, torch.zeros(2, dtype=torch.int64, device="cuda")),
           lambda: M.dropout(m.x, m.y, 0.5, None), lambda: M.dropout(m.idx, m.idx, 0.5, None),
           lambda: M.w4_linear(m.dd, m.h, m.w[2], m.z, m.ws[2]),
           lambda: M.w4_linear(m.dd, m.h, m.w[0], m.z, m.ws[2], offsets=m.offsets),
           lambda: M.w4_linear(m.dd, m.h, m.w[2], m.z, m.ws[2], offsets=m.offsets[1:]),
           lambda: M.w4_linear(m.dd, m.h.bfloat16(), m.w[2], m.z, m.ws[2], offsets=m.offsets),
           lambda: M.w4_glu(m.gd, m.xs, m.w[0], m.w[2], m.h, m.ws[1], offsets=m.offsets)]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} went through")
    with pytest.raises(M.MoeError) as e:
        M.w4_linear(m.dd, m.h, m.w[2], m.z, m.ws[2][:128], offsets=m.offsets)
    assert e.value.code == M.ERR_WORKSPACE
