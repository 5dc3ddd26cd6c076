"""Definitions of the dense operators in 64 bits, for the tests, and the error
bounds their kernels are held to."""
from __future__ import annotations

import math

import torch

import trellis_quantized_moe_exl3_amd as M

DT = {torch.bfloat16: M.DT_BF16, torch.float16: M.DT_F16}
K0, C0 = math.sqrt(2.0 / math.pi), 0.044715
# |act'| and |act''| of silu stay below 1.1 and 0.5, of gelu below 1.13 and 1.13
# (its curvature is 2 phi(0) = 0.798 at 0; the tanh form stays within 0.9)
SLOPE, CURVE = 1.13, 1.13
# the kernels' exponential and reciprocal: a few fp32 steps, the argument's own
# rounding scaled by its size (|z| <= 64 where the factor is not 0 or 1)
FUNC = 2.0 ** -17


def act(name, g):
    """act(g) and act'(g) in the type of g."""
    if name == M.ACT_SILU:
        p = torch.sigmoid(g)
        return g * p, p * (1 + g * (1 - p))
    t = torch.tanh(K0 * (g + C0 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * K0 * (1 + 3 * C0 * g * g)


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def least(dtype):
    """Half of the smallest subnormal step."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def sum_err(n):
    """Bound of an fp32 sum of n terms over the sum of their magnitudes: n
    roundings (or truncations) of at most 2^-23."""
    return (n + 8) * 2.0 ** -23


def glu(x, wg, wu, a, dtype):
    """h, pre in 64 bits and the bound of |kernel - h|."""
    x, wg, wu = x.double(), wg.double(), wu.double()
    g, u = x @ wg.t(), x @ wu.t()
    v, _ = act(a, g)
    h = v * u
    e = sum_err(x.shape[1])
    dg, du = e * (x.abs() @ wg.abs().t()), e * (x.abs() @ wu.abs().t())
    err = SLOPE * u.abs() * dg + (v.abs() + SLOPE * dg) * du + FUNC * h.abs()
    return h, torch.stack((g, u)), err + half_step(dtype) * (h.abs() + err) + least(dtype), torch.stack((dg, du))


def glu_backward(x, wg, wu, pre, dh, a, dtype):
    """dx, dwg, dwu in 64 bits from the kernel's own pre, each with its bound."""
    x, wg, wu, dh = x.double(), wg.double(), wu.double(), dh.double()
    g, u = pre.double()
    v, s = act(a, g)
    dg, du = dh * u * s, dh * v
    hs, tiny = half_step(dtype), least(dtype)
    # the slope is a sum of terms up to |g| + 1 times the logistic's error
    eg = FUNC * (dh * u).abs() * (1 + g.abs()) + hs * dg.abs() + tiny
    eu = FUNC * du.abs() + hs * du.abs() + tiny
    e = sum_err(2 * wg.shape[0])
    dx = dg @ wg + du @ wu
    bx = (eg + e * dg.abs()) @ wg.abs() + (eu + e * du.abs()) @ wu.abs()
    e = sum_err(x.shape[0])
    dwg, dwu = dg.t() @ x, du.t() @ x
    bg, bu = (eg + e * dg.abs()).t() @ x.abs(), (eu + e * du.abs()).t() @ x.abs()
    return [(r, b + hs * (r.abs() + b) + tiny) for r, b in ((dx, bx), (dwg, bg), (dwu, bu))]


def lora(x, w, a, b, ids, base, scales, ranks, dtype):
    """y in 64 bits and the bound of |kernel - y|."""
    T, N = x.shape[0], b.shape[1]
    x = x.double()
    y = torch.zeros(T, N, dtype=torch.float64, device=x.device)
    err = torch.zeros_like(y)
    if w is not None:
        y += x @ w.double().t()
        err += sum_err(x.shape[1]) * (x.abs() @ w.double().abs().t())
    if base is not None:
        y += base.double()
    hs = half_step(dtype)
    for e in range(a.shape[0]):
        rows = torch.nonzero(ids == e).flatten()
        r = a.shape[1] if ranks is None else int(ranks[e])
        if rows.numel() == 0 or r == 0:
            continue
        s = 1.0 if scales is None else float(scales[e])
        ae, be = a[e, :r].double(), b[e, :, :r].double()
        u = s * (x[rows] @ ae.t())
        eu = abs(s) * sum_err(x.shape[1]) * (x[rows].abs() @ ae.abs().t())
        eu = eu + hs * (u.abs() + eu) + least(dtype)
        y[rows] += u @ be.t()
        err[rows] += (eu + sum_err(r) * u.abs()) @ be.abs().t()
    # the joining additions (projection, base, adapter) in fp32
    err = err + 4 * 2.0 ** -23 * y.abs()
    return y, err + hs * (y.abs() + err) + least(dtype)


def inside(t, rows_after=2, cols_after=16, fill=float("nan")):
    """A copy of the matrix t as the top left part of a larger one filled with
    `fill`: the view, and the whole."""
    big = torch.full((t.shape[0] + rows_after, t.shape[1] + cols_after), fill, dtype=t.dtype, device=t.device)
    big[:t.shape[0], :t.shape[1]] = t
    return big[:t.shape[0], :t.shape[1]], big


def followed(t, fill=float("nan")):
    """A contiguous copy of t with `fill` right behind it."""
    flat = torch.full((t.numel() + 4096,), fill, dtype=t.dtype, device=t.device)
    v = flat[:t.numel()].view(t.shape)
    v.copy_(t)
    return v


def ints(gen, shape, lim, dtype, density=1.0):
    """Random integers in [-lim, lim], exact in every type used here."""
    v = torch.randint(-lim, lim + 1, shape, generator=gen, device="cuda").float()
    if density < 1.0:
        v = v * (torch.rand(shape, generator=gen, device="cuda") < density)
    return v.to(dtype)


def gauss(gen, shape, std, dtype):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def poisoned(n):
    return torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")


def assert_close(got, ref, bound, what, norm=None):
    """|got - ref| within bound everywhere, and in the 2-norm within `norm`
    of the reference's."""
    got = got.double()
    assert torch.isfinite(got).all(), what
    over = (got - ref).abs() - bound
    assert (over <= 0).all(), f"{what}: {int((over > 0).sum())} outside, worst by {over.max().item():.3e}"
    if norm is not None and ref.norm() > 0:
        rel = ((got - ref).norm() / ref.norm()).item()
        assert rel <= norm, f"{what}: 2-norm {rel:.3e} over {norm:.3e}"
