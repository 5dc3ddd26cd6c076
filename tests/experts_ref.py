"""Definitions of the operators around a MoE layer's own experts in 64 bits,
for the tests, and the error bounds their kernels are held to.  (A rounding to
fp32 is off by 2^-24 of the value; the bounds count 2^-23 for each, as the
matrix cores may truncate.)"""
from __future__ import annotations

import numpy as np
import torch

from dense_ref import FUNC, SLOPE, act, half_step, least, sum_err  # noqa: F401

STEP = 2.0 ** -23
MASK = 0xFFFFFFFF


def philox(counters, key: int):
    """Philox4x32-10 of 64-bit counters: uint32 [n][4]."""
    c = [np.asarray(counters, np.uint64) & np.uint64(MASK), np.asarray(counters, np.uint64) >> np.uint64(32)]
    c += [np.zeros_like(c[0]), np.zeros_like(c[0])]
    k = [key & MASK, key >> 32 & MASK]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k[0]), b & np.uint64(MASK),
             (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k[1]), a & np.uint64(MASK)]
        k = [(k[0] + 0x9E3779B9) & MASK, (k[1] + 0xBB67AE85) & MASK]
    return np.stack(c, -1).astype(np.uint32)


def keep(rows: int, cols: int, p: float, seed: int, offset: int):
    """Which elements dropout keeps (bool, on the GPU if there is one), and their
    factor."""
    blocks = -(-cols // 8)
    with np.errstate(over="ignore"):
        n = np.arange(rows * blocks, dtype=np.uint64) + np.uint64(offset % 2 ** 64)
    bits = philox(n, seed % 2 ** 64)
    half = np.stack((bits & 0xFFFF, bits >> 16), -1).reshape(rows, blocks * 8)[:, :cols]
    n = int(np.floor(p * 65536 + 0.5))
    return torch.from_numpy(half >= n), (65536 / (65536 - n) if n < 65536 else 0.0)


def drop(v, p, rng):
    """D(v) in 64 bits; rng: the two int64."""
    if p == 0:
        return v
    m, f = keep(v.shape[0], v.shape[1], p, *(int(i) for i in rng.tolist()))
    return torch.where(m.to(v.device), v * f, torch.zeros_like(v))


def sort(idx, E: int):
    """counts, offsets, slots in order, pos of a stable sort (int64, CPU)."""
    e = idx.cpu().numpy().reshape(-1).astype(np.int64)
    order = np.argsort(np.where((e >= 0) & (e < E), e, E), kind="stable")
    counts = np.bincount(e[(e >= 0) & (e < E)], minlength=E)
    order = order[:counts.sum()]
    pos = np.full(e.size, -1)
    pos[order] = np.arange(order.size)
    return (torch.from_numpy(v) for v in (counts, np.concatenate(([0], np.cumsum(counts))), order, pos))


def spread(x, pos, w, rows, dtype):
    """The sorted rows (64 bits), the bound, and which of them a slot names; x
    [T][H] in 64 bits already dropped out."""
    T, H = x.shape
    k = pos.numel() // T
    at = pos.flatten().long()
    ok = (at >= 0) & (at < rows)
    v = x.repeat_interleave(k, 0)[ok]
    if w is not None:
        v = v * w.double().flatten()[ok][:, None]
    out = torch.zeros(rows, H, dtype=torch.float64, device=x.device)
    out[at[ok]] = v
    named = torch.zeros(rows, dtype=torch.bool, device=x.device)
    named[at[ok]] = True
    err = 2 * STEP * out.abs()   # the factor of x, and the weight
    return out, err + half_step(dtype) * (out.abs() + err) + least(dtype), named


def slot_rows(z, pos, T):
    at = pos.flatten().long()
    ok = (at >= 0) & (at < z.shape[0])
    rows = torch.zeros(at.numel(), z.shape[1], dtype=torch.float64, device=z.device)
    rows[ok] = z.double()[at[ok]]
    return rows.view(T, -1, z.shape[1]), ok.view(T, -1)


def gather(z, pos, w, T, base, p, rng, dtype):
    """base + D(sum of the slots' rows) and the bound."""
    rows, ok = slot_rows(z, pos, T)
    k = rows.shape[1]
    f = torch.ones(T, k, dtype=torch.float64, device=z.device) if w is None else w.double().view(T, k)
    f = torch.where(ok, f, torch.zeros_like(f))[:, :, None]
    y, size = (rows * f).sum(1), (rows * f).abs().sum(1)
    y, size = drop(y, p, rng), drop(size, p, rng)
    b = torch.zeros_like(y) if base is None else base.double()
    err = (k + 3) * STEP * (size + b.abs())
    y = y + b
    return y, err + half_step(dtype) * (y.abs() + err) + least(dtype)


def products(z, pos, x):
    """<x[t], z[pos[a]]> of every slot and the bound; x in 64 bits."""
    rows, ok = slot_rows(z, pos, x.shape[0])
    v = (rows * x[:, None]).sum(2)
    return v, sum_err(x.shape[1] + 2) * (rows * x[:, None]).abs().sum(2) + 1e-30


# ---- 4-bit weights


def w4_matrix(codes, scales, zeros, e=0):
    """W_e, and s (47 + z) for each weight: what bounds the sums of x (16 + q) and
    (16 + z) x before the scale."""
    N, K = codes.shape[1], codes.shape[2] * 2
    q = torch.empty(N, K, dtype=torch.float64, device=codes.device)
    q[:, 0::2], q[:, 1::2] = codes[e] % 16, codes[e] // 16
    g = K // scales.shape[2]
    z = torch.full_like(q, 8.0) if zeros is None else zeros[e].double().repeat_interleave(g, 1)
    s = scales[e].double().repeat_interleave(g, 1)
    return s * (q - z), s.abs() * (47 + z)


def w4_product(x, codes, scales, zeros, e=0):
    """x W_e^T in 64 bits and the bound of the kernel's fp32 sums."""
    w, size = w4_matrix(codes, scales, zeros, e)
    x = x.double()
    G = scales.shape[2]
    g = w.shape[1] // G
    err = (g + 12) * STEP * (x.abs() @ size.t()) + (G + 24) * STEP * (x.abs() @ w.abs().t())
    return x @ w.t(), err


def w4(x, stacks, bounds, base, name, dtype):
    """y or h (two stacks, activation `name`) in 64 bits and the bound."""
    N = stacks[0][0].shape[1]
    y = torch.zeros(x.shape[0], N, dtype=torch.float64, device=x.device)
    err = torch.zeros_like(y)
    for e, (lo, hi) in enumerate(zip(bounds, bounds[1:])):
        if hi <= lo:
            continue
        p = [w4_product(x[lo:hi], *s, e) for s in stacks]
        if len(p) == 1:
            y[lo:hi], err[lo:hi] = p[0]
            continue
        (g, dg), (u, du) = p
        v, _ = act(name, g)
        y[lo:hi] = v * u
        err[lo:hi] = SLOPE * u.abs() * dg + (v.abs() + SLOPE * dg) * du + FUNC * (v * u).abs()
    if base is not None:
        y = y + base.double()
        err = err + STEP * y.abs()
    return y, err + half_step(dtype) * (y.abs() + err) + least(dtype)


def w4_stack(gen, E, N, K, group, dtype, zeros=True, exact=False):
    """Random codes, scales (powers of two with `exact`) and zeros."""
    codes = torch.randint(0, 256, (E, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
    if exact:
        scales = 2.0 ** torch.randint(-2, 2, (E, N, K // group), generator=gen, device="cuda").float()
    else:
        scales = (torch.rand(E, N, K // group, generator=gen, device="cuda") - 0.3) * 0.4 * K ** -0.5
    z = torch.randint(0, 16, (E, N, K // group), generator=gen, device="cuda", dtype=torch.uint8) if zeros else None
    return codes, scales.to(dtype), z
