"""Plain 64-bit forms of the norms, router, expert layer and 4-bit linear, on
the CPU, and how far f32 arithmetic may be from them.

Bounds count roundings: U = 2^-24 is half an f32 step, a sum of n terms taken
in any order is off by at most (n - 1) U times the sum of the terms' sizes to
first order, and the kernels' sums are trees over lanes of short runs, so the
depths used below are far above what they take. H = 2^-8 is half a bf16 step."""
import numpy as np
import torch

import oracle
from block_scaled_fp8_fp8blk_amd import inputs as I

U, H = 2.0 ** -24, 2.0 ** -8


def normal(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32))


def block_norm(resid, y, post_w, gate, scale, pre_w, eps):
    """(r', its bound, x, its bound), in 64 bits; r' before its rounding to resid's type, x before bf16.

    A statistic of at most 65536 squares in runs of at most 64 and a tree of
    10 levels is off by 80 U; 1/sqrt halves that, and the divisions, products
    and the fused multiply-add add fewer than 20: 64 U of each term."""
    r = resid.double()
    term = torch.zeros_like(r)
    if y is not None:
        n = y.double()
        if post_w is not None:
            n = n / (n.square().mean(1, keepdim=True) + eps).sqrt() * post_w.double()
        if gate is not None:
            n = n * gate.double()
        term = scale * n
    out = r + term
    dr = 64 * U * (term.abs() + out.abs())
    if pre_w is None:
        return out, dr, None, None
    inv = 1 / (out.square().mean(1, keepdim=True) + eps).sqrt()
    x = out * inv * pre_w.double()
    return out, dr, x, dr * inv * pre_w.double().abs() + 64 * U * x.abs()


def scores(x, w, score):
    l = x.double() @ w.double().t()
    if score == 0:
        return torch.softmax(l, 1)
    return torch.sigmoid(l) if score == 1 else (l.clamp(min=0) + torch.log1p(torch.exp(-l.abs()))).sqrt()


def route(x, w, bias, score, top_k, normalize, scale):
    """(ids, weights in 64 bits, the smallest gap between neighbours in the order that decides)."""
    s = scores(x, w, score)
    choice = s if bias is None else s + bias.double()
    choice = torch.where(choice.isnan(), torch.full_like(choice, -np.inf), choice)
    order = choice.sort(dim=1, descending=True, stable=True)
    ids = order.indices[:, :top_k].clone()
    left = order.values[:, :top_k] > -np.inf
    p = torch.where(left, s.gather(1, ids), 0.0)
    ids[~left] = -1
    if normalize:
        total = p.sum(1, keepdim=True)
        p = torch.where(total > 0, p / total, 0.0)
    v = order.values[:, :top_k + 1]
    gap = (v[:, :-1] - v[:, 1:]).abs()
    gap = gap[torch.isfinite(gap)]
    return ids, scale * p, gap.min().item() if gap.numel() else np.inf


class Slab:
    """Random stacked FP4 weights: codes, scales, global scales, and their values in 64 bits."""

    def __init__(self, rng, fmt, experts, rows, cols, scale_range=None, with_global=True):
        lo, hi = scale_range or ((120, 124) if fmt == I.MXFP4 else I.FP4_SCALE_RANGE[fmt])
        B = I.FP4_BLOCK[fmt]
        self.codes = rng.integers(0, 256, (experts, rows, cols // 2), dtype=np.uint8)
        self.scales = rng.integers(lo, hi + 1, (experts, rows, cols // B), dtype=np.uint8)
        self.top = None
        self.values = torch.stack([torch.from_numpy(oracle.fp4_dequant_bf16(fmt, c, s).view(np.int16)).view(torch.bfloat16)
                                   for c, s in zip(self.codes, self.scales)]).double()
        if fmt == I.NVFP4 and with_global:
            self.top = rng.uniform(0.5, 1.5, experts).astype(np.float32) / 64
            self.values = self.values * torch.from_numpy(self.top).double()[:, None, None]

    def on(self, dev):
        return [None if a is None else torch.from_numpy(a).to(dev) for a in (self.codes, self.scales, self.top)]


def moe(gate, up, down, x, ids, weights, base, limit):
    """(y, its bound) in 64 bits. With W = sum |w v| for a sum of n products,
    g and u are off by (n + 48) U W; silu has a slope of at most 1.1, and its
    own evaluation and the product by u add 16 U |h|; the sum for y is off by
    (inter + 48 + K) U of its terms."""
    M, K = ids.shape
    hidden, inter = down.values.shape[1:]
    y = torch.zeros(M, hidden, dtype=torch.float64) if base is None else base.double()
    bound = (K + 4) * U * y.abs()
    for m in range(M):
        v = x[m].double()
        for k in range(K):
            e = int(ids[m, k])
            if not 0 <= e < gate.values.shape[0]:
                continue
            g, u, d = gate.values[e] @ v, up.values[e] @ v, down.values[e]
            dg, du = ((hidden + 48) * U * (w.values[e].abs() @ v.abs()) for w in (gate, up))
            if limit > 0:
                g, u = g.clamp(max=limit), u.clamp(-limit, limit)
            s = g * torch.sigmoid(g)
            h = s * u
            dh = 1.1 * dg * (u.abs() + du) + s.abs() * du + 16 * U * h.abs()
            p = float(weights[m, k])
            y[m] += p * (d @ h)
            bound[m] += abs(p) * (d.abs() @ dh + (inter + 48 + K) * U * (d.abs() @ h.abs()))
    return y, bound


def int4(codes, scales, zeros, group, x):
    """(y, its bound) in 64 bits: sums over the codes and over x times the zero
    point, at most cols / 32 + group + 32 roundings of sum |s x| (q + z)."""
    q = torch.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1).double()
    cols = q.shape[1]
    z = torch.full_like(q, 8.0) if zeros is None else zeros.double().repeat_interleave(group, 1)
    s = scales.double().repeat_interleave(group, 1)
    v = x.double()
    return v @ ((q - z) * s).t(), (cols // 32 + group + 32) * U * (v.abs() @ ((q + z) * s.abs()).t())


def assert_within(got, want, bound, what):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    off = (got - want).abs()
    bad = off > bound
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} values out of bounds; worst "
                           f"{float((off / bound.clamp(min=1e-300)).max()):.3g} times the bound")
