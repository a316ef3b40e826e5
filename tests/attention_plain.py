"""Plain 64-bit forms of rotary positions, paged caches and attention, and how
far f32 arithmetic may be from them.

Bounds count roundings, as in layer_plain: U = 2^-24 is half an f32 step, H =
2^-8 half a bf16 step, and half an e4m3 step is 2^-4 of a normal value and 2^-10
of a subnormal one."""
import math

import numpy as np
import torch

from layer_plain import H, U

DEV = "cuda:0"
E4M3 = torch.float8_e4m3fn


def normal(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32))


# --- rotary positions ---------------------------------------------------------------

def rotated(positions, freqs, interleaved, rot_first, mscale, parts, norm=None, eps=1e-6):
    """([N, heads, cols] in 64 bits, its bound before the last rounding).

    A norm's sum of n squares, its root, two divisions and two products: (n / 2 +
    8) U of x. Cosine and sine: half an f32 step, the series' rest of 2^-29, and
    the 64-bit angle's own rounding and reduction, 2^-51 of it (one step for the
    product, as the reference has too, one in the multiple of pi/2 taken off).
    Then two products and a sum, 2 U each."""
    first, rot = parts
    rot = rot.double()
    first = rot[..., :0] if first is None else first.double()
    dr, df = torch.zeros_like(rot), torch.zeros_like(first)
    if norm is not None:
        w, R = norm.double(), rot.shape[-1]
        whole = norm.numel() != first.shape[-1]
        over = torch.cat((first, rot), -1) if whole else first
        rms = (over.square().mean(-1, keepdim=True) + eps).sqrt()
        loss = (over.shape[-1] / 2 + 8) * U
        wf = (w[R:] if rot_first else w[:w.numel() - R]) if whole else w
        first = first / rms * wf
        df = loss * first.abs()
        if whole:
            rot = rot / rms * (w[:R] if rot_first else w[w.numel() - R:])
            dr = loss * rot.abs()
    angle = positions.double()[:, None, None] * freqs.double()
    c, s = mscale * angle.cos(), mscale * angle.sin()
    turn = (U + 2.0 ** -29 + angle.abs() * 2.0 ** -51) * abs(mscale) + 4 * U * abs(mscale)
    if interleaved:
        a, b, da, db = rot[..., 0::2], rot[..., 1::2], dr[..., 0::2], dr[..., 1::2]
    else:
        (a, b), (da, db) = rot.chunk(2, -1), dr.chunk(2, -1)
    x, y = a * c - b * s, a * s + b * c
    off = (a.abs() + b.abs()) * turn + (da + db) * abs(mscale)
    if interleaved:
        rot, dr = torch.stack((x, y), -1).flatten(-2), torch.stack((off, off), -1).flatten(-2)
    else:
        rot, dr = torch.cat((x, y), -1), torch.cat((off, off), -1)
    order = (lambda f, r: torch.cat((r, f), -1)) if rot_first else (lambda f, r: torch.cat((f, r), -1))
    return order(first, rot), order(df, dr)


def stored(value, bound, scale=None):
    """A row as the cache holds it, and its bound: bf16, or e4m3 of value / scale."""
    if scale is None:
        return value, bound + H * (value.abs() + bound) + 2.0 ** -134
    v, d = (value / scale).clamp(-448, 448), bound / scale + 2 * U * (value / scale).abs()
    return v, d + 2.0 ** -4 * (v.abs() + d) + 2.0 ** -10


# --- paged caches ---------------------------------------------------------------------

class Paged:
    """Sequences of `lens` tokens in pages in any order. What no sequence holds, and
    the rest of each last page, is NaN; table entries past a sequence are nonsense."""

    def __init__(self, fb, rng, lens, heads, k, v, page=16, e4m3=False, layout="slots", spare=2, wild=True):
        self.fb, self.lens, self.page, self.k_cols, self.v_cols, self.e4m3 = fb, lens, page, k, v, e4m3
        need = [-(-n // page) for n in lens]
        pages = sum(need) + spare
        order = rng.permutation(pages).astype(np.int32)
        width = max(max(need), 1) + 1
        table = rng.choice(np.array([-1, pages, 2 ** 31 - 1, -2 ** 31], dtype=np.int64), (len(lens), width)).astype(np.int32) \
            if wild else np.zeros((len(lens), width), dtype=np.int32)
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = order[at:at + n]
            at += n
        self.table = torch.from_numpy(table).to(DEV)
        self.k_scale, self.v_scale = (0.021, 0.017) if e4m3 else (1.0, 1.0)
        latent = v is None
        total = sum(lens)
        kind = E4M3 if e4m3 else torch.bfloat16
        self.keys = (normal(rng, total, heads, k) / self.k_scale).to(kind).to(DEV)
        self.values = None if latent else (normal(rng, total, heads, v) / self.v_scale).to(kind).to(DEV)
        self.cache_k = self._buffer(pages, page, heads, k, kind, layout)
        self.cache_v = None if latent else self._buffer(pages, page, heads, v, kind, layout)
        if layout == "shared" and not latent and k == v:
            both = torch.full((pages, 2, page, heads, k), float("nan"), dtype=torch.float32).to(kind).to(DEV)
            self.cache_k, self.cache_v = both[:, 0], both[:, 1]
        self.fill()
        self.cache = fb.fp8blk_cache(self.cache_k, self.cache_v, self.k_scale, self.v_scale, **({"v_cols": 512} if latent else {}))

    @staticmethod
    def _buffer(pages, page, heads, cols, kind, layout):
        shape = (pages, heads, page, cols) if layout == "heads" else (pages, page, heads, cols + (32 if layout == "wide" else 0))
        t = torch.full(shape, float("nan"), dtype=torch.float32).to(kind).to(DEV)
        return t.transpose(1, 2) if layout == "heads" else t[..., :cols]

    def where(self, s, n):
        """Pages and slots of a sequence's first n tokens."""
        j = torch.arange(n, device=DEV)
        return self.table[s].long()[j // self.page], j % self.page

    def fill(self):
        at = 0
        for s, n in enumerate(self.lens):
            p, i = self.where(s, n)
            for cache, rows in ((self.cache_k, self.keys), (self.cache_v, self.values)):
                if cache is not None:
                    raw = torch.uint8 if self.e4m3 else torch.int16
                    cache.view(raw)[p, i] = rows[at:at + n].view(raw)
            at += n

    def rows(self, s):
        """A sequence's keys and values as the cache holds them, in 64 bits."""
        n = min(self.lens[s], self.table.shape[1] * self.page)
        p, i = self.where(s, n)
        raw = torch.uint8 if self.e4m3 else torch.int16
        get = lambda c: c.view(raw)[p, i].view(c.dtype).double()  # noqa: E731
        k = get(self.cache_k) * self.k_scale
        return k, k[..., :512] if self.cache_v is None else get(self.cache_v) * self.v_scale


def attend(k, v, q, at, scale, causal=True, window=0, sinks=None, absent=None):
    """(out, bound, before the rounding to bf16) of one sequence, in 64 bits: keys k
    [L, h, Dk], values v [L, h, Dv], q [rows, H, Dk], row i at position at + i;
    absent: keys that no page holds. A row of values reaches a row of the output only
    where that sees it.

    z is a sum of Dk products in f32, times a scale: (Dk + 8) U of the sum of their
    sizes; the difference to the maximum, in units of log 2, loses 2 U of both;
    weights are within exp(2 dz) of theirs beside their sum; rounded to bf16 above and
    below, w (1 + e) with e up to H, they move the quotient by sum w e (v - out) and H of
    that: 1.01 H (size + |out|); and the sums over L keys, with every rescaling on the
    way, lose at most (L + 64) steps."""
    L, h, Dk = k.shape
    rows, heads, _ = q.shape
    q = q.double()
    j = torch.arange(L, device=k.device)
    p = at + torch.arange(rows, device=k.device)[:, None]
    seen = torch.ones(rows, L, dtype=torch.bool, device=k.device)
    if causal:
        seen &= j <= p
    if window:
        seen &= j > p - window
    if absent is not None:
        seen &= ~absent
    out = torch.zeros(rows, heads, v.shape[-1], dtype=torch.float64, device=k.device)
    bound = torch.zeros_like(out)
    clean = lambda t: torch.where(t.isfinite(), t, 0.0)  # noqa: E731
    for head in range(heads):
        kk, vv, qq = k[:, head * h // heads], v[:, head * h // heads], q[:, head]
        z = torch.where(seen, scale * (qq @ kk.t()), -math.inf) if kk.isfinite().all() else \
            torch.where(seen, scale * (qq[:, None] * kk[None]).sum(-1), -math.inf)
        size = abs(scale) * (clean(qq).abs() @ clean(kk).abs().t())
        dz = torch.where(seen, (Dk + 8) * U * size + 8 * U * clean(z).abs(), 0.0).amax(1, keepdim=True) if L else z.new_zeros(rows, 1)
        top = z.amax(1, keepdim=True) if L else z.new_full((rows, 1), -math.inf)
        top = torch.where(top == -math.inf, 0.0, top)
        e = torch.where(seen, torch.exp(z - top), 0.0)
        total = e.sum(1, keepdim=True)
        none = total == 0
        if sinks is not None:
            total = total + torch.exp(sinks[head].double() - top)
        w = torch.where(none, 0.0, e / torch.where(none, 1.0, total))
        o = w @ clean(vv)
        odd = ~vv.isfinite()
        for key in odd.any(1).nonzero()[:, 0].tolist():  # w * inf and w * NaN where it is seen
            o = o + torch.where(seen[:, key, None] & odd[key], w[:, key, None] * vv[key], 0.0)
        size = w @ clean(vv).abs()
        out[:, head] = o
        bound[:, head] = size * (2.02 * dz + (L + 64) * 2 * U) + 1.01 * H * (size + clean(o).abs()) + 2.0 ** -130
    return out, bound


def assert_attends(out, want, bound, what):
    """out (bf16) within the bound and its own rounding; NaN and infinities where the definition has them."""
    if not out.numel():
        return
    got = out.double()
    fine = want.isfinite()
    assert torch.equal(fine, got.isfinite()), f"{what}: {int((fine != got.isfinite()).sum())} values finite on one side only"
    far = (got - want).abs() - bound - H * (want.abs() + bound) - 2.0 ** -134
    far = torch.where(fine, far, -1.0)
    worst = float((torch.where(fine, (got - want).abs(), 0.0) / (bound + H * want.abs() + 1e-30)).max())
    assert not (far > 0).any(), f"{what}: {int((far > 0).sum())} of {far.numel()} past the bound, worst {worst:.2f} of it"


class Call:
    """One attention call over a Paged cache, and its definition."""

    def __init__(self, fb, rng, paged, new, heads, causal=True, window=0, sinks=False, behind=0, scale=None, spread=1.5, before=0):
        self.fb, self.paged, self.new, self.heads, self.causal, self.window = fb, paged, new, heads, causal, window
        self.scale = 1 / math.sqrt(paged.k_cols) if scale is None else scale
        starts = [before]
        for n in new:
            starts.append(starts[-1] + n)
        self.first = starts
        self.N = starts[-1] + behind
        self.q = (spread * normal(rng, max(self.N, 1), heads, paged.k_cols)).bfloat16().to(DEV)
        self.sinks = normal(rng, heads).to(DEV) if sinks else None
        self.starts = torch.tensor(starts, dtype=torch.int32, device=DEV)
        self.lens = torch.tensor(paged.lens, dtype=torch.int32, device=DEV)
        self.v_cols = 512 if paged.values is None else paged.v_cols
        self.out = torch.full((self.q.shape[0], heads, self.v_cols), 7.0, dtype=torch.bfloat16, device=DEV)
        self.max_new, self.max_len = max(max(new), 1), max(max(paged.lens), 1)
        self.entry = fb.fp8blk_latent_attn if paged.values is None else fb.fp8blk_paged_attn

    def workspace(self):
        n = self.fb.fp8blk_attn_bytes(self.paged.cache, self.heads, len(self.new), self.max_new, self.max_len, self.window)
        return torch.full((n,), 255, dtype=torch.uint8, device=DEV)  # NaN, whatever reads it

    def args(self, ws, q=None, out=None):
        return (self.paged.cache, self.q if q is None else q, self.paged.table, self.lens, self.starts, self.max_new, self.max_len,
                self.scale, self.out if out is None else out, ws, self.causal, self.window, self.sinks)

    def run(self, **kw):
        self.entry(*self.args(self.workspace()), **kw)
        torch.cuda.synchronize()
        return self.out

    def check(self, what, out=None):
        out = self.out if out is None else out
        for s, n in enumerate(self.new):
            if not n:
                continue
            k, v = self.paged.rows(s)
            lo = self.first[s]
            want, bound = attend(k, v, self.q[lo:lo + n], self.paged.lens[s] - n, self.scale, self.causal, self.window, self.sinks)
            assert_attends(out[lo:lo + n], want, bound, f"{what}, sequence {s} of {len(self.new)}: {n} new of {self.paged.lens[s]}")
        for rows in (out[:self.first[0]], out[self.first[-1]:self.N]):
            assert (rows == 7).all(), f"{what}: rows outside of all sequences were written"
