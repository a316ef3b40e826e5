"""GPU: fp8blk_rope_append against its plain form in 64 bits."""
import math

import numpy as np
import pytest
import torch

from attention_plain import DEV, E4M3, normal, rotated, stored

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, fb, seed, N, heads, kv, pass_cols, rot, v_cols, kind="f32", e4m3=False, page=16, pages=None, interleaved=False, rot_first=True,
                 norm="none", mscale=1.0, far=0, base=10000.0, factor=1.0, spread=2.0):
        rng = np.random.default_rng(seed)
        self.fb, self.N, self.eps, self.e4m3 = fb, N, 1e-5, e4m3
        kind = torch.float32 if kind == "f32" else torch.bfloat16
        make = lambda *s: (spread * normal(rng, *s)).to(kind).to(DEV)  # noqa: E731
        cols = pass_cols + rot
        self.q, self.k = ((make(N, h, pass_cols) if pass_cols else None, make(N, h, rot)) for h in (heads, kv))
        self.v = make(N, kv, v_cols) if v_cols else None
        width = {"none": 0, "pass": pass_cols, "whole": cols}[norm]
        w = lambda: (1 + 0.3 * normal(rng, width)).bfloat16().to(DEV) if width else None  # noqa: E731
        self.q_norm, self.k_norm = w(), w()
        self.freqs = fb.fp8blk_rope_freqs(rot, base, factor).to(DEV)
        self.rope = fb.fp8blk_rope(self.freqs, interleaved, rot_first, mscale)
        self.opts = (interleaved, rot_first, mscale)
        pages = -(-N // page) + 2 if pages is None else pages
        self.slots = torch.from_numpy(rng.permutation(pages * page)[:N].astype(np.int32)).to(DEV)
        self.positions = torch.from_numpy((far + rng.integers(0, max(N, 50), N)).astype(np.int32)).to(DEV)
        store = E4M3 if e4m3 else torch.bfloat16
        self.ck = torch.full((pages, page, kv, cols), 0.25, device=DEV).to(store)
        self.cv = torch.full((pages, page, kv, v_cols), 0.25, device=DEV).to(store) if v_cols else None
        self.scales = (0.037, 0.011) if e4m3 else (1.0, 1.0)
        self.q_out = torch.full((N, heads, cols), float("nan"), dtype=torch.bfloat16, device=DEV)
        self.make_cache()

    def make_cache(self):
        self.cache = self.fb.fp8blk_cache(self.ck, self.cv, *self.scales, **({"v_cols": 16} if self.cv is None else {}))

    def args(self):
        return (self.rope, self.positions, self.q, self.q_out, self.k, self.v, self.cache, self.slots, self.q_norm, self.k_norm, self.eps)

    def run(self, **kw):
        self.fb.fp8blk_rope_append(*self.args(), **kw)
        torch.cuda.synchronize()

    def check(self, what):
        def near(got, want, bound, name):
            far = (got.double() - want).abs() > bound
            assert not far.any(), f"{what} {name}: {int(far.sum())} of {far.numel()} past the bound"
        interleaved, rot_first, mscale = self.opts
        rows = lambda parts, norm: rotated(self.positions, self.freqs, interleaved, rot_first, mscale, parts, norm, self.eps)  # noqa: E731
        near(self.q_out, *stored(*rows(self.q, self.q_norm)), "q")
        live = (self.slots >= 0) & (self.slots < self.ck.shape[0] * self.ck.shape[1])
        page, slot = self.slots[live].long() // self.ck.shape[1], self.slots[live].long() % self.ck.shape[1]
        for name, cache, (want, bound), scale in (("k", self.ck, rows(self.k, self.k_norm), self.scales[0]),
                                                  ("v", self.cv, (self.v, 0 if self.v is None else torch.zeros_like(self.v).double()), self.scales[1])):
            if cache is None:
                continue
            raw = torch.uint8 if self.e4m3 else torch.int16
            near(cache.view(raw)[page, slot].view(cache.dtype), *stored(want[live].double(), bound[live], scale if self.e4m3 else None), name)
            rest = torch.ones(cache.shape[:2], dtype=torch.bool, device=DEV)
            rest[page, slot] = False
            assert (cache.view(raw)[rest].view(cache.dtype).float() == 0.25).all(), f"{what} {name}: another slot was written"


@pytest.mark.parametrize("pass_cols,rot,v_cols", [(0, 128, 128), (64, 64, 128), (0, 64, 64), (8, 8, 16), (40, 24, 64), (0, 256, 256), (512, 64, 0),
                                                  (128, 64, 128), (768, 256, 1024), (72, 40, 48)])
@pytest.mark.parametrize("N,heads,kv", [(1, 32, 4), (3, 5, 1), (17, 8, 8), (300, 12, 2)])
def test_matches_plain(gpu, pass_cols, rot, v_cols, N, heads, kv):
    i = pass_cols // 8 + rot // 8 + N
    norm = ("none", "whole", "pass" if pass_cols else "whole")[i % 3]
    e4m3 = bool(v_cols) and i % 2 == 0
    what = f"N {N} heads {heads}/{kv} {pass_cols}+{rot} v {v_cols} norm {norm} e4m3 {e4m3}"
    print(what, flush=True)
    c = Case(gpu, i, N, heads, kv, pass_cols, rot, v_cols, ("f32", "bf16")[i // 2 % 2], e4m3, (1, 16, 64)[i % 3], None, i % 4 < 2, i % 5 < 3, norm, 1.25)
    c.run()
    c.check(what)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot_first", [False, True])
@pytest.mark.parametrize("norm", ["none", "pass", "whole"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("e4m3", [False, True])
def test_options(gpu, interleaved, rot_first, norm, kind, e4m3):
    c = Case(gpu, 5, 7, 6, 3, 96, 32, 64, kind, e4m3, 8, None, interleaved, rot_first, norm, 0.5)
    c.run()
    c.check(f"{interleaved} {rot_first} {norm} {kind} {e4m3}")


def test_far_and_negative_positions(gpu):
    """Angles of a million turns, of the largest position, of negative ones."""
    c = Case(gpu, 6, 9, 2, 1, 0, 128, 64)
    c.positions = torch.tensor([0, 1, 1 << 20, 5000001, 2 ** 31 - 1, -1, -77777, -2 ** 31, 3], dtype=torch.int32, device=DEV)
    c.run()
    c.check("positions")


def test_scaled_frequencies(gpu):
    """By parts: more than 32 turns in the original context stay, below one is divided."""
    f, g = gpu.fp8blk_rope_freqs(128, 10000.0), gpu.fp8blk_rope_freqs(128, 10000.0, 8.0, 4096, 32.0, 1.0)
    turns = 4096 * f / (2 * math.pi)
    assert torch.allclose(f, 10000.0 ** (-torch.arange(0, 128, 2, dtype=torch.float64) / 128), rtol=1e-14)
    assert torch.equal(g[turns >= 32], f[turns >= 32]) and torch.equal(g[turns <= 1], f[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 32)
    keep = (turns[mid] - 1) / 31
    assert mid.any() and torch.allclose(g[mid], f[mid] * (keep + (1 - keep) / 8), rtol=1e-14)
    c = Case(gpu, 7, 20, 4, 2, 0, 128, 128, far=30000, factor=8.0, mscale=1.2)
    c.run()
    c.check("scaled")


def test_slots_that_are_nowhere(gpu):
    """Padding and slots past the cache are not written; q is rotated all the same."""
    c = Case(gpu, 8, 12, 4, 2, 64, 64, 128, page=4, pages=6)
    c.slots[[0, 3, 7, 11]] = torch.tensor([-1, 24, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32, device=DEV)
    c.run()
    c.check("slots")


def test_only_q_and_only_the_cache(gpu):
    c = Case(gpu, 9, 5, 4, 2, 0, 64, 64)
    q_only, cache_only = torch.empty_like(c.q_out), c.ck.clone()
    gpu.fp8blk_rope_append(c.rope, c.positions, c.q, q_only, None, None, None, None)
    assert torch.equal(c.ck, cache_only)
    c.run()
    assert torch.equal(q_only, c.q_out)
    ck, cv = c.ck.clone(), c.cv.clone()
    c.ck.fill_(0.25), c.cv.fill_(0.25), c.q_out.fill_(3)
    gpu.fp8blk_rope_append(c.rope, c.positions, None, None, c.k, c.v, c.cache, c.slots)
    torch.cuda.synchronize()
    assert torch.equal(ck, c.ck) and torch.equal(cv, c.cv) and (c.q_out == 3).all()


@pytest.mark.parametrize("layout", ["heads", "shared", "wide"])
def test_cache_layouts_and_strided_inputs(gpu, layout):
    """Slices of two linears' outputs, a rotated part that heads share, pages of heads of slots, keys beside values."""
    c = Case(gpu, 10, 21, 6, 2, 64, 64, 128, page=8)
    wide_q, wide_kv = (torch.randn(21, n, device=DEV) for n in (6 * 128 + 32, 2 * 256))
    q = wide_q[:, 32:].view(21, 6, 128)
    kv = wide_kv.view(21, 2, 256)
    c.q = q[..., 64:], q[..., :64]
    c.k = kv[..., :64], kv[:, :1, 64:128].expand(21, 2, 64)
    c.v = kv[..., 128:]
    if layout == "heads":
        c.ck, c.cv = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (c.ck, c.cv))
    elif layout == "shared":
        both = torch.full((c.ck.shape[0], 2, 8, 2, 128), 0.25, dtype=torch.bfloat16, device=DEV)
        c.ck, c.cv = both[:, 0], both[:, 1]
    else:
        wide = torch.full((c.ck.shape[0], 8, 2, 256 + 16), 0.25, dtype=torch.bfloat16, device=DEV)
        c.ck, c.cv = wide[..., :128], wide[..., 144:]
    out = torch.full((6, 21, 136), 5.0, dtype=torch.bfloat16, device=DEV)
    c.q_out = out.transpose(0, 1)[..., :128]
    c.make_cache()
    c.run()
    c.check(layout)
    assert (out[..., 128:] == 5).all()


def test_values_that_are_not_finite_stay_where_they_are(gpu):
    """An infinity or NaN reaches its own pair (its own head, with a norm); e4m3 holds +-448 and NaN."""
    c = Case(gpu, 11, 4, 2, 1, 0, 64, 64, e4m3=True)
    c.k[1][1, 0, 5] = float("inf")
    c.v[2, 0, 7:10] = torch.tensor([float("inf"), float("-inf"), float("nan")], device=DEV)
    c.v[3, 0, 0] = 1e30
    c.q[1][0, 1, 3] = float("nan")
    c.run()
    q = c.q_out.float()
    assert q[0, 1, [3, 35]].isnan().all() and int(q.isnan().sum()) == 2
    flat = c.cv.view(torch.uint8).view(-1, 64)[c.slots.long()].view(E4M3).float()
    assert flat[2, 7] == 448 and flat[2, 8] == -448 and flat[2, 9].isnan() and flat[3, 0] == 448 and int(flat.isnan().sum()) == 1
    k = c.ck.view(torch.uint8).view(-1, 64)[c.slots.long()].view(E4M3).float()
    assert set((k[1].isnan() | (k[1].abs() == 448)).nonzero()[:, 0].tolist()) == {5, 37}


def test_tokens_do_not_depend_on_the_others(gpu):
    c = Case(gpu, 12, 700, 5, 2, 64, 64, 128, norm="whole", far=100000)
    c.run()
    for i in (0, 1, 333, 699):
        one = slice(i, i + 1)
        q_out, ck, cv = torch.empty_like(c.q_out[one]), c.ck.clone(), c.cv.clone()
        ck[:], cv[:] = 0.25, 0.25
        cache = gpu.fp8blk_cache(ck, cv)
        gpu.fp8blk_rope_append(c.rope, c.positions[one], tuple(t[one] for t in c.q), q_out, tuple(t[one] for t in c.k), c.v[one], cache,
                               c.slots[one], c.q_norm, c.k_norm, c.eps)
        at = int(c.slots[i])
        assert torch.equal(q_out[0], c.q_out[i])
        for a, b in ((ck, c.ck), (cv, c.cv)):
            assert torch.equal(a.view(-1, *a.shape[2:])[at], b.view(-1, *b.shape[2:])[at])


def test_a_cache_past_32_bit_offsets(gpu):
    """4.5 GB of keys: the last pages lie past 2^31 values and 2^32 bytes."""
    c = Case(gpu, 13, 6, 4, 4, 0, 128, 128, page=64, pages=2)
    pages = (2 ** 31 + 2 ** 27) // (64 * 4 * 128)
    c.ck, c.cv = (torch.full((pages, 64, 4, 128), 0.25, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    c.slots = torch.tensor([pages * 64 - 1, 0, pages * 64 - 65, 2 ** 31 // 512, 2 ** 31 // 512 - 1, 77], dtype=torch.int32, device=DEV)
    c.make_cache()
    c.run()
    c.check("far slots")


def test_captured_and_replayed(gpu):
    """New positions, slots and inputs in the same buffers, replayed between eager calls on another stream."""
    c = Case(gpu, 14, 16, 8, 2, 64, 64, 128, norm="whole", pages=9)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu.fp8blk_rope_append(*c.args())
    rng = np.random.default_rng(3)
    for step in range(4):
        c.positions.copy_(torch.from_numpy(rng.integers(0, 10 ** 6, 16).astype(np.int32)))
        c.slots.copy_(torch.from_numpy(rng.permutation(9 * 16)[:16].astype(np.int32)))
        c.q[1].copy_(normal(rng, 16, 8, 64)), c.k[0].copy_(normal(rng, 16, 2, 64))
        c.ck.fill_(0.25), c.cv.fill_(0.25), c.q_out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        c.check(f"replay {step}")
        before = [t.clone() for t in (c.q_out, c.ck, c.cv)]
        c.run(stream=side)
        assert all(torch.equal(a, b) for a, b in zip(before, (c.q_out, c.ck, c.cv)))
