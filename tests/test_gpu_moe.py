"""GPU: fp4_moe against its plain form in 64 bits."""
import numpy as np
import pytest
import torch

from block_scaled_fp8_fp8blk_amd import inputs as I
from layer_plain import Slab, U, assert_within, moe, normal

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
MX, NV = I.MXFP4, I.NVFP4


class Layer:
    def __init__(self, gpu, fmt, E, hidden, inter, seed, limit=0.0, **kw):
        rng = np.random.default_rng(seed)
        self.gate, self.up = (Slab(rng, fmt, E, inter, hidden, **kw) for _ in range(2))
        self.down = Slab(rng, fmt, E, hidden, inter, **kw)
        self.hidden, self.inter, self.limit, self.rng, self.E = hidden, inter, limit, rng, E
        self.handle = gpu.fp4_moe_weights(fmt, *self.gate.on(DEV), *self.up.on(DEV), *self.down.on(DEV), limit=limit)

    def tokens(self, M, K, base=True):
        x = normal(self.rng, M, self.hidden).bfloat16()
        ids = torch.from_numpy(np.stack([self.rng.permutation(self.E)[:K] if K <= self.E else self.rng.integers(0, self.E, K)
                                         for _ in range(M)]).astype(np.int32))
        p = torch.from_numpy(self.rng.uniform(0.05, 1.0, (M, K)).astype(np.float32))
        return x, ids, p, normal(self.rng, M, self.hidden) * 4 if base else None

    def run(self, gpu, x, ids, p, base, in_place=False):
        M, K = ids.shape
        y = torch.full((M, self.hidden), float("nan"), device=DEV)
        b = None if base is None else base.to(DEV)
        if in_place:
            y.copy_(b)
            b = y
        ws = torch.full((gpu.fp4_moe_bytes(self.inter, M, K),), 0xFF, dtype=torch.uint8, device=DEV)
        gpu.fp4_moe(self.handle, x.to(DEV), ids.to(DEV), p.to(DEV), b, y, ws)
        torch.cuda.synchronize()
        return y

    def check(self, gpu, x, ids, p, base, what):
        y = self.run(gpu, x, ids, p, base)
        assert_within(y, *moe(self.gate, self.up, self.down, x, ids, p, base, self.limit), what)
        return y


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("M,K,E,hidden,inter", [(1, 1, 1, 32, 32), (1, 2, 8, 64, 96), (1, 8, 16, 1024, 512), (2, 4, 5, 160, 1056),
                                                (3, 4, 32, 1440, 736), (5, 8, 12, 544, 256), (8, 2, 4, 256, 2080),
                                                (13, 6, 9, 416, 320), (16, 8, 24, 512, 384), (16, 16, 16, 96, 64),
                                                (16, 1, 2, 2080, 128), (16, 8, 10, 1440, 736), (12, 6, 7, 1056, 2080),
                                                (16, 5, 4, 2080, 352), (9, 4, 20, 2592, 416), (1, 1, 2, 64, 20480),
                                                (2, 1, 2, 65536, 32), (1, 2, 3, 8224, 4128), (4, 2, 2, 64, 5632),
                                                (4, 2, 2, 96, 10752), (4, 1, 1, 16384, 32)])
def test_matches_plain(gpu, fmt, M, K, E, hidden, inter):
    print("moe", fmt, M, K, E, hidden, inter, flush=True)
    L = Layer(gpu, fmt, E, hidden, inter, M * hidden + inter + fmt, limit=(0.0, 3.0)[M % 2])
    L.check(gpu, *L.tokens(M, K, base=K % 2 == 0), f"{fmt} {M}x{K} of {E}, {hidden}x{inter}")


@pytest.mark.parametrize("fmt", [MX, NV])
def test_workload_shape(gpu, fmt):
    """A decode token and a verify panel over experts of 4096 x 2048."""
    L = Layer(gpu, fmt, 10, 4096, 2048, 77)
    for M in (1, 4):
        L.check(gpu, *L.tokens(M, 8), f"{fmt} M={M}")


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("hidden,inter", [(288, 160), (1056, 1600)])
def test_ids_without_an_expert_add_nothing(gpu, fmt, hidden, inter):
    L = Layer(gpu, fmt, 6, hidden, inter, 5)
    x, ids, p, base = L.tokens(5, 4)
    ids[0] = -1
    ids[1] = torch.tensor([6, 2, -1, 100])
    ids[2] = torch.tensor([2 ** 31 - 1, -2 ** 31, 7, 8])
    p[0, 2] = float("nan")  # of a choice that is none
    y = L.check(gpu, x, ids, p, base, "ids outside")
    assert torch.equal(y[0].cpu(), base[0]) and torch.equal(y[2].cpu(), base[2])
    y = L.run(gpu, x, ids, p, None)
    assert (y[0] == 0).all() and (y[2] == 0).all()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("M,K", [(1, 16), (16, 16), (7, 5)])
@pytest.mark.parametrize("hidden,inter", [(160, 96), (1056, 544)])
def test_the_same_expert_many_times(gpu, fmt, M, K, hidden, inter):
    """Every choice the same expert (up to 256 of one), and two experts in turn."""
    L = Layer(gpu, fmt, 3, hidden, inter, 8)
    x, ids, p, base = L.tokens(M, K)
    ids[:] = 1
    L.check(gpu, x, ids, p, base, "one expert")
    ids[:, 1::2] = 2
    L.check(gpu, x, ids, p, base, "two experts")


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("hidden,inter,K", [(1056, 544, 5), (2080, 544, 4), (1056, 2080, 4), (2080, 768, 6)])
def test_tokens_do_not_depend_on_the_panel(gpu, fmt, hidden, inter, K):
    L = Layer(gpu, fmt, 7, hidden, inter, 15)
    x, ids, p, base = L.tokens(16, K)
    y = L.run(gpu, x, ids, p, base)
    for n in (1, 3, 6, 9):
        for at in (0, 16 - n):
            s = slice(at, at + n)
            assert torch.equal(L.run(gpu, x[s], ids[s], p[s], base[s]), y[s]), (n, at)
    assert torch.equal(L.run(gpu, x, ids, p, base, in_place=True), y)


@pytest.mark.parametrize("fmt,lo,hi", [(MX, 0, 6), (MX, 90, 150), (NV, 0, 9), (NV, 0x70, 0x7E)])
def test_extreme_block_scales(gpu, fmt, lo, hi):
    """Subnormal products and scales of very different sizes in one row."""
    L = Layer(gpu, fmt, 4, 192, 128, 31, scale_range=(lo, hi), with_global=False)
    x, ids, p, base = L.tokens(3, 3)
    if (fmt, lo) == (MX, 0):  # weights near 2^-124: h underflows, y is the base
        y = L.run(gpu, x, ids, p, base)
        assert torch.equal(y.cpu(), base)
        return
    if (fmt, lo) == (MX, 90):
        x *= 2.0 ** -23
    if hi == 0x7E:
        x *= 2.0 ** -10
    L.check(gpu, x, ids, p, base, f"{fmt} scales {lo}..{hi}")


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("hidden,inter", [(160, 96), (1440, 1376)])
def test_values_that_are_not_finite_stay_in_their_token(gpu, fmt, hidden, inter):
    L = Layer(gpu, fmt, 4, hidden, inter, 41)
    x, ids, p, base = L.tokens(6, 3)
    clean = L.run(gpu, x, ids, p, base)
    x[2, 9], p[4, 1] = float("nan"), float("inf")
    y = L.run(gpu, x, ids, p, base)
    ok = [0, 1, 3, 5]
    assert torch.equal(y[ok], clean[ok]) and y[2].isnan().all() and not torch.isfinite(y[4]).any()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("limit", [0.0, 2.0])
def test_a_nan_passes_the_limit(gpu, fmt, limit):
    """Also with a limit, which an infinite gate or up is brought down to, a
    NaN in x gives NaN."""
    L = Layer(gpu, fmt, 3, 96, 64, 43, limit=limit)
    x, ids, p, base = L.tokens(3, 2)
    x[1, 40] = float("nan")
    y = L.run(gpu, x, ids, p, base)
    assert y[1].isnan().all() and torch.isfinite(y[[0, 2]]).all()


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("inter", [64, 4128])
def test_an_infinite_h_gives_infinite_outputs(gpu, fmt, inter):
    """h past the largest f32: h times a weight is infinite, with its sign."""
    L = Layer(gpu, fmt, 1, 64, inter, 47, with_global=False, scale_range=(120, 120) if fmt == MX else (56, 56))
    for slab, code in ((L.gate, 0x22), (L.up, 0x22), (L.down, 0xAA)):  # 1, 1, -1
        slab.codes[:] = code
    L.handle = gpu.fp4_moe_weights(fmt, *L.gate.on(DEV), *L.up.on(DEV), *L.down.on(DEV))
    x = torch.full((2, 64), 2.0 ** 70).bfloat16()
    x[1] = 0.0
    y = L.run(gpu, x, torch.zeros((2, 1), dtype=torch.int32), torch.ones(2, 1), None)
    assert (y[0] == -float("inf")).all() and (y[1] == 0).all()


def test_large_gates(gpu):
    """silu far from 0: exp(-g) overflows to infinity and h is 0, or h is g u."""
    L = Layer(gpu, MX, 2, 96, 64, 51, scale_range=(127, 131))
    x, ids, p, base = L.tokens(4, 2)
    L.check(gpu, x, ids, p, base, "large gates")


def test_experts_past_32_bit_offsets(gpu):
    """Slabs of more than 2^32 bytes: the last of 1024 experts of 4096 x 2304."""
    E, hidden, inter = 1024, 4096, 2304
    dev = [torch.zeros((E, r, c // 2), dtype=torch.uint8, device=DEV) for r, c in ((inter, hidden), (inter, hidden), (hidden, inter))]
    sc = [torch.full((E, r, c // 32), 120, dtype=torch.uint8, device=DEV) for r, c in ((inter, hidden), (inter, hidden), (hidden, inter))]
    assert dev[0].numel() > 1 << 32
    rng = np.random.default_rng(61)
    small = [Slab(rng, MX, 2, *s) for s in ((inter, hidden), (inter, hidden), (hidden, inter))]
    at = torch.tensor([3, E - 1], device=DEV)
    for d, s, slab in zip(dev, sc, small):
        d[at], s[at] = torch.from_numpy(slab.codes).to(DEV), torch.from_numpy(slab.scales).to(DEV)
    layer = gpu.fp4_moe_weights(MX, dev[0], sc[0], None, dev[1], sc[1], None, dev[2], sc[2], None)
    x = normal(rng, 2, hidden).bfloat16()
    p = torch.tensor([[0.25, 0.75], [0.5, 0.125]])
    ids = torch.tensor([[3, E - 1], [E - 1, 500]], dtype=torch.int32)
    y = torch.empty((2, hidden), device=DEV)
    ws = torch.empty(gpu.fp4_moe_bytes(inter, 2, 2), dtype=torch.uint8, device=DEV)
    gpu.fp4_moe(layer, x.to(DEV), ids.to(DEV), p.to(DEV), None, y, ws)
    torch.cuda.synchronize()
    near = torch.tensor([[0, 1], [1, -1]])
    assert_within(y, *moe(*small, x, near, p, None, 0.0), "experts past 2^32")


@pytest.mark.parametrize("high", [253, 254])
@pytest.mark.parametrize("M,K,hidden,inter", [(3, 2, 96, 96), (1, 1, 64, 64), (5, 4, 1056, 160), (3, 5, 96, 2080), (16, 6, 2080, 544)])
def test_block_scales_past_a_rows_end_do_not_count(gpu, high, M, K, hidden, inter):
    """MXFP4 scale codes of 253 and 254 stand beside small codes only (here 0),
    and times the 6 at the end of a row before, or of their own row, they would
    be infinite. Down and the sum in one launch, and in two."""
    L = Layer(gpu, MX, 8, hidden, inter, 53)
    for slab in (L.gate, L.up, L.down):
        slab.codes[..., :16] = slab.codes[..., -32:-16] = 0x00
        slab.scales[..., 0] = slab.scales[..., -2] = high
        slab.values[..., :32] = slab.values[..., -64:-32] = 0.0
        slab.codes[..., -16:], slab.scales[..., -1], slab.values[..., -32:] = 0x77, 121, 6 * 2.0 ** -6
        codes, scales, _ = slab.on(DEV)
        ws = torch.empty(gpu.fp8blk_workspace_bytes(gpu.OP_LOAD_CHECK, 8, 64), dtype=torch.uint8, device=DEV)
        for c, s in zip(codes, scales):
            assert gpu.fp4_load_check(MX, c, s, ws)[0] == gpu.OK
    L.handle = gpu.fp4_moe_weights(MX, *L.gate.on(DEV), *L.up.on(DEV), *L.down.on(DEV))
    L.check(gpu, *L.tokens(M, K), f"scale codes {high}")


class Picking(Layer):
    """A layer whose outputs are h itself: tokens of one column each, so that
    gate and up are exact, and rows of down that hold a single 1."""

    def __init__(self, gpu, fmt, hidden, inter, seed, top=(1.0, 1.0)):
        super().__init__(gpu, fmt, 3, hidden, inter, seed, with_global=False)
        self.at = self.rng.integers(0, inter, (3, hidden))
        self.down.codes[:], self.down.scales[:] = 0, 127 if fmt == MX else 0x38
        e, r = np.ogrid[:3, :hidden]
        self.down.codes[e, r, self.at // 2] = np.where(self.at % 2, 0x20, 0x02)
        self.gate.top, self.up.top = (np.full(3, t, dtype=np.float32) for t in top)
        self.handle = gpu.fp4_moe_weights(fmt, *self.gate.on(DEV), *self.up.on(DEV), *self.down.on(DEV))

    def one_column_tokens(self, M, K, size):
        """Each token's first choice is an expert, the others are none."""
        col = torch.from_numpy(self.rng.integers(0, self.hidden, M))
        x = torch.zeros(M, self.hidden).bfloat16()
        x[torch.arange(M), col] = torch.from_numpy(self.rng.uniform(0.5, 1.0, M) * size).bfloat16()
        ids = torch.full((M, K), -1, dtype=torch.int32)
        ids[:, 0] = torch.from_numpy(self.rng.integers(0, 3, M))
        return x, ids, torch.ones(M, K), col

    def h(self, x, ids, col):
        """The h that every output picks, in 64 bits."""
        out = torch.empty(x.shape[0], self.hidden, dtype=torch.float64)
        for m, e in enumerate(ids[:, 0].tolist()):
            v = float(x[m, col[m]])
            g, u = (s.values[e][:, col[m]] * v * float(s.top[e]) for s in (self.gate, self.up))
            out[m] = (g * torch.sigmoid(g) * u)[torch.from_numpy(self.at[e])]
        return out


@pytest.mark.parametrize("fmt,size", [(MX, 4.0), (NV, 0.25)])
@pytest.mark.parametrize("top", [0, -60, -112, 110])
@pytest.mark.parametrize("K,hidden,inter", [(2, 256, 96), (5, 256, 2080), (3, 96, 512)])
def test_h_keeps_all_its_bits(gpu, fmt, size, top, K, hidden, inter):
    """h to f32 accuracy from its three bf16 pieces, across its range. exp is
    good to 2 f32 steps, 4 U, which 1 + exp passes on at most whole; that sum,
    the division and the product by u round once each: 7 U, and 12 with room.
    Two pieces would leave up to 128 U. Below 2^-110 the last piece is a
    subnormal bf16, good to 2^-134."""
    L = Picking(gpu, fmt, hidden, inter, 71 + inter, top=(1.0, 2.0 ** top))
    x, ids, p, col = L.one_column_tokens(16, K, size)
    want = L.h(x, ids, col)
    assert_within(L.run(gpu, x, ids, p, None), want, 12 * U * want.abs() + 2.0 ** -134, f"h around 2^{top}")


@pytest.mark.parametrize("fmt", [MX, NV])
def test_subnormal_weights_reach_the_output(gpu, fmt):
    """Block scales of the smallest codes, their weights subnormal in bf16 for
    MXFP4, on activations that bring gate and up back to ordinary sizes."""
    L = Layer(gpu, fmt, 4, 192, 128, 33, scale_range=(0, 6), with_global=False)
    L.down = Slab(L.rng, fmt, 4, 192, 128, with_global=False)
    L.handle = gpu.fp4_moe_weights(fmt, *L.gate.on(DEV), *L.up.on(DEV), *L.down.on(DEV))
    x, ids, p, base = L.tokens(5, 3)
    x *= 2.0 ** (120 if fmt == MX else 4)
    L.check(gpu, x, ids, p, base * 0.125, f"{fmt} scales 0..6")


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("K,hidden,inter", [(1, 64, 64), (5, 64, 2080)])
def test_an_h_past_bf16s_largest_is_a_number(gpu, fmt, K, hidden, inter):
    """(2 - 2^-10) 2^127 is an f32, and nearer to infinity than to bf16's
    largest value: h stays that number, exactly."""
    L = Picking(gpu, fmt, hidden, inter, 83, top=(2.0 ** 64, (2.0 - 2.0 ** -10) * 2.0 ** 63))
    for slab in (L.gate, L.up):  # 1, before the global scales
        slab.codes[:], slab.scales[:] = 0x22, 127 if fmt == MX else 0x38
    L.handle = gpu.fp4_moe_weights(fmt, *L.gate.on(DEV), *L.up.on(DEV), *L.down.on(DEV))
    ids = torch.full((2, K), -1, dtype=torch.int32)
    ids[:, 0] = torch.tensor([0, 2])
    x = torch.zeros(2, hidden).bfloat16()
    x[:, 7] = torch.tensor([1.0, 0.5]).bfloat16()
    y = L.run(gpu, x, ids, torch.ones(2, K), None).cpu()
    assert (y[0] == (2.0 - 2.0 ** -10) * 2.0 ** 127).all() and (y[1] == (2.0 - 2.0 ** -10) * 2.0 ** 125).all()
