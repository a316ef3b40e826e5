"""GPU: the norms, router, expert layer and 4-bit linear run together as a
decode or verify step runs them, eager, on another stream, and captured in a
HIP graph."""
import gc
import weakref

import numpy as np
import pytest
import torch

from block_scaled_fp8_fp8blk_amd import inputs as I
from layer_plain import H, Slab, U, assert_within, block_norm, int4, moe, normal, route

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EPS = 1e-6


class Step:
    """One block: norm, router, experts with a 4-bit shared linear as their
    base, and the norms that lead to the next block."""

    def __init__(self, gpu, M, fmt=I.NVFP4, E=20, K=4, hidden=1056, inter=352, seed=1):
        rng = np.random.default_rng(seed)
        self.gpu, self.M, self.K, self.fmt = gpu, M, K, fmt
        self.slabs = [Slab(rng, fmt, E, *s) for s in ((inter, hidden), (inter, hidden), (hidden, inter))]
        self.resid = normal(rng, M, hidden)
        self.w1, self.w2, self.w3 = ((1 + 0.1 * normal(rng, hidden)).bfloat16() for _ in range(3))
        self.gate = normal(rng, 1, hidden).bfloat16()
        self.router = (normal(rng, E, hidden) / 16).bfloat16()
        self.bias = 0.1 * normal(rng, E)
        self.codes = torch.from_numpy(rng.integers(0, 256, (hidden, hidden // 2), dtype=np.uint8))
        self.scales = (normal(rng, hidden, hidden // 32) * 0.01).bfloat16()
        d = self.d = {k: v.to(DEV) for k, v in vars(self).items() if isinstance(v, torch.Tensor)}
        top = [s.on(DEV) for s in self.slabs]
        self.layer = gpu.fp4_moe_weights(fmt, *top[0], *top[1], *top[2], limit=7.0)
        d["x"] = torch.empty(M, hidden, dtype=torch.bfloat16, device=DEV)
        d["ids"] = torch.empty(M, K, dtype=torch.int32, device=DEV)
        d["p"] = torch.empty(M, K, device=DEV)
        d["y"] = torch.empty(M, hidden, device=DEV)
        d["out"] = torch.empty(M, hidden, device=DEV)
        d["next"] = torch.empty(M, hidden, dtype=torch.bfloat16, device=DEV)
        self.ws1 = torch.empty(gpu.fp8blk_workspace_bytes(gpu.OP_MOE_ROUTE, E, hidden, M), dtype=torch.uint8, device=DEV)
        self.ws2 = torch.empty(gpu.fp4_moe_bytes(inter, M, K), dtype=torch.uint8, device=DEV)

    def run(self, stream=None):
        g, d = self.gpu, self.d
        g.fp8blk_block_norm(d["resid"], None, None, None, 0.0, None, d["w1"], EPS, d["x"], stream=stream)
        g.fp8blk_moe_route(d["router"], d["bias"], d["x"], g.SCORE_SIGMOID, True, 1.5, d["ids"], d["p"], self.ws1, stream=stream)
        g.int4_gemv(d["codes"], d["scales"], None, 32, d["x"], d["y"], stream=stream)
        g.fp4_moe(self.layer, d["x"], d["ids"], d["p"], d["y"], d["y"], self.ws2, stream=stream)
        g.fp8blk_block_norm(d["resid"], d["y"], d["w2"], d["gate"], 0.5, d["out"], d["w3"], EPS, d["next"], stream=stream)

    def outputs(self):
        return [self.d[k].clone() for k in ("x", "ids", "p", "y", "out", "next")]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("fmt", [I.MXFP4, I.NVFP4])
@pytest.mark.parametrize("M", [1, 6, 16])
def test_step_matches_plain(gpu, fmt, M):
    s = Step(gpu, M, fmt, seed=M)
    s.run()
    x, ids, p, y, out, nxt = (t.cpu() for t in s.outputs())
    _, _, x64, dx = block_norm(s.resid, None, None, None, 0.0, s.w1, EPS)
    assert_within(x, x64, dx + H * (x64.abs() + dx), "x")
    ids64, p64, gap = route(x, s.router, s.bias, 1, s.K, True, 1.5)  # each stage on the x before it as it was rounded
    assert gap > 1e-11 and torch.equal(ids.long(), ids64)
    assert_within(p, p64, (U + 1e-12) * p64, "weights")
    base, db = int4(s.codes, s.scales, None, 32, x)
    y64, dy = moe(*s.slabs, x, ids, p, base, 7.0)
    assert_within(y, y64, dy + 2 * db, "y")
    r64, dr, n64, dn = block_norm(s.resid, y, s.w2, s.gate, 0.5, s.w3, EPS)
    assert_within(out, r64, dr, "resid")
    assert_within(nxt, n64, dn + H * (n64.abs() + dn), "next")


@pytest.mark.parametrize("M", [1, 5, 16])
def test_step_on_another_stream(gpu, M):
    s = Step(gpu, M, seed=30 + M)
    s.run()
    torch.cuda.synchronize()
    want = s.outputs()
    side = torch.cuda.Stream()
    for k in ("x", "y", "out", "next"):
        s.d[k].fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    s.run(stream=side)  # named
    side.synchronize()
    assert _same(s.outputs(), want)
    for k in ("x", "y", "out", "next"):
        s.d[k].fill_(float("nan"))
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # current
        s.run()
    side.synchronize()
    assert _same(s.outputs(), want)


@pytest.mark.parametrize("M", [1, 16])
def test_two_steps_at_once(gpu, M):
    """Two steps with buffers of their own on two streams, in turn with eager work."""
    a, b = Step(gpu, M, seed=50), Step(gpu, M, I.MXFP4, seed=51)
    a.run(), b.run()
    torch.cuda.synchronize()
    wa, wb = a.outputs(), b.outputs()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        a.run(stream=sa)
        b.run(stream=sb)
    torch.cuda.synchronize()
    assert _same(a.outputs(), wa) and _same(b.outputs(), wb)


@pytest.mark.parametrize("M", [1, 7, 16])
def test_captured_step(gpu, M):
    """Captured once and replayed with new inputs, eager runs and
    synchronizations between the replays; two graphs share the workspaces."""
    s = Step(gpu, M, seed=70 + M)
    s.run()
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        cap = torch.cuda.Stream()
        with torch.cuda.graph(g, stream=cap):
            s.run()
        graphs.append(g)
    rng = np.random.default_rng(99)
    for rep in range(4):
        s.d["resid"].copy_(normal(rng, *s.resid.shape).to(DEV) * (1 + rep))
        s.run()
        torch.cuda.synchronize()
        want = s.outputs()
        for g in graphs:
            for k in ("x", "y", "out", "next", "p"):
                s.d[k].fill_(float("nan"))
            s.d["ids"].fill_(-5)
            g.replay()
            torch.cuda.synchronize()
            assert _same(s.outputs(), want), (rep, M)


def test_prepared_calls(gpu):
    s = Step(gpu, 3, seed=90)
    s.run()
    torch.cuda.synchronize()
    want, d = s.outputs(), s.d
    calls = [gpu.prepared("fp8blk_block_norm", d["resid"], None, None, None, 0.0, None, d["w1"], EPS, d["x"]),
             gpu.prepared("fp8blk_moe_route", d["router"], d["bias"], d["x"], gpu.SCORE_SIGMOID, True, 1.5, d["ids"], d["p"], s.ws1),
             gpu.prepared("int4_gemv", d["codes"], d["scales"], None, 32, d["x"], d["y"]),
             gpu.prepared("fp4_moe", s.layer, d["x"], d["ids"], d["p"], d["y"], d["y"], s.ws2),
             gpu.prepared("fp8blk_block_norm", d["resid"], d["y"], d["w2"], d["gate"], 0.5, d["out"], d["w3"], EPS, d["next"])]
    for k in ("x", "y", "out", "next"):
        d[k].fill_(float("nan"))
    assert [c() for c in calls] == [gpu.OK] * 5
    torch.cuda.synchronize()
    assert _same(s.outputs(), want)


def test_prepared_calls_keep_their_tensors(gpu):
    """A prepared call is the only owner of what it was given."""
    s = Step(gpu, 3, seed=91)
    s.run()
    torch.cuda.synchronize()
    want, d = s.outputs(), s.d
    outs = {k: torch.full_like(d[k], -5 if k == "ids" else float("nan")) for k in ("x", "ids", "p", "y", "out", "next")}
    mine = lambda t: None if t is None else t.clone()
    layer = lambda: gpu.fp4_moe_weights(s.fmt, *[mine(t) for t in s.layer.keep], limit=7.0)
    args = [("fp8blk_block_norm", d["resid"].clone(), None, None, None, 0.0, None, d["w1"].clone(), EPS, outs["x"]),
            ("fp8blk_moe_route", d["router"].clone(), d["bias"].clone(), outs["x"], gpu.SCORE_SIGMOID, True, 1.5, outs["ids"],
             outs["p"], s.ws1.clone()),
            ("int4_gemv", d["codes"].clone(), d["scales"].clone(), None, 32, outs["x"], outs["y"]),
            ("fp4_moe", layer(), outs["x"], outs["ids"], outs["p"], outs["y"], outs["y"], s.ws2.clone()),
            ("fp8blk_block_norm", d["resid"].clone(), outs["y"], d["w2"].clone(), d["gate"].clone(), 0.5, outs["out"],
             d["w3"].clone(), EPS, outs["next"])]
    owned = [t for a in args for t in a if isinstance(t, torch.Tensor)] + [t for t in args[3][1].keep if t is not None]
    refs = [weakref.ref(t) for t in owned]
    calls = [gpu.prepared(*a) for a in args]
    del args, owned
    gc.collect()
    assert all(r() is not None for r in refs)
    assert [c() for c in calls] == [gpu.OK] * 5
    torch.cuda.synchronize()
    assert _same([outs[k] for k in ("x", "ids", "p", "y", "out", "next")], want)


def test_prepared_linears_keep_their_tensors(gpu):
    """The same of a linear and of a group's list of members."""
    codes = torch.full((32, 128), 0x38, dtype=torch.uint8, device=DEV)  # 1
    grid, x = torch.ones(1, 1, device=DEV), torch.ones(1, 128, dtype=torch.bfloat16, device=DEV)
    y = [torch.zeros(1, 32, device=DEV) for _ in range(2)]
    members = [(codes.clone(), grid.clone(), y[1])]
    one = [codes.clone(), grid.clone(), x.clone(), y[0]]
    refs = [weakref.ref(t) for t in one + list(members[0])]
    calls = [gpu.prepared("fp8blk_gemv", *one), gpu.prepared("fp8blk_gemv_grouped", members, x.clone())]
    members.clear()
    one.clear()
    gc.collect()
    assert all(r() is not None for r in refs)
    assert [c() for c in calls] == [gpu.OK] * 2
    torch.cuda.synchronize()
    assert (y[0] == 128).all() and (y[1] == 128).all()


def _offset(t, bytes_off):
    """A copy of t that lies that many bytes behind an aligned address."""
    n = t.element_size()
    room = torch.empty(t.numel() + bytes_off // n, dtype=t.dtype, device=DEV)
    room[bytes_off // n:].copy_(t.reshape(-1))
    return room[bytes_off // n:].view(t.shape)


@pytest.mark.parametrize("fmt", [I.MXFP4, I.NVFP4])
@pytest.mark.parametrize("M,hidden,inter", [(1, 1056, 352), (6, 1056, 352), (6, 160, 2080)])
def test_smallest_alignments(gpu, fmt, M, hidden, inter):
    """Every buffer that need not be 16-byte aligned, at its smallest alignment."""
    s = Step(gpu, M, fmt, K=5, hidden=hidden, inter=inter, seed=97)
    s.run()
    torch.cuda.synchronize()
    want, d = s.outputs(), s.d
    keep = list(s.layer.keep)
    for i in (1, 4, 7):  # block scales
        keep[i] = _offset(keep[i], 4 if fmt == I.MXFP4 else 8)
    for i in (2, 5, 8):  # global scales
        keep[i] = keep[i] if keep[i] is None else _offset(keep[i], 4)
    s.layer = gpu.fp4_moe_weights(fmt, *keep, limit=7.0)
    for k in ("bias", "ids", "p"):
        d[k] = _offset(d[k], 4)
    d["scales"] = _offset(d["scales"], 2)
    for k in ("x", "p", "y", "out", "next"):
        d[k].fill_(float("nan"))
    s.run()
    torch.cuda.synchronize()
    assert _same(s.outputs(), want)


@pytest.mark.parametrize("M,rows,cols,group", [(1, 45, 2080, 32), (5, 9001, 2080, 32), (3, 9001, 1088, 64), (16, 20001, 384, 128)])
def test_smallest_alignments_of_a_4_bit_linear(gpu, M, rows, cols, group):
    rng = np.random.default_rng(rows)
    codes = torch.from_numpy(rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8)).to(DEV)
    scales = (normal(rng, rows, cols // group) * 0.01).bfloat16().to(DEV)
    zeros = torch.from_numpy(rng.integers(0, 16, (rows, cols // group), dtype=np.uint8)).to(DEV)
    x = normal(rng, M, cols).bfloat16().to(DEV)
    y, z = torch.empty(M, rows, device=DEV), _offset(torch.full((M, rows), float("nan"), device=DEV), 4)
    gpu.int4_gemv(codes, scales, zeros, group, x, y)
    gpu.int4_gemv(codes, _offset(scales, 2), _offset(zeros, 1), group, x, z)
    torch.cuda.synchronize()
    assert torch.equal(y, z)
