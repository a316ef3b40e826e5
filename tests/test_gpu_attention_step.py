"""GPU: positions, cache, attention and the linears around them run together as a
layer runs them: a prompt in chunks, single tokens, a verify panel."""
import math

import numpy as np
import pytest
import torch

from attention_plain import DEV, attend, normal, rotated
from layer_plain import H

pytestmark = pytest.mark.gpu


class Layer:
    """q and kv linears, positions and cache, attention, the o linear's input."""

    def __init__(self, gpu, latent, seqs=2, room=400, page=16, seed=0):
        rng = np.random.default_rng(seed)
        self.gpu, self.latent, self.room, self.page, self.seqs = gpu, latent, room, page, seqs
        self.heads, self.kv, self.pass_cols, self.rot = (8, 1, 512, 64) if latent else (8, 2, 64, 64)
        self.k = self.pass_cols + self.rot
        self.v = 512 if latent else 128
        pages = seqs * room // page
        self.table = torch.from_numpy(rng.permutation(pages).astype(np.int32).reshape(seqs, -1)).to(DEV)
        self.ck = torch.zeros(pages, page, self.kv, self.k, dtype=torch.bfloat16, device=DEV)
        self.cv = None if latent else torch.zeros(pages, page, self.kv, self.v, dtype=torch.bfloat16, device=DEV)
        self.cache = gpu.fp8blk_cache(self.ck, self.cv, **({"v_cols": 512} if latent else {}))
        self.freqs = gpu.fp8blk_rope_freqs(self.rot).to(DEV)
        self.rope = gpu.fp8blk_rope(self.freqs, latent, not latent)
        self.norm = (1 + 0.1 * normal(rng, 512 if latent else 128)).bfloat16().to(DEV)
        self.scale = 1 / math.sqrt(self.k)
        self.len = [0] * seqs
        self.ws = torch.empty(max(1, max(gpu.fp8blk_attn_bytes(self.cache, self.heads, seqs, n, room) for n in (1, 16, room))), dtype=torch.uint8, device=DEV)

    def step(self, new, q, kv):
        """Rows of q [N, heads, k] and kv [N, kv heads, k (+ v)] in f32, new[s] of each sequence."""
        seq = [s for s, n in enumerate(new) for _ in range(n)]
        at = [self.len[s] + i for s, n in enumerate(new) for i in range(n)]
        table = self.table.cpu().numpy()
        slots = [int(table[s, p // self.page]) * self.page + p % self.page for s, p in zip(seq, at)]
        ints = lambda v: torch.tensor(v, dtype=torch.int32, device=DEV)  # noqa: E731
        P, R = self.pass_cols, self.rot
        cut = (lambda t: (t[..., :P], t[..., P:P + R])) if self.latent else (lambda t: (t[..., R:R + P], t[..., :R]))
        q_rot = torch.empty(len(at), self.heads, self.k, dtype=torch.bfloat16, device=DEV)
        self.gpu.fp8blk_rope_append(self.rope, ints(at), cut(q), q_rot, cut(kv), None if self.latent else kv[..., self.k:], self.cache, ints(slots),
                                    k_norm=self.norm)
        self.len = [a + b for a, b in zip(self.len, new)]
        out = torch.empty(len(at), self.heads, self.v, dtype=torch.bfloat16, device=DEV)
        call = self.gpu.fp8blk_latent_attn if self.latent else self.gpu.fp8blk_paged_attn
        call(self.cache, q_rot, self.table, ints(self.len), ints([sum(new[:s]) for s in range(self.seqs + 1)]), max(new), self.room, self.scale, out, self.ws)
        return out

    def inputs(self, rng, n):
        return (normal(rng, n, self.heads, self.k).to(DEV), normal(rng, n, self.kv, self.k + (0 if self.latent else self.v)).to(DEV))


@pytest.mark.parametrize("latent", [False, True])
def test_prompt_tokens_and_panels_against_the_whole(gpu, latent):
    """Chunks of 100 and 37 tokens, then single tokens, then a panel of 5: each row against attention over all tokens before it in 64 bits, with
    only the bf16 roundings of q, k and v on the way."""
    rng = np.random.default_rng(1)
    layer = Layer(gpu, latent)
    plan = [[100, 37], [63, 80], [1, 1], [1, 1], [5, 5], [0, 1], [1, 0]]
    qs, kvs, outs = ([[] for _ in range(2)] for _ in range(3))
    for new in plan:
        q, kv = layer.inputs(rng, sum(new))
        out = layer.step(new, q, kv)
        at = 0
        for s, n in enumerate(new):
            for whole, part in ((qs, q), (kvs, kv), (outs, out)):
                whole[s].append(part[at:at + n])
            at += n
    torch.cuda.synchronize()
    P, R = layer.pass_cols, layer.rot
    for s in range(2):
        q, kv, out = (torch.cat(t[s]) for t in (qs, kvs, outs))
        p = torch.arange(q.shape[0], device=DEV)
        cut = (lambda t: (t[..., :P], t[..., P:P + R])) if latent else (lambda t: (t[..., R:R + P], t[..., :R]))
        q64, _ = rotated(p, layer.freqs, latent, not latent, 1.0, cut(q))
        k64, _ = rotated(p, layer.freqs, latent, not latent, 1.0, cut(kv), layer.norm)
        v64 = k64[..., :512] if latent else kv[..., layer.k:].double()
        want, bound = attend(k64, v64, q64, 0, layer.scale)
        # q, k and v each rounded to bf16: z off by 2 H of the sum of its products' sizes (and a little for the second order), weights by twice that
        size = torch.stack([layer.scale * (q64[:, h].abs() @ k64[:, h * layer.kv // layer.heads].abs().t()).amax(1) for h in range(layer.heads)], 1)
        weights = ((bound / H).amax(-1, keepdim=True) + want.abs().amax(-1, keepdim=True))  # at least the sum of the weighted sizes
        off = bound + weights * (torch.expm1(2 * 2.05 * H * size)[..., None] + H) + H * want.abs()
        assert ((out.double() - want).abs() <= off).all()
        # what the bound above allows grows with the scores; on average rows are far nearer: three roundings of independent values
        rel = float((out.double() - want).norm() / want.norm())
        assert rel < 3 * H, rel


@pytest.mark.parametrize("latent", [False, True])
def test_a_panel_equals_single_steps(gpu, latent):
    """Five drafted tokens at once, and one after another: the same bits in the cache and in the outputs."""
    rng = np.random.default_rng(2)
    a, b = Layer(gpu, latent), Layer(gpu, latent)
    q, kv = a.inputs(rng, 200)
    for layer in (a, b):
        layer.step([150, 50], q, kv)
    q, kv = a.inputs(rng, 10)
    panel = a.step([5, 5], q, kv)
    for i in range(5):
        out = b.step([1, 1], q[[i, 5 + i]], kv[[i, 5 + i]])
        assert torch.equal(out[0], panel[i]) and torch.equal(out[1], panel[5 + i]), i
    assert torch.equal(a.ck, b.ck) and (latent or torch.equal(a.cv, b.cv))


def test_between_the_linears(gpu):
    """The kv and q linears' f32 outputs as they are, and the o linear on the attention's bf16 output, captured and replayed."""
    rng = np.random.default_rng(3)
    M, hidden, heads, kv = 4, 256, 8, 2
    weights = {n: (normal(rng, r, c) / math.sqrt(c)).bfloat16().to(DEV) for n, r, c in
               (("q", heads * 128, hidden), ("kv", kv * 256, hidden), ("o", hidden, heads * 128))}
    x = normal(rng, M, hidden).bfloat16().to(DEV)
    y_q, y_kv = torch.empty(M, heads * 128, device=DEV), torch.empty(M, kv * 256, device=DEV)
    q, kv_rows = y_q.view(M, heads, 128), y_kv.view(M, 2, kv, 128)
    ck, cv = (torch.zeros(40, 16, kv, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    cache = gpu.fp8blk_cache(ck, cv)
    table = torch.arange(40, dtype=torch.int32, device=DEV).view(M, 10)
    freqs = gpu.fp8blk_rope_freqs(128).to(DEV)
    rope = gpu.fp8blk_rope(freqs)
    q_rot, out = (torch.empty(M, heads, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    y_o = torch.empty(M, hidden, device=DEV)
    positions, slots, lens = (torch.zeros(M, dtype=torch.int32, device=DEV) for _ in range(3))
    starts = torch.arange(M + 1, dtype=torch.int32, device=DEV)
    ws = torch.empty(max(1, gpu.fp8blk_attn_bytes(cache, heads, M, 1, 160)), dtype=torch.uint8, device=DEV)

    def step():
        gpu.bf16_gemv_twin_grouped([(weights["q"], y_q), (weights["kv"], y_kv)], x)
        gpu.fp8blk_rope_append(rope, positions, (None, q), q_rot, (None, kv_rows[:, 0]), kv_rows[:, 1], cache, slots)
        gpu.fp8blk_paged_attn(cache, q_rot, table, lens, starts, 1, 160, 1 / math.sqrt(128), out, ws)
        gpu.bf16_gemv_twin(weights["o"], out.view(M, heads * 128), y_o)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    ks, vs = [], []
    for t in range(12):
        positions.fill_(t), lens.fill_(t + 1)
        slots.copy_(torch.arange(M, dtype=torch.int32) * 160 + t)
        x.copy_(normal(rng, M, hidden).bfloat16())
        graph.replay()
        torch.cuda.synchronize()
        replayed = y_o.clone()
        step()
        torch.cuda.synchronize()
        assert torch.equal(replayed, y_o), t
        p = torch.full((M,), t, device=DEV)
        q64 = (x.double() @ weights["q"].double().t()).view(M, heads, 128)
        kv64 = (x.double() @ weights["kv"].double().t()).view(M, 2, kv, 128)
        q64, k64 = (rotated(p, freqs, False, True, 1.0, (None, r))[0] for r in (q64, kv64[:, 0]))
        ks.append(k64), vs.append(kv64[:, 1])
        for m in range(M):
            want, _ = attend(torch.stack([k[m] for k in ks]), torch.stack([v[m] for v in vs]), q64[m:m + 1], t, 1 / math.sqrt(128))
            y = want.reshape(-1) @ weights["o"].double().t()
            # q, k, v, the weights and the attention's output are each rounded to bf16, the sums of 1024 products to f32
            assert float((y_o[m].double() - y).norm() / y.norm()) < 6 * H, (t, m)
