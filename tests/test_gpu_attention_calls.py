"""GPU: calls of rotary positions, append and attention that a server makes beside the
plain ones: shared pages, sizes on the host that are not those on the device, inputs
that every head shares, prepared calls, several at a time; and what the binding refuses."""
import numpy as np
import pytest
import torch

from attention_plain import DEV, E4M3, Call, Paged, assert_attends, attend, normal

pytestmark = pytest.mark.gpu

WIDTHS = [(64, 64), (128, 128), (192, 128), (256, 256), (512, None), (576, None)]  # None: a latent cache
IDS = ["64", "128", "192+128", "256", "latent512", "latent576"]


def _call(gpu, seed, lens, new, k, v, group=4, page=16, kv=2, **kw):
    rng = np.random.default_rng(seed)
    kv = 1 if v is None else kv
    return Call(gpu, rng, Paged(gpu, rng, lens, kv, k, v, page), new, kv * group, **kw)


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("T", [1, 9, 70])
def test_pages_in_common(gpu, k, v, T):
    """Two sequences of one prefix, and one whose table names a page twice."""
    c = _call(gpu, 30, [300, 310, 100], [T, T, T], k, v)
    table = c.paged.table
    table[1, :16] = table[0, :16]
    table[2, 3] = table[2, 1]
    c.run()
    c.check(f"{k} {T}")


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("T,most", [(5, 3), (40, 7), (90, 41), (260, 129)])
def test_more_new_tokens_than_max_new(gpu, k, v, T, most):
    """The first max_new tokens of a sequence get their rows, the others keep what they held."""
    c = _call(gpu, 31, [900, 300], [T, most - 1], k, v)
    c.max_new = most
    c.run()
    for s, lo, n in ((0, 0, most), (1, T, most - 1)):
        kk, vv = c.paged.rows(s)
        want, bound = attend(kk, vv, c.q[lo:lo + n], c.paged.lens[s] - c.new[s], c.scale)
        assert_attends(c.out[lo:lo + n], want, bound, f"{k} {T} {most} sequence {s}")
    assert (c.out[most:T] == 7).all()


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("T", [1, 50])
@pytest.mark.parametrize("window", [0, 300])
def test_longer_than_max_len(gpu, k, v, T, window):
    c = _call(gpu, 32, [5000, 40], [T, 1], k, v, window=window)
    for most in (1, 900, 2 ** 30 - 1 if T > 1 else 10 ** 6):
        c.max_len = most
        c.out.fill_(7.0)
        c.run()
        c.check(f"{k} {T} {window} max_len {most}")


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("T", [1, 7, 100])
def test_values_that_are_all_alike(gpu, k, v, T):
    """Their mean is that value, whatever the weights: these are rounded alike above and
    below, and sums of 3000 f32 lose less than 2 * 3064 * 2^-24 < 2^-11, which does not move a
    bf16 value by half a step (2^-9)."""
    c = _call(gpu, 38, [3000, 70], [T, 1], k, v, group=3, spread=4.0)
    cache = c.paged.cache_k if v is None else c.paged.cache_v
    row = torch.linspace(-3, 3, c.v_cols).bfloat16().to(DEV)
    cache[..., :c.v_cols] = row
    c.run()
    assert torch.equal(c.out, row.expand_as(c.out))


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("T", [1, 30])
def test_heads_that_share_a_row_of_q(gpu, k, v, T):
    """A head stride of 0, and q and out as slices of wider buffers."""
    c = _call(gpu, 33, [400], [T], k, v, group=5)
    one = c.q[:, :1].clone()
    c.q = one.expand(-1, c.heads, -1)
    wide = torch.full((T, c.heads, c.v_cols + 24), 7.0, dtype=torch.bfloat16, device=DEV)
    c.out = wide[..., 16:16 + c.v_cols]
    c.run()
    c.check(f"{k} {T}")
    assert (wide[..., :16] == 7).all() and (wide[..., 16 + c.v_cols:] == 7).all()


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("S", [1, 3, 8, 13])
def test_splits_of_unequal_sequences(gpu, k, v, S):
    """Chunks and single tokens whose keys are split, most sequences far shorter than the longest."""
    lens = [5300 if s == S // 2 else 37 * s + 66 for s in range(S)]
    for T in (1, 66):
        c = _call(gpu, 34, lens, [T] * S, k, v, group=2, page=64)
        c.run()
        c.check(f"{k} {S} {T}")


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
def test_calls_at_the_same_time(gpu, k, v):
    """Two streams, a workspace each, over one cache: as one after the other."""
    c = _call(gpu, 35, [5000, 700], [3, 1], k, v, page=64)
    want = c.run().clone()
    streams, outs, spaces = [torch.cuda.Stream() for _ in range(2)], [torch.full_like(c.out, 7.0) for _ in range(2)], [c.workspace() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, out, ws in zip(streams, outs, spaces):
            c.entry(*c.args(ws, out=out), stream=s)
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, want)


def test_prepared(gpu):
    """Each entry point prepared once, run twice, with new values in the same buffers in between."""
    rng = np.random.default_rng(36)
    for name, k, v in (("fp8blk_paged_attn", 128, 128), ("fp8blk_latent_attn", 576, None)):
        c = _call(gpu, 36, [3000, 9], [2, 1], k, v)
        call = gpu.prepared(name, *c.args(c.workspace()))
        for step in range(2):
            c.q.copy_(normal(rng, *c.q.shape).bfloat16())
            c.out.fill_(7.0)
            assert call() == gpu.OK
            torch.cuda.synchronize()
            c.check(f"{name} {step}")
    rope = gpu.fp8blk_rope(gpu.fp8blk_rope_freqs(64, 1e4).to(DEV))
    q, k, v = (normal(rng, 5, h, n).to(DEV) for h, n in ((8, 64), (2, 64), (2, 64)))
    positions, slots = (torch.from_numpy(rng.permutation(64)[:5].astype(np.int32)).to(DEV) for _ in range(2))
    bufs = [[torch.full(s, 7.0, dtype=torch.bfloat16, device=DEV) for s in ((5, 8, 64), (4, 16, 2, 64), (4, 16, 2, 64))] for _ in range(2)]
    args = [(rope, positions, (None, q), b[0], (None, k), v, gpu.fp8blk_cache(b[1], b[2]), slots) for b in bufs]
    call = gpu.prepared("fp8blk_rope_append", *args[0])
    for step in range(2):
        positions.copy_(positions + 1000 * step)
        q.copy_(normal(rng, 5, 8, 64))
        gpu.fp8blk_rope_append(*args[1])
        assert call() == gpu.OK
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*bufs)), step


def test_what_the_binding_refuses(gpu):
    c = _call(gpu, 37, [3000, 9], [2, 1], 128, 128)
    ws = c.workspace()
    names = ("cache", "q", "table", "lens", "starts", "max_new", "max_len", "scale", "out", "ws", "causal", "window", "sinks")

    def call(entry=gpu.fp8blk_paged_attn, **kw):
        return entry(**{**dict(zip(names, c.args(ws))), **kw})

    for error, kw in ((TypeError, dict(q=c.q.half())), (TypeError, dict(out=c.out.float())), (ValueError, dict(q=c.q[..., :64])),
                      (ValueError, dict(out=c.out[:, :4])), (ValueError, dict(out=c.out[:2])), (TypeError, dict(table=c.paged.table.long())),
                      (ValueError, dict(lens=c.lens[:1])), (TypeError, dict(lens=c.lens.long())), (ValueError, dict(starts=c.starts[:2])),
                      (ValueError, dict(sinks=torch.zeros(3, device=DEV))), (TypeError, dict(sinks=torch.zeros(c.heads, dtype=torch.bfloat16, device=DEV))),
                      (TypeError, dict(q=c.q.cpu())), (ValueError, dict(lens=c.lens.cpu())), ((TypeError, ValueError), dict(table=c.paged.table.cpu())),
                      (gpu.Fp8BlkError, dict(ws=ws[:256])), (gpu.Fp8BlkError, dict(max_len=0)), (gpu.Fp8BlkError, dict(out=c.q[..., :128])),
                      (gpu.Fp8BlkError, dict(window=-1)), (gpu.Fp8BlkError, dict(entry=gpu.fp8blk_latent_attn)), (gpu.Fp8BlkError, dict(scale=float("nan")))):
        with pytest.raises(error):
            call(**kw)
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)  # noqa: E731
    for error, make in ((TypeError, lambda: gpu.fp8blk_cache(bf(2, 16, 2, 64), bf(2, 16, 2, 64).to(E4M3))), (TypeError, lambda: gpu.fp8blk_cache(bf(2, 16, 2, 64).float(), None)),
                        (ValueError, lambda: gpu.fp8blk_cache(bf(2, 16, 2, 64), bf(2, 16, 1, 64))), (ValueError, lambda: gpu.fp8blk_cache(bf(2, 16, 2, 64), bf(2, 16, 2, 64), v_cols=64)),
                        (TypeError, lambda: gpu.fp8blk_cache(bf(2, 16, 2, 64).cpu(), None)), (ValueError, lambda: gpu.fp8blk_cache(bf(2, 16, 64), None))):
        with pytest.raises(error):
            make()
    for bad in (gpu.fp8blk_cache(bf(200, 16, 2, 136)[..., :128], bf(200, 16, 2, 128)), gpu.fp8blk_cache(bf(200, 24, 2, 128), bf(200, 24, 2, 128)),
                gpu.fp8blk_cache(bf(200, 16, 3, 128), bf(200, 16, 3, 128)), gpu.fp8blk_cache(bf(200, 16, 2, 128), bf(200, 16, 2, 64))):
        with pytest.raises((gpu.Fp8BlkError, ValueError)):  # a stride, page size, number of heads or width that no call takes
            call(cache=bad)
    rope, cache = gpu.fp8blk_rope(gpu.fp8blk_rope_freqs(64, 1e4).to(DEV)), gpu.fp8blk_cache(bf(2, 16, 2, 64), bf(2, 16, 2, 64))
    n32 = torch.arange(4, dtype=torch.int32, device=DEV)
    good = dict(rope=rope, positions=n32, q=(None, bf(4, 8, 64)), q_out=bf(4, 8, 64), k=(None, bf(4, 2, 64)), v=bf(4, 2, 64), cache=cache, slots=n32)
    gpu.fp8blk_rope_append(**good)
    for error, kw in ((TypeError, dict(positions=n32.long())), (ValueError, dict(slots=n32[:3])), (TypeError, dict(slots=n32.long())), (ValueError, dict(q_out=None)),
                      (TypeError, dict(q_out=bf(4, 8, 64).float())), (ValueError, dict(q_out=bf(4, 4, 64))), (ValueError, dict(k=None)), (ValueError, dict(cache=None)),
                      (ValueError, dict(v=None)), (ValueError, dict(v=bf(4, 1, 64))), (ValueError, dict(k=(None, bf(4, 1, 64)))), (ValueError, dict(k=(bf(4, 2, 8), bf(4, 2, 64)))),
                      (ValueError, dict(q=(None, bf(3, 8, 64)))), (ValueError, dict(q=(bf(4, 8, 8), None))), (TypeError, dict(q=(None, bf(4, 8, 64).half()))),
                      ((TypeError, ValueError), dict(k=(None, bf(4, 2, 64).cpu()))), (ValueError, dict(q_norm=bf(32))), (ValueError, dict(positions=n32[None])),
                      (gpu.Fp8BlkError, dict(eps=-1.0))):
        with pytest.raises(error):
            gpu.fp8blk_rope_append(**{**good, **kw})
