"""CPU: what rotary positions, paged caches and attention refuse, at the C ABI
(addresses that are never read) and in the Python binding."""
import ctypes
import math
import os

import pytest
import torch

import block_scaled_fp8_fp8blk_amd as fb

P = 1 << 24  # a fake, aligned address: every call here refuses before any device work
S = 1 << 24  # distance between fake buffers
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fb.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return fb.load()


def cache(**kw):
    a = dict(k=P, v=P + S, pages=8, page_size=16, heads=2, k_cols=128, v_cols=128, k_page=4096, k_slot=256, k_head=128, v_page=4096,
             v_slot=256, v_head=128, type=fb.TYPE_BF16, k_scale=1.0, v_scale=1.0)
    a.update(kw)
    return fb.CacheRecord(**a)


BAD_CACHES = [
    dict(k=None), dict(k=P + 8), dict(v=P + S + 2), dict(pages=0), dict(pages=-1), dict(pages=1 << 27), dict(page_size=0), dict(page_size=24),
    dict(page_size=1 << 17), dict(heads=0), dict(heads=fb.MAX_HEADS + 1), dict(k_cols=0), dict(k_cols=120), dict(v_cols=8),
    dict(v_cols=fb.MAX_HEAD_COLS + 16), dict(k_page=64), dict(k_slot=0), dict(k_head=120), dict(k_slot=264), dict(v_page=-4096), dict(v_head=0),
    dict(v_slot=136), dict(k_page=1 << 60), dict(type=0), dict(type=3), dict(k_scale=0.5), dict(v_scale=2.0),
    dict(type=2, k_scale=0.0), dict(type=2, v_scale=-1.0), dict(type=2, k_scale=NAN), dict(type=2, v_scale=INF), dict(type=2, k_scale=1e-38)]


def heads(**kw):
    a = dict(pass_=P + 3 * S, rot=P + 4 * S, pass_token=1024, pass_head=64, rot_token=1024, rot_head=64, heads=2, pass_cols=64, norm_cols=0,
             norm=None, type=0)
    a.update(kw)
    return fb.HeadsRecord(**a)


def append(lib, rope=None, positions=P + 10 * S, N=4, q=None, q_out=P + 9 * S, q_strides=(256, 128), k=None, v=None, c=None, slots=P + 11 * S,
           eps=1e-6, drop=()):
    r = fb.RopeRecord(**{**dict(freqs=P + 12 * S, rot=64, interleaved=0, rot_first=1, mscale=1.0), **(rope or {})})
    hq, hk = heads(**(q or {})), heads(**{**dict(pass_=P + 5 * S, rot=P + 6 * S), **(k or {})})
    hv = heads(**{**dict(pass_=P + 7 * S, rot=None, rot_token=0, rot_head=0, pass_cols=128, pass_head=128), **(v or {})})
    record = cache(**(c or {}))
    args = dict(rope=ctypes.byref(r), positions=positions, N=N, q=ctypes.byref(hq), q_out=q_out, t=q_strides[0], h=q_strides[1],
                k=ctypes.byref(hk), v=ctypes.byref(hv), cache=ctypes.byref(record), slots=slots, eps=eps)
    for name in drop:
        args[name] = None
    return lib.fp8blk_rope_append(*args.values(), None)


@pytest.mark.parametrize("kw", [
    dict(rope=dict(freqs=None)), dict(rope=dict(freqs=P + 4)), dict(rope=dict(rot=0)), dict(rope=dict(rot=60)), dict(rope=dict(rot=264)),
    dict(rope=dict(mscale=NAN)), dict(rope=dict(mscale=INF)), dict(positions=None), dict(positions=P + 2), dict(N=0), dict(N=fb.MAX_PANEL + 1),
    dict(eps=-1.0), dict(eps=NAN), dict(eps=INF), dict(slots=P + 1), dict(drop=["rope"]), dict(drop=["q"]), dict(drop=["q_out"]), dict(drop=["k"]),
    dict(drop=["v"]), dict(drop=["cache"]), dict(drop=["slots"]), dict(drop=["k", "cache", "slots"]), dict(drop=["q", "q_out", "k", "v", "cache", "slots"]),
    dict(q=dict(heads=0)), dict(q=dict(heads=fb.MAX_HEADS + 1)), dict(q=dict(pass_cols=60)), dict(q=dict(pass_cols=1024)), dict(q=dict(pass_cols=0)),
    dict(q=dict(pass_=None)), dict(q=dict(rot=None)), dict(q=dict(pass_=P + 8)), dict(q=dict(rot=P + 4)), dict(q=dict(type=2)), dict(q=dict(type=-1)),
    dict(q=dict(pass_token=-8)), dict(q=dict(pass_head=4)), dict(q=dict(rot_token=12)), dict(q=dict(rot_head=1 << 41)), dict(q=dict(norm_cols=128)),
    dict(q=dict(norm=P + 13 * S, norm_cols=0)), dict(q=dict(norm=P + 13 * S, norm_cols=72)), dict(q=dict(norm=P + 13 * S + 2, norm_cols=128)),
    dict(q_out=P + 9 * S + 8), dict(q_strides=(64, 128)), dict(q_strides=(256, 64)), dict(q_strides=(260, 128)),
    dict(k=dict(heads=1)), dict(k=dict(pass_cols=128)), dict(v=dict(heads=4)), dict(v=dict(pass_cols=64)), dict(v=dict(rot=P + 4 * S)),
    dict(v=dict(norm=P, norm_cols=128)), dict(c=dict(v=None)),
    # outputs over inputs and over each other
    dict(q_out=P + 3 * S), dict(q_out=P + 4 * S - 16), dict(q_out=P + 5 * S), dict(q_out=P + 7 * S), dict(q_out=P + 10 * S), dict(q_out=P + 11 * S),
    dict(q_out=P + 12 * S), dict(q_out=P), dict(q_out=P + S + 32), dict(c=dict(k=P + 3 * S)), dict(c=dict(v=P + 6 * S)), dict(c=dict(k=P + 10 * S)),
    dict(c=dict(v=P + 12 * S)), dict(q=dict(norm=P + 9 * S, norm_cols=128))] + [dict(c=b) for b in BAD_CACHES])
def test_append_refusals(lib, kw):
    assert append(lib, **kw) == fb.ERR_ARG


@pytest.mark.parametrize("a", [(0, 1e4, 1, 1, 1, 1), (12, 1e4, 1, 1, 1, 1), (512, 1e4, 1, 1, 1, 1), (64, 0.0, 1, 1, 1, 1), (64, NAN, 1, 1, 1, 1),
                               (64, INF, 1, 1, 1, 1), (64, 1e4, 0.5, 1, 1, 1), (64, 1e4, INF, 1, 1, 1), (64, 1e4, 2, 0, 32, 1), (64, 1e4, 2, 4096, 1, 32),
                               (64, 1e4, 2, 4096, 32, -1), (64, 1e4, 2, 4096, NAN, 1), (64, 1e4, 2, NAN, 32, 1)])
def test_freqs_refusals(lib, a):
    with pytest.raises(fb.Fp8BlkError):
        fb.fp8blk_rope_freqs(*a)
    assert lib.fp8blk_rope_freqs(64, 1e4, 1.0, 1.0, 1.0, 1.0, None) == fb.ERR_ARG


def test_freqs_where_the_parts_meet(lib):
    """fast == slow: no pair in between; a pair with exactly that many turns stays."""
    original = 32 * 2 * math.pi
    f = fb.fp8blk_rope_freqs(8, 16.0, 4.0, original, 8.0, 8.0)  # turns: 32, 16, 8, 4
    assert f.tolist() == pytest.approx([1.0, 0.5, 0.25, 0.125 / 4], rel=1e-14)


def attn(lib, latent=False, c=None, q=P + 2 * S, q_strides=(1024, 128), N=4, heads=8, batch=None, scale=0.1, window=0, sinks=None, out=P + 3 * S,
         out_strides=(1024, 128), ws=P + 8 * S, wsb=1 << 40, drop=()):
    base = dict(v=None, heads=1, k_cols=576, v_cols=512, k_page=16 * 576, k_slot=576, k_head=576) if latent else {}
    record = cache(**{**base, **(c or {})})
    if latent:
        q_strides, out_strides = ((8 * 576, 576) if t == (1024, 128) else t for t in (q_strides, out_strides))
    b = fb.BatchRecord(**{**dict(table=P + 4 * S, lens=P + 5 * S, starts=P + 6 * S, seqs=2, max_pages=9, max_new=2, max_len=100), **(batch or {})})
    args = dict(cache=ctypes.byref(record), q=q, qt=q_strides[0], qh=q_strides[1], N=N, heads=heads, batch=ctypes.byref(b), scale=scale, causal=1,
                window=window, sinks=sinks, out=out, ot=out_strides[0], oh=out_strides[1], ws=ws, wsb=wsb)
    for name in drop:
        args[name] = None
    return (lib.fp8blk_latent_attn if latent else lib.fp8blk_paged_attn)(*args.values(), None)


@pytest.mark.parametrize("latent", [False, True])
@pytest.mark.parametrize("kw", [
    dict(drop=["cache"]), dict(drop=["batch"]), dict(q=None), dict(out=None), dict(q=P + 2 * S + 8), dict(out=P + 3 * S + 2), dict(N=0),
    dict(N=fb.MAX_PANEL + 1), dict(heads=0), dict(heads=1025), dict(q_strides=(-8, 640)), dict(q_strides=(4608, 4)), dict(out_strides=(4608, 32)),
    dict(out_strides=(16, 640)), dict(out_strides=(4612, 640)), dict(scale=NAN), dict(scale=INF), dict(window=-1), dict(window=1 << 30),
    dict(sinks=P + 2), dict(batch=dict(table=None)), dict(batch=dict(lens=None)), dict(batch=dict(starts=None)), dict(batch=dict(table=P + 1)),
    dict(batch=dict(lens=P + 2)), dict(batch=dict(starts=P + 3)), dict(batch=dict(seqs=0)), dict(batch=dict(seqs=fb.MAX_PANEL + 1)),
    dict(batch=dict(max_pages=0)), dict(batch=dict(max_pages=(1 << 30) + 1)), dict(batch=dict(max_new=0)), dict(batch=dict(max_new=fb.MAX_PANEL + 1)),
    dict(batch=dict(max_len=0)), dict(batch=dict(max_len=1 << 30)), dict(scale=-3e38), dict(batch=dict(seqs=1 << 16, max_new=1025)),
    dict(batch=dict(seqs=1 << 15, max_new=1 << 16), heads=64), dict(N=1 << 16, heads=1024, batch=dict(seqs=4097)),
    # out over q, the cache and the batch
    dict(out=P + 2 * S), dict(out=P + 2 * S + 48), dict(out=P), dict(out=P + 4 * S), dict(out=P + 5 * S), dict(out=P + 6 * S),
    dict(sinks=P + 3 * S + 16)] + [dict(c=b) for b in BAD_CACHES if "v" not in b and not any(k.startswith("v_") for k in b)])
def test_attention_refusals(lib, latent, kw):
    assert attn(lib, latent, **kw) == fb.ERR_ARG


@pytest.mark.parametrize("kw", [
    dict(heads=7), dict(c=dict(v=None)), dict(c=dict(v=P + S + 8)), dict(out=P + S), dict(c=dict(k_cols=64, v_cols=128)), dict(c=dict(v_cols=64)),
    dict(c=dict(k_cols=96, v_cols=96)), dict(c=dict(k_cols=512, v_cols=512, k_head=512, k_slot=1024, v_head=512, v_slot=1024)),
    dict(c=dict(k_cols=128, v_cols=128, v_slot=112)), dict(c=dict(type=2, k_scale=2.0 ** 90), scale=2.0 ** 40)])
def test_paged_attention_refusals(lib, kw):
    assert attn(lib, **kw) == fb.ERR_ARG


@pytest.mark.parametrize("kw", [
    dict(c=dict(v=P + S, v_page=16 * 576, v_slot=576, v_head=576)), dict(c=dict(type=2)), dict(c=dict(heads=2)), dict(c=dict(v_cols=256)),
    dict(c=dict(k_cols=544)), dict(c=dict(v_cols=592)), dict(c=dict(k_cols=640, k_slot=640, k_head=640, k_page=10240))])
def test_latent_attention_refusals(lib, kw):
    assert attn(lib, True, **kw) == fb.ERR_ARG


def test_workspace(lib):
    """attn_bytes is 0 for sizes that the call refuses, and one byte less than it
    asks for, or none, is refused; the longest caches ask for no more splits than
    a launch has room for."""
    def need(latent=False, heads=8, seqs=2, max_new=2, max_len=100000, window=0):
        base = dict(v=None, heads=1, k_cols=576, v_cols=512, k_page=16 * 576, k_slot=576, k_head=576) if latent else {}
        return lib.fp8blk_attn_bytes(ctypes.byref(cache(**base)), heads, seqs, max_new, max_len, window)
    for latent in (False, True):
        n = need(latent)
        assert n > 0
        long = dict(batch=dict(max_len=100000))
        assert attn(lib, latent, wsb=n - 1, **long) == attn(lib, latent, ws=None, **long) == attn(lib, latent, ws=P + 8 * S + 128, **long) == fb.ERR_WORKSPACE
        assert need(latent, seqs=1 << 16, heads=128) == need(latent, seqs=0) == need(latent, max_len=1 << 30) == 0
        cols = 514 if latent else 130
        for seqs in (1, 100, 255):  # rows of the join's launch, and splits of f32 sums
            n = need(latent, seqs=seqs, max_new=16, max_len=(1 << 30) - 1)
            assert n % (seqs * 16 * 8 * cols * 4) == 0 and seqs * n // (seqs * 16 * 8 * cols * 4) <= 1 << 15


U8, F32, BF, I32 = torch.uint8, torch.float32, torch.bfloat16, torch.int32


def test_the_binding_takes_gpu_tensors(lib):
    z = torch.zeros
    with pytest.raises(TypeError, match="CUDA"):
        fb.fp8blk_rope(z(32, dtype=torch.float64))
    with pytest.raises(TypeError, match="CUDA"):
        fb.fp8blk_cache(z(2, 16, 2, 128, dtype=BF), z(2, 16, 2, 128, dtype=BF))
