"""CPU: the workspace of attention calls: one for the largest batch, chunk and cache takes all smaller ones."""
import ctypes
import os
import random

import pytest

import block_scaled_fp8_fp8blk_amd as fb

P = 1 << 24  # a fake, aligned address: nothing here reads it


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(fb.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return fb.load()


def record(heads, k, v):
    d = k if v is None else max(k, v)
    strides = {f"{n}_{part}": s for n in "kv" for part, s in (("page", 16 * heads * d), ("slot", heads * d), ("head", d))}
    return fb.CacheRecord(k=P, v=None if v is None else 2 * P, pages=8, page_size=16, heads=heads, k_cols=k, v_cols=512 if v is None else v,
                          type=fb.TYPE_BF16, k_scale=1.0, v_scale=1.0, **strides)


CACHES = [(4, 32, 128, 128), (8, 64, 64, 64), (2, 16, 256, 256), (16, 16, 192, 128), (1, 1, 128, 128), (3, 33, 64, 64), (1, 16, 576, None), (1, 128, 576, None),
          (1, 33, 512, None), (1, 1, 512, None)]


@pytest.mark.parametrize("kv,heads,k,v", CACHES)
@pytest.mark.parametrize("window", [0, 100, 4000])
def test_the_most_bytes_of_all_smaller_calls(lib, kv, heads, k, v, window):
    """Small bounds whole, large ones at sizes drawn over their logarithm and beside the
    bounds; and it is not far above what some call needs."""
    cache = record(kv, k, v)
    need = lambda s, t, n: lib.fp8blk_attn_bytes(ctypes.byref(cache), heads, s, t, n, window)  # noqa: E731
    most = lambda s, t, n: lib.fp8blk_attn_most_bytes(ctypes.byref(cache), heads, s, t, n, window)  # noqa: E731
    for S, T, L in ((3, 20, 700), (12, 3, 900)):
        top = most(S, T, L)
        assert all(need(s, t, n) <= top for s in range(1, S + 1) for t in range(1, T + 1) for n in range(1, L + 1, 13))
    rng = random.Random(kv + heads + k + window)
    some = lambda hi: max(1, min(hi, rng.choice((int(round(hi ** rng.random())), hi, hi - 1))))  # noqa: E731
    for S, T, L in ((1, 1, 16384), (1, 16, 4096), (32, 1, 16384), (127, 1, 4096), (256, 16, 8000), (600, 1, 5000), (1, 512, 8192), (1, 8192, 8192),
                    (8, 300, 9000), (65536, 1, 131072), (65536, 65536, (1 << 30) - 1)):
        top, seen = most(S, T, L), 0
        assert most(S, T, L) >= most(max(S // 2, 1), max(T // 2, 1), L)
        # the last tokens of whole row tiles, in launches of up to some hundred workgroups
        sizes = [(s, max(1, min(T, tiles * (128 if v else 64) * kv // heads)), L) for s in range(1, min(S, 5) + 1) for tiles in range(1, 400 // s + 2)]
        for size in sizes + [(some(S), some(T), some(L)) for _ in range(2000)]:
            n = need(*size)
            assert n <= top, (size, n, top)
            seen = max(seen, n)
        assert top <= 4 * seen, (S, T, L, seen, top)


def test_refused_sizes_need_none(lib):
    cache = record(4, 128, 128)
    most = lambda *a: lib.fp8blk_attn_most_bytes(ctypes.byref(cache), *a)  # noqa: E731
    assert most(32, 8, 1, 4096, 0) > 0 and lib.fp8blk_attn_most_bytes(None, 32, 8, 1, 4096, 0) == 0
    for bad in ((30, 8, 1, 4096, 0), (0, 8, 1, 4096, 0), (32, 0, 1, 4096, 0), (32, 8, 0, 4096, 0), (32, 8, 1, 0, 0), (32, 8, 1, 4096, -1), (32, 8, 1, 1 << 30, 0),
                (32, 65537, 1, 4096, 0), (32, 8, 65537, 4096, 0), (32, 8, 1, 4096, 1 << 30)):
        assert most(*bad) == 0
