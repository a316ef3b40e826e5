"""GPU: a verify panel's rows are those of single tokens bit for bit, for every kernel and split that panels take."""
import numpy as np
import pytest
import torch

from attention_plain import DEV, Call, Paged

pytestmark = pytest.mark.gpu


def _same(gpu, seed, L, k, v, heads, kv, page, e4m3, window, rows, T=16, also=90):
    rng = np.random.default_rng(seed)
    c = Call(gpu, rng, Paged(gpu, rng, [L, also], kv, k, v, page, e4m3), [T, min(9, also)], heads, sinks=True, window=window)
    print(L, k, v, heads, kv, page, e4m3, window, flush=True)
    c.run()
    for i in rows:
        lens = torch.tensor([L - T + 1 + i, 0], dtype=torch.int32, device=DEV)
        starts = torch.tensor([0, 1, 1], dtype=torch.int32, device=DEV)
        for n in (1, 2):  # alone, and as the last row of a panel of two
            if i < n - 1:
                continue
            out = torch.empty_like(c.out[:n])
            starts[1:] = n
            c.entry(c.paged.cache, c.q[i - n + 1:i + 1], c.paged.table, lens, starts, n, c.max_len, c.scale, out, c.workspace(), True, window, c.sinks)
            assert torch.equal(out[n - 1].view(torch.int16), c.out[i].view(torch.int16)), (i, n)
    return c


@pytest.mark.parametrize("k", [512, 576])
@pytest.mark.parametrize("heads", [16, 33, 64, 128])
@pytest.mark.parametrize("L", [300, 4000, 9001, 20000])
def test_latent_panels_of_many_heads(gpu, k, heads, L):
    """32 and 64 rows a workgroup (2 sequences of more than 8192 or 4096 keys of 64 or 128 heads), with splits and without, windows that begin in one."""
    for window in (0, L // 3):
        c = _same(gpu, 50, L, k, None, heads, 1, 64 if L > 300 else 1, False, window, (0, 1, 9, 15))
        if L <= 4000:
            c.check(f"{k} {heads} {L}")


@pytest.mark.parametrize("k,v", [(64, 64), (128, 128), (192, 128), (256, 256)])
@pytest.mark.parametrize("page", [1, 16, 64])
@pytest.mark.parametrize("e4m3", [False, True])
def test_panels_over_small_pages_and_several_row_tiles(gpu, k, v, page, e4m3):
    for heads, kv, window in ((8, 2, 0), (20, 1, 0), (16, 1, 1000)):
        c = _same(gpu, 51, 3000, k, v, heads, kv, page, e4m3, window, (0, 3, 15))
        c.check(f"{k} {page} {e4m3} {heads}")
