"""GPU: attention calls whose sizes on the host are far above what there is to do."""
import numpy as np
import pytest
import torch

from attention_plain import Call, Paged, assert_attends, attend

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("seqs,heads,max_new", [(32, 128, 65536), (63, 128, 65536), (64, 128, 65536), (4096, 16, 8192)])
def test_latent_launches_of_the_most_rows(gpu, seqs, heads, max_new):
    """Bounds at the documented limit, seqs * heads * ceil(max_new / 128) up to 2^22, of which
    few rows are there: launches of 2^31 threads and more."""
    assert seqs * heads * -(-max_new // 128) <= 1 << 22
    rng = np.random.default_rng(40)
    lens = [1 + 7 * s % 90 for s in range(seqs)]
    c = Call(gpu, rng, Paged(gpu, rng, lens, 1, 576, None, 16), [1 + int(lens[s] > 2 and s % 5 == 0) for s in range(seqs)], heads, behind=1)
    c.max_new = max_new
    print(seqs, heads, max_new, flush=True)
    c.run()
    for s in (0, 1, 5, seqs // 2, seqs - 1):
        lo, n = c.first[s], c.new[s]
        want, bound = attend(*c.paged.rows(s), c.q[lo:lo + n], lens[s] - n, c.scale)
        assert_attends(c.out[lo:lo + n], want, bound, f"{seqs} {heads} {max_new} sequence {s}")
    assert (c.out[-1] == 7).all()


@pytest.mark.parametrize("k,v,heads", [(128, 128, 16), (64, 64, 40), (576, None, 16), (576, None, 128)])
def test_one_workspace_for_every_step(gpu, k, v, heads):
    """Decode, a verify panel and chunks of fewer and more sequences with a workspace for the largest of each, of which some need none and smaller ones some."""
    rng = np.random.default_rng(42)
    lens = [5000, 400, 1300, 60]
    paged = Paged(gpu, rng, lens, 1 if v is None else 4, k, v, 16)
    ws = torch.full((gpu.fp8blk_attn_most_bytes(paged.cache, heads, 4, 400, 5000),), 255, dtype=torch.uint8, device=paged.cache_k.device)
    for new in ([1, 1, 1, 1], [16, 3, 1, 0], [400, 1, 90, 7], [0, 0, 40, 0], [5, 0, 0, 0]):
        c = Call(gpu, rng, paged, new, heads, behind=1)
        c.entry(*c.args(ws))
        c.check(f"{k} {heads} {new}")
