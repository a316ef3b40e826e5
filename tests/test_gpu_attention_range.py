"""GPU: attention at the ends of its numbers' range: scores whose rounding steps are
far above 1, and rows that give 0 whatever the values are."""
import numpy as np
import pytest
import torch

from attention_plain import DEV, Call, Paged
from layer_plain import H, U

pytestmark = pytest.mark.gpu

WIDTHS = [(64, 64), (128, 128), (192, 128), (256, 256), (512, None), (576, None)]  # None: a latent cache
IDS = ["64", "128", "192+128", "256", "latent512", "latent576"]


def _call(gpu, seed, lens, new, k, v, group=4, page=16, kv=2, e4m3=False, **kw):
    rng = np.random.default_rng(seed)
    kv = 1 if v is None else kv
    return Call(gpu, rng, Paged(gpu, rng, lens, kv, k, v, page, e4m3), new, kv * group, **kw)


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("T", [1, 7, 100])
@pytest.mark.parametrize("power", [22, 33, 50, 120])
def test_scores_of_any_size(gpu, k, v, e4m3, T, power):
    """Scores of 2^power that differ by 2^-4 of themselves or not at all: a row is the mean of
    the values whose scores are its highest. Every product is exact in f32, so equal scores
    get equal weights, and all others' are below 2^-2000; what is left is a sum of up to L f32
    ((L + 64) steps, as for any row) and the output's rounding. Heads of scale below 0 too."""
    if e4m3 and v is None:
        pytest.skip("latent caches are bf16")
    L = 700
    for scale in (0.11, -1.7):
        c = _call(gpu, power + T, [L, 30], [T, 1], k, v, e4m3=e4m3, scale=scale)
        p, i = c.paged.where(0, L)
        rng = np.random.default_rng(power)
        mantissa = lambda *s: torch.from_numpy((1 + rng.integers(0, 8, s) / 8) * rng.choice([-1.0, 1.0], s)).to(DEV)  # noqa: E731
        h = c.paged.cache_k.shape[2]
        raw, keys = torch.uint8 if e4m3 else torch.int16, (16 * mantissa(L, h)).to(c.paged.cache_k.dtype)  # 3 bits: e4m3 has them too
        c.paged.cache_k.view(raw)[p, i, :, 0] = keys.view(raw)
        c.q.zero_()
        c.q[:, :, 0] = (2.0 ** (power - 4) / (c.paged.k_scale if e4m3 else 1.0) * mantissa(c.N, c.heads)).bfloat16()
        c.run()
        kk, vv = c.paged.rows(0)
        code = kk[:, :, 0] / c.paged.k_scale
        at = torch.arange(L - T, L, device=DEV)[:, None]
        seen = torch.arange(L, device=DEV) <= at
        for head in range(c.heads):
            of = head * h // c.heads
            z = scale * c.q[:T, head, 0].double()[:, None] * code[:, of].round()
            z[~seen] = -float("inf")
            w = (z == z.amax(1, keepdim=True)).double()
            w /= w.sum(1, keepdim=True)
            want, size = w @ vv[:, of], w @ vv[:, of].abs()
            got = c.out[:T, head].double()
            far = (got - want).abs() - H * want.abs() - 1.01 * (L + 64) * 2 * U * size - 2.0 ** -130
            assert not (~(far <= 0)).any(), f"{k} e4m3 {e4m3} T {T} 2^{power} scale {scale} head {head}: {int((~(far <= 0)).sum())} values off"


@pytest.mark.parametrize("k,v", WIDTHS, ids=IDS)
@pytest.mark.parametrize("T", [1, 8, 70])
@pytest.mark.parametrize("L", [200, 3000])
@pytest.mark.parametrize("sinks", [False, True])
def test_rows_of_no_weight_over_values_that_are_not_finite(gpu, k, v, T, L, sinks):
    """A row whose scores are all -inf gives 0, also where a value that it sees is an infinity
    or NaN; the other rows have it. Latent values are keys too: there it is an infinity in
    the column that makes the row's scores -inf."""
    c = _call(gpu, 41, [L, 20], [T, 1], k, v, sinks=sinks)
    p, i = c.paged.where(0, L)
    c.paged.cache_k[p, i, :, 0] = 1.0
    c.q[0, 1] = 0
    c.q[0, 1, 0] = float("-inf")
    for n, j in enumerate((3, L // 2, L - T)):  # seen by every row: inside whole tiles, and in the one where rows begin to differ
        if v is None:
            c.paged.cache_k[p[j], i[j], :, 0] = float("inf")
        else:
            c.paged.cache_v[p[j], i[j], :, 5 + n] = float("nan") if n == 1 else float("inf")
    c.run()
    assert (c.out[0, 1] == 0).all(), f"{k} {T} {L}: {int((c.out[0, 1] != 0).sum())} values are not 0"
    if v is not None:
        assert (~c.out[:T, [0, 2, 3], 5:8].isfinite()).all() and c.out[:T, [0, 2, 3], 8:].isfinite().all()
