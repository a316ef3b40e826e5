"""GPU: fp8blk_rope_append at the ends of its numbers' range and of its launch's forms."""
import pytest
import torch

from test_gpu_rope_append import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("norm", ["pass", "whole"])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("spread,eps", [(1e19, 1e-5), (1e30, 0.0), (3e37, 1e-5), (1e-20, 0.0), (1e-25, 1e-38), (1e-36, 0.0), (1e-25, 1e-5), (1e-18, 1e-36)])
def test_norms_of_any_size(gpu, norm, kind, spread, eps):
    """Rows whose squares leave f32's range, above or below, and eps above, beside and below
    them: x / sqrt(mean x^2 + eps) is of a size of 1 or below all the same. bf16 and f32
    values of 1e-36 are normal ones still; one row is of ordinary size, one 0 (with eps)."""
    c = Case(gpu, 3, 9, 6, 3, 512 if norm == "pass" else 64, 64, 0 if norm == "pass" else 64, kind, False, 16, norm=norm, mscale=1.25, spread=spread)
    c.eps = eps
    for parts in (c.q, c.k):
        for t in parts:
            t[1] = torch.randn(t.shape[1:], device=t.device).to(t.dtype)
            if eps:
                t[2] = 0
    c.run()
    c.check(f"{norm} {kind} {spread} {eps}")


@pytest.mark.parametrize("N", [1024, 1025, 2500])
@pytest.mark.parametrize("pass_cols,rot,v_cols,heads,kv", [(0, 128, 128, 12, 4), (64, 64, 128, 5, 1), (512, 64, 0, 16, 1), (24, 40, 64, 33, 3)])
@pytest.mark.parametrize("e4m3", [False, True])
def test_many_tokens(gpu, N, pass_cols, rot, v_cols, heads, kv, e4m3):
    """Past 1024 tokens a workgroup takes all of a token's rows, one after the other; slots that are none among them."""
    if e4m3 and not v_cols:
        pytest.skip("latent caches are bf16")
    norm = "pass" if not v_cols else ("whole", "none")[N % 2]
    c = Case(gpu, N, N, heads, kv, pass_cols, rot, v_cols, ("f32", "bf16")[heads % 2], e4m3, 16, None, heads % 3 == 0, kv > 1, norm, 0.75)
    c.slots[::7] = -1
    c.run()
    c.check(f"{N} {pass_cols}+{rot} {heads}/{kv} {norm} {e4m3}")


def test_a_tokens_bits_do_not_depend_on_the_others(gpu):
    """Both forms of the launch, and one token alone."""
    c = Case(gpu, 5, 1500, 12, 2, 64, 64, 128, norm="whole", far=3000)
    c.run()
    want = [t.clone() for t in (c.q_out, c.ck, c.cv)]
    for lo, hi in ((0, 1), (700, 1000), (1499, 1500)):
        d = Case(gpu, 5, 1500, 12, 2, 64, 64, 128, norm="whole", far=3000)
        cut = lambda parts: tuple(t[lo:hi] for t in parts)  # noqa: E731
        gpu.fp8blk_rope_append(c.rope, c.positions[lo:hi], cut(c.q), d.q_out[lo:hi], cut(c.k), c.v[lo:hi], d.cache, c.slots[lo:hi], c.q_norm, c.k_norm, c.eps)
        page, slot = c.slots[lo:hi].long() // 16, c.slots[lo:hi].long() % 16
        assert torch.equal(d.q_out[lo:hi], want[0][lo:hi]) and torch.equal(d.ck[page, slot], want[1][page, slot]) and torch.equal(d.cv[page, slot], want[2][page, slot])
