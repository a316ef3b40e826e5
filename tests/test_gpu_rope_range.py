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
