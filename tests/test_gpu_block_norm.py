"""GPU: fp8blk_block_norm against its plain form in 64 bits."""
import numpy as np
import pytest
import torch

from layer_plain import H, U, assert_within, block_norm, normal

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _case(seed, N, cols, resid="f32", gate="cols", post=True, spread=1.0):
    rng = np.random.default_rng(seed)
    r = normal(rng, N, cols) * 4 * spread
    r = r.bfloat16() if resid == "bf16" else r
    y = normal(rng, N, cols) * spread
    g = {"none": None, "flat": (cols,), "cols": (1, cols), "rows": (N, cols)}[gate]
    return dict(resid=r, y=y, post_w=(1 + 0.2 * normal(rng, cols)).bfloat16() if post else None,
                gate=None if g is None else normal(rng, *g).bfloat16(), pre_w=(1 + 0.2 * normal(rng, cols)).bfloat16())


def _run(gpu, c, scale, eps, inplace=False, stream=None):
    d = {k: None if v is None else v.to(DEV) for k, v in c.items()}
    out = None if c["y"] is None else d["resid"] if inplace else torch.full_like(d["resid"], float("nan"))
    x = None if c["pre_w"] is None else torch.full(d["resid"].shape, float("nan"), dtype=torch.bfloat16, device=DEV)
    gpu.fp8blk_block_norm(d["resid"], d["y"], d["post_w"], d["gate"], scale, out, d["pre_w"], eps, x, stream=stream)
    torch.cuda.synchronize()
    return out, x


def _check(c, scale, eps, out, x, what):
    r64, dr, x64, dx = block_norm(c["resid"], c["y"], c["post_w"], c["gate"], scale, c["pre_w"], eps)
    if out is not None:
        assert out.dtype == c["resid"].dtype
        assert_within(out, r64, dr + (H * r64.abs() if out.dtype == torch.bfloat16 else 0), what + " resid_out")
    if x is not None:
        assert_within(x, x64, dx + H * (x64.abs() + dx) + 2.0 ** -134, what + " x_next")


@pytest.mark.parametrize("N,cols", [(1, 16), (1, 4096), (2, 48), (3, 1040), (5, 2064), (16, 7168), (17, 8208),
                                    (33, 12304), (2, 16400), (3, 32784), (1, 65536), (257, 512), (4100, 272)])
@pytest.mark.parametrize("resid", ["f32", "bf16"])
def test_matches_plain(gpu, N, cols, resid):
    print("block norm", N, cols, resid, flush=True)
    gate = ("none", "flat", "cols", "rows")[(N + cols // 16) % 4]
    c = _case(N * cols, N, cols, resid, gate, post=(N % 3 != 0))
    out, x = _run(gpu, c, 0.75, 1e-6)
    _check(c, 0.75, 1e-6, out, x, f"{N}x{cols} {resid} {gate}")


@pytest.mark.parametrize("gate", ["none", "flat", "cols", "rows"])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("resid", ["f32", "bf16"])
def test_options(gpu, gate, post, resid):
    c = _case(11, 6, 528, resid, gate, post)
    out, x = _run(gpu, c, -1.5, 1e-5)
    _check(c, -1.5, 1e-5, out, x, f"{gate} {post} {resid}")
    again, x2 = _run(gpu, c, -1.5, 1e-5, inplace=True)
    assert torch.equal(again, out) and torch.equal(x2, x)
    # only the sum
    only = dict(c, pre_w=None)
    out2, none = _run(gpu, only, -1.5, 1e-5)
    assert none is None and torch.equal(out2, out)
    # only the norm
    first = dict(c, y=None, post_w=None, gate=None)
    none, x3 = _run(gpu, first, 0.0, 1e-5)
    assert none is None
    _check(first, 0.0, 1e-5, None, x3, "first norm")


def test_rows_do_not_depend_on_the_panel(gpu):
    for cols in (1040, 4096, 16400):
        c = _case(5, 700, cols, "bf16", "rows", True)
        out, x = _run(gpu, c, 1.0, 1e-6)
        for i in (0, 1, 350, 699):
            one = {k: v[i:i + 1] if k in ("resid", "y", "gate") else v for k, v in c.items()}
            o1, x1 = _run(gpu, one, 1.0, 1e-6)
            assert torch.equal(o1[0], out[i]) and torch.equal(x1[0], x[i]), (cols, i)


def test_zero_rows_and_values_that_are_not_finite(gpu):
    """A zero row gives zeros (eps > 0) or NaN (eps = 0: 0/0, as the formula
    says); a row with an infinity or NaN keeps it to itself."""
    c = _case(9, 5, 272, "f32", "none", True)
    c["resid"][1] = 0
    c["y"][1] = 0
    c["y"][2, 7] = float("inf")
    c["resid"][3, 100] = float("nan")
    out, x = _run(gpu, c, 1.0, 1e-6)
    assert (x[1] == 0).all() and (out[1] == 0).all()
    assert x[2].isnan().any() and x[3].isnan().all()
    ok = {k: v[[0, 1, 4]] if k in ("resid", "y") else v for k, v in c.items()}
    _check(ok, 1.0, 1e-6, out[[0, 1, 4]], x[[0, 1, 4]], "the other rows")
    _, x = _run(gpu, dict(c, y=None, post_w=None, gate=None), 1.0, 0.0)
    assert x[1].isnan().all() and torch.isfinite(x[[0, 2, 4]].float()).all()


def test_rows_behind_the_panel_are_left_alone(gpu):
    c = _case(3, 9, 1040, "bf16", "rows", True)
    d = {k: v.to(DEV) for k, v in c.items()}
    out = torch.full((12, 1040), 7.0, dtype=torch.bfloat16, device=DEV)
    x = torch.full((12, 1040), 7.0, dtype=torch.bfloat16, device=DEV)
    gpu.fp8blk_block_norm(d["resid"], d["y"], d["post_w"], d["gate"], 1.0, out[:9], d["pre_w"], 1e-6, x[:9])
    torch.cuda.synchronize()
    assert (out[9:] == 7).all() and (x[9:] == 7).all()
    _check(c, 1.0, 1e-6, out[:9], x[:9], "first rows")


def test_many_rows_past_32_bit_offsets(gpu):
    """65536 rows of 49152 columns: the last rows lie past 2^31 elements."""
    N, cols = 65536, 49152
    resid = torch.zeros((N, cols), dtype=torch.bfloat16, device=DEV)
    c = _case(21, 3, cols, "bf16", "none", False)
    at = [0, 40000, N - 1]
    resid[at] = c["resid"].to(DEV)
    x = torch.empty((N, cols), dtype=torch.bfloat16, device=DEV)
    gpu.fp8blk_block_norm(resid, None, None, None, 0.0, None, c["pre_w"].to(DEV), 1e-6, x)
    torch.cuda.synchronize()
    _check(dict(c, y=None), 0.0, 1e-6, None, x[at], "rows past 2^31")
    assert (x[12345] == 0).all() and (x[N - 2] == 0).all()


@pytest.mark.parametrize("spread,eps", [(2.0 ** 54, 1e-6), (2.0 ** -58, 0.0)])
def test_the_range_of_the_squares(gpu, spread, eps):
    """Rows near both ends of what f32 sums of squares hold: 4096 of 2^112, and
    squares around 2^-112 beside an eps of 0."""
    c = _case(27, 3, 4096, "f32", "none", True, spread)
    first = dict(c, y=None, post_w=None)
    none, x = _run(gpu, first, 0.0, eps)
    _check(first, 0.0, eps, None, x, f"{spread}")
    out, x = _run(gpu, c, 0.25 * spread, eps)
    _check(c, 0.25 * spread, eps, out, x, f"{spread}")
