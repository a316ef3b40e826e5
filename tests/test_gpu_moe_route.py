"""GPU: fp8blk_moe_route against its plain form in 64 bits."""
import numpy as np
import pytest
import torch

from layer_plain import U, normal, route

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _run(gpu, x, w, bias, score, K, normalize, scale):
    M, E, cols = x.shape[0], w.shape[0], w.shape[1]
    ids = torch.full((M, K), -7, dtype=torch.int32, device=DEV)
    p = torch.full((M, K), float("nan"), device=DEV)
    ws = torch.full((gpu.fp8blk_workspace_bytes(gpu.OP_MOE_ROUTE, E, cols, M),), 0xFF, dtype=torch.uint8, device=DEV)
    gpu.fp8blk_moe_route(w.to(DEV), None if bias is None else bias.to(DEV), x.to(DEV), score, normalize, scale, ids, p, ws)
    torch.cuda.synchronize()
    return ids.cpu(), p.cpu()


def _check(got, x, w, bias, score, K, normalize, scale, what):
    ids, p, gap = route(x, w, bias, score, K, normalize, scale)
    assert gap > 1e-11, f"{what}: the inputs hold a tie ({gap})"
    assert torch.equal(got[0].long(), ids), f"{what}: {int((got[0].long() != ids).sum())} choices differ"
    # 64-bit scores are good to 1e-12; then one rounding to f32
    off = (got[1].double() - p).abs()
    assert (off <= (U + 1e-12) * p.abs() + 2.0 ** -150).all(), f"{what}: weights off by {float((off / p.abs()).max())}"


def _inputs(seed, M, E, cols, bias):
    rng = np.random.default_rng(seed)
    x = normal(rng, M, cols).bfloat16()
    w = (normal(rng, E, cols) * 2 / cols ** 0.5).bfloat16()
    return x, w, normal(rng, E) * 0.3 if bias else None


@pytest.mark.parametrize("score", [0, 1, 2])
@pytest.mark.parametrize("M,E,cols,K", [(1, 1, 16, 1), (1, 8, 48, 2), (1, 256, 4096, 8), (2, 64, 512, 6), (4, 100, 2064, 4),
                                        (7, 65, 1040, 16), (13, 160, 2064, 6), (16, 256, 7168, 8), (16, 1024, 1024, 16),
                                        (17, 257, 528, 3), (33, 16, 272, 16), (130, 96, 2880, 4), (515, 128, 1552, 8),
                                        (64, 1000, 80, 5), (1, 32, 65536, 4), (40, 256, 8208, 8)])
def test_matches_plain(gpu, score, M, E, cols, K):
    print("route", score, M, E, cols, K, flush=True)
    bias, norm = (M + E) % 2 == 0, (M + K) % 2 == 0
    x, w, b = _inputs(M * E + cols + score, M, E, cols, bias)
    _check(_run(gpu, x, w, b, score, K, norm, 2.5), x, w, b, score, K, norm, 2.5, f"{score} {M}x{E}x{cols} top {K}")


@pytest.mark.parametrize("M", [1, 5, 40])
def test_ties_go_to_the_lower_index(gpu, M):
    """Equal experts (rows repeated far apart) are chosen in order of index."""
    x, w, _ = _inputs(3, M, 12, 528, False)
    w = w.repeat(11, 1)  # expert e + 12 i equals expert e
    for score in (0, 1, 2):
        ids, p = _run(gpu, x, w, None, score, 16, False, 1.0)
        best = route(x, w[:12], None, score, 2, False, 1.0)[0]
        assert torch.equal(ids[:, :11].long(), best[:, :1] + 12 * torch.arange(11)), score
        assert torch.equal(ids[:, 11:].long(), best[:, 1:] + 12 * torch.arange(5)), score
        assert (p[:, :11] == p[:, :1]).all()


def test_close_logits_are_told_apart(gpu):
    """Experts that differ by one bf16 step in one column of 4096 and a little in
    another: many logits differ by less than 2^-24 of their size, which sums in
    32 bits cannot order."""
    rng = np.random.default_rng(4)
    x = (normal(rng, 6, 4096).abs() + 0.5).bfloat16()
    base = (normal(rng, 4096).abs() + 0.5).bfloat16()
    w = base.repeat(64, 1)
    at = torch.from_numpy(rng.permutation(4096)[:64].copy())
    w[torch.arange(64), at] = (base[at].view(torch.int16) + 1).view(torch.bfloat16)
    w[:, 0] = 2.0 ** -20 * (1 + torch.arange(64)).bfloat16()  # makes every pair differ
    b = 1e-9 * torch.from_numpy(rng.permutation(64).astype(np.float32))
    for score, bias in ((0, None), (2, b)):
        _check(_run(gpu, x, w, bias, score, 8, True, 1.0), x, w, bias, score, 8, True, 1.0, "close logits")


@pytest.mark.parametrize("left", [0, 1, 3, 8])
@pytest.mark.parametrize("M", [2, 40])
def test_masked_experts(gpu, left, M):
    """A bias of -inf takes an expert out; what is missing is -1 with weight 0.
    f32's lowest value is a number: such experts still come last."""
    x, w, _ = _inputs(6, M, 90, 528, False)
    keep = torch.tensor([5, 17, 40, 41, 63, 64, 70, 89])[:left]
    bias = torch.full((90,), -float("inf"))
    bias[keep] = torch.linspace(0, 0.2, left)
    for norm in (True, False):
        _check(_run(gpu, x, w, bias, 1, 6, norm, 1.0), x, w, bias, 1, 6, norm, 1.0, f"{left} left")
    bias[80:84] = torch.finfo(torch.float32).min
    bias[keep] = 0.0
    ids, _ = _run(gpu, x, w, bias, 1, 6, False, 1.0)
    want = min(left, 6)
    assert all(set(r[:want].tolist()) <= set(keep.tolist()) for r in ids)
    if left < 6:  # s + lowest rounds to the same 64-bit number or orders by s: in any case among the four
        assert all(set(r[want:min(want + 4, 6)].tolist()) <= {80, 81, 82, 83} for r in ids)


def test_values_that_are_not_finite_still_give_usable_ids(gpu):
    x, w, _ = _inputs(8, 20, 70, 272, False)
    x[3, 5], x[4, 6], w[9, 7] = float("nan"), float("inf"), float("nan")
    for score in (0, 1, 2):
        ids, _ = _run(gpu, x, w, None, score, 8, True, 1.0)
        assert ((ids >= -1) & (ids < 70)).all()
        for row in ids.tolist():
            real = [i for i in row if i >= 0]
            assert len(set(real)) == len(real)
        if score:  # one bad expert does not take the others with it
            ok = [m for m in range(20) if m not in (3, 4)]
            assert (ids[ok] >= 0).all() and (ids[ok] != 9).all()


def test_large_logits(gpu):
    """Logits near +-1e5: softmax and softplus stay finite, sums of 0 leave weights of 0."""
    x, w, _ = _inputs(10, 3, 30, 272, False)
    w = (w.float() * 3e4).bfloat16()
    for score in (0, 1, 2):
        ids, p = _run(gpu, x, w, None, score, 4, True, 1.0)
        assert torch.isfinite(p).all() and ((ids >= 0) & (ids < 30)).all()
    assert torch.equal(_run(gpu, x, w, None, 2, 4, True, 1.0)[0].long(), route(x, w, None, 2, 4, True, 1.0)[0])
    low = torch.full((1, 16), -1e4).bfloat16()
    ids, p = _run(gpu, low, torch.ones(4, 16).bfloat16(), None, 1, 2, True, 1.0)
    assert ids.tolist() == [[0, 1]] and p.tolist() == [[0.0, 0.0]]


def test_tokens_do_not_depend_on_the_panel(gpu):
    for E in (48, 256):
        x, w, b = _inputs(12, 300, E, 1040, True)
        ids, p = _run(gpu, x, w, b, 2, 6, True, 1.5)
        for n in (1, 7, 16, 17, 64):
            i1, p1 = _run(gpu, x[:n], w, b, 2, 6, True, 1.5)
            assert torch.equal(i1, ids[:n]) and torch.equal(p1, p[:n]), (E, n)


@pytest.mark.parametrize("M,E,cols", [(200, 250, 336), (515, 250, 1552), (990, 250, 336), (2030, 250, 336), (4100, 250, 1040)])
def test_large_panels(gpu, M, E, cols):
    """1, 2, 4 and 8 tiles a workgroup, with rows and experts missing from the
    last, and the same tokens alone."""
    x, w, b = _inputs(M + cols, M, E, cols, True)
    ids, p = _run(gpu, x, w, b, 1, 6, True, 1.5)
    want, q, _ = route(x, w, b, 1, 6, True, 1.5)
    v = (torch.sigmoid(x.double() @ w.double().t()) + b.double()).sort(dim=1, descending=True).values
    clear = ((v[:, :6] - v[:, 1:7]) > 1e-11).all(1)  # of so many choices some may tie
    assert clear.float().mean() > 0.999 and torch.equal(ids[clear].long(), want[clear])
    assert ((p.double() - q).abs() <= (U + 1e-12) * q.abs() + 2.0 ** -150)[clear].all()
    for at in (0, M // 2, M - 1):
        i1, p1 = _run(gpu, x[at:at + 1], w, b, 1, 6, True, 1.5)
        assert torch.equal(i1, ids[at:at + 1]) and torch.equal(p1, p[at:at + 1]), at


def test_largest_panel(gpu):
    x, w, b = _inputs(14, 65536, 9, 16, True)
    ids, p = _run(gpu, x, w, b, 1, 2, True, 1.0)
    want, q, _ = route(x, w, b, 1, 2, True, 1.0)
    # 16-column logits of so many tokens may tie; those that do not have to agree
    s = torch.sigmoid(x.double() @ w.double().t()) + b.double()
    v = s.sort(dim=1, descending=True).values
    clear = ((v[:, :2] - v[:, 1:3]) > 1e-11).all(1)
    assert clear.float().mean() > 0.999
    assert torch.equal(ids[clear].long(), want[clear])


@pytest.mark.parametrize("M", [1, 20, 2100])
def test_small_softplus_scores_keep_their_order(gpu, M):
    """sqrt(log(1 + exp(l))) is exp(l / 2) for l far below 0, in 64 bits a
    normal number down to l = -1416, though exp(l) is none below -708."""
    l = torch.tensor([-760.0, -748.0, -800.0, -752.0, -1408.0, -744.0, -712.0, -1440.0, -4992.0] + [-6016.0] * 7)
    w = torch.zeros(16, 16).bfloat16()
    w[:, 3] = l.bfloat16()  # exact
    assert torch.equal(w[:, 3].float(), l)
    x = torch.zeros(M, 16).bfloat16()
    x[:, 3] = 1.0
    ids, p = _run(gpu, x, w, None, 2, 7, True, 2.0)
    assert (ids == torch.tensor([6, 5, 1, 3, 0, 2, 4])).all()
    want = torch.exp((l[[6, 5, 1, 3, 0, 2, 4]].double() + 712) / 2)
    want = 2.0 * want / want.sum()
    assert ((p.double() - want).abs() <= (U + 1e-12) * want + 2.0 ** -150).all()
    x[:, 3] = 2.0 ** -1  # -372 .. -3008: no underflow before -1416
    ids, p = _run(gpu, x, w, None, 2, 4, True, 2.0)
    assert (ids == torch.tensor([6, 5, 1, 3])).all()
