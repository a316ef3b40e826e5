"""CPU: that the bounds of the plain forms' tests tell the mistakes apart that
they are there for."""
import numpy as np

from layer_plain import U


def _pieces(h, n):
    """The sum of n bf16 pieces of f32 values, each the nearest to what is left."""
    left, total = h.astype(np.float32), np.zeros(h.shape)
    for _ in range(n):
        bits = left.view(np.uint32)
        piece = ((bits + 0x7FFF + (bits >> 16 & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
        total += piece
        left = (left - piece).astype(np.float32)
    return total


def test_the_bound_of_h_tells_two_pieces_from_three():
    """An expert layer's h = silu(g) u is an f32: three bf16 pieces hold it
    whole, two miss the 12 U that its tests allow.

    With |h| = f 2^e, 1 <= f < 2, one piece leaves a rest that is uniform in
    +-2^(e-8). In half of the cases it lies in its top binade, and the second
    piece leaves +-128 U 2^e of it, past 12 U |h| in 1 - 12 f / 128 of those; in
    a quarter +-64 U 2^e, then +-32 U 2^e, ...: for f around 1.4 in all 0.43 +
    0.18 + 0.06 + 0.01 = 0.68 of the values, of 4096 within 0.03 by four
    standard deviations. One piece leaves 12 U or less in 12 f / 2^16."""
    rng = np.random.default_rng(3)
    g, u = rng.standard_normal((2, 4096)) * 3
    for scale in (1.0, 2.0 ** -60, 2.0 ** 110):
        h = (g / (1 + np.exp(-g)) * u * scale).astype(np.float32)
        off = [np.abs(_pieces(h, n) - h.astype(np.float64)) / np.abs(h.astype(np.float64)) for n in (1, 2, 3)]
        assert (off[2] == 0).all()
        assert (off[1] > 12 * U).mean() > 0.64
        assert (off[0] > 12 * U).mean() > 0.99
