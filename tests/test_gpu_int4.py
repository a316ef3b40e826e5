"""GPU: int4_gemv against its plain form in 64 bits."""
import numpy as np
import pytest
import torch

from layer_plain import assert_within, int4, normal

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _case(seed, M, rows, cols, group, zeros=True):
    rng = np.random.default_rng(seed)
    codes = torch.from_numpy(rng.integers(0, 256, (rows, cols // 2), dtype=np.uint8))
    scales = (normal(rng, rows, cols // group) * 0.02).bfloat16()
    z = torch.from_numpy(rng.integers(0, 16, (rows, cols // group), dtype=np.uint8)) if zeros else None
    return codes, scales, z, group, normal(rng, M, cols).bfloat16()


def _run(gpu, codes, scales, zeros, group, x):
    y = torch.full((x.shape[0], codes.shape[0]), float("nan"), device=DEV)
    gpu.int4_gemv(codes.to(DEV), scales.to(DEV), None if zeros is None else zeros.to(DEV), group, x.to(DEV), y)
    torch.cuda.synchronize()
    return y


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("M,rows,cols", [(1, 1, 128), (1, 16, 256), (1, 4096, 4096), (2, 17, 384), (3, 1000, 640),
                                         (4, 130, 2176), (5, 2001, 2176), (8, 513, 1024), (9, 63, 4224), (16, 777, 1408),
                                         (16, 31, 8320), (1, 3, 65536), (16, 5, 65536), (7, 2048, 128)])
def test_matches_plain(gpu, group, M, rows, cols):
    print("int4", group, M, rows, cols, flush=True)
    for zeros in (True, False):
        c = _case(M * rows + cols + group, M, rows, cols, group, zeros)
        assert_within(_run(gpu, *c), *int4(*c), f"g{group} {M}x{rows}x{cols} zeros {zeros}")


@pytest.mark.parametrize("cols", [32, 96, 160, 2080, 4064])
def test_odd_numbers_of_groups(gpu, cols):
    for M in (1, 2, 5, 16):
        c = _case(cols + M, M, 45, cols, 32)
        assert_within(_run(gpu, *c), *int4(*c), f"M={M} cols={cols}")
    c = _case(cols, 3, 45, 2 * cols, 64)
    assert_within(_run(gpu, *c), *int4(*c), f"g64 cols={2 * cols}")


@pytest.mark.parametrize("M,rows,cols,group", [(3, 8209, 1056, 32), (16, 16400, 544, 32), (5, 70001, 352, 32), (1, 70001, 2080, 32),
                                               (9, 33000, 1088, 64), (16, 20000, 4160, 64), (12, 66003, 192, 64),
                                               (2, 66003, 4224, 64), (4, 9000, 8320, 128), (16, 66003, 128, 128),
                                               (16, 66000, 4096, 32), (8, 66000, 8192, 32), (16, 66003, 5248, 128)])
def test_many_rows(gpu, M, rows, cols, group):
    """Persistent workgroups: the first and last rows and 300 between them."""
    rng = np.random.default_rng(rows + cols)
    print("int4", group, M, rows, cols, flush=True)
    for zeros in (True, False):
        c = _case(rows + cols + M, M, rows, cols, group, zeros)
        y = _run(gpu, *c)
        at = torch.from_numpy(np.unique(np.r_[0:40, rng.integers(0, rows, 300), rows - 40:rows]))
        some = (c[0][at], c[1][at], None if c[2] is None else c[2][at], group, c[4])
        assert_within(y[:, at.to(DEV)], *int4(*some), f"g{group} {M}x{rows}x{cols} zeros {zeros}")
        assert torch.isfinite(y).all()


@pytest.mark.parametrize("rows,cols", [(100, 2080), (4096, 4096), (700, 8192), (12288, 1056), (70000, 352)])
def test_rows_do_not_depend_on_the_panel(gpu, rows, cols):
    codes, scales, z, g, x = _case(7, 16, rows, cols, 32)
    y = _run(gpu, codes, scales, z, g, x)
    for n in (1, 2, 3, 4, 5, 8, 11):
        assert torch.equal(_run(gpu, codes, scales, z, g, x[16 - n:]), y[16 - n:]), n


def test_every_code_and_zero_point(gpu):
    """One weight row for each zero point 0 .. 255, whose codes run through all
    sixteen values; x picks one column at a time, so every result is exact."""
    codes = torch.tensor([(2 * i % 16) | ((2 * i + 1) % 16) << 4 for i in range(16)], dtype=torch.uint8).repeat(256, 1)
    zeros = torch.arange(256, dtype=torch.uint8)[:, None]
    scales = torch.full((256, 1), 0.5).bfloat16()
    for c0 in (0, 16):
        x = torch.zeros(16, 32).bfloat16()
        x[torch.arange(16), c0 + torch.arange(16)] = 1
        y = _run(gpu, codes, scales, zeros, 32, x).cpu()
        q = torch.arange(32) % 16
        assert torch.equal(y, 0.5 * (q[c0:c0 + 16, None] - torch.arange(256)[None, :]).float())


def test_codes_at_the_zero_point_give_nothing(gpu):
    """Rows whose codes all equal the default zero point are zeros whatever x
    holds (padding rows), beside rows that are not."""
    codes, scales, _, g, x = _case(19, 6, 40, 1024, 64, zeros=False)
    codes[5] = codes[20] = 0x88
    y = _run(gpu, codes, scales, None, g, x)
    assert (y[:, 5] == 0).all() and (y[:, 20] == 0).all() and (y[:, 6] != 0).all()


@pytest.mark.parametrize("rows,cols,group", [(50, 640, 128), (50, 2080, 32), (70000, 352, 32), (70000, 640, 128)])
def test_values_that_are_not_finite_stay_in_their_row(gpu, rows, cols, group):
    codes, scales, z, g, x = _case(23, 5, rows, cols, group)
    clean = _run(gpu, codes, scales, z, g, x)
    x[1, 77], x[3, 300] = float("nan"), float("inf")
    y = _run(gpu, codes, scales, z, g, x)
    assert torch.equal(y[[0, 2, 4]], clean[[0, 2, 4]]) and y[1].isnan().all() and not torch.isfinite(y[3]).any()
    scales[7, 0] = float("nan")
    y = _run(gpu, codes, scales, z, g, x)
    assert y[:, 7].isnan().all() and torch.equal(y[0, :7], clean[0, :7]) and torch.equal(y[0, 8:], clean[0, 8:])


def test_scales_of_any_size(gpu):
    codes, scales, z, g, x = _case(29, 4, 60, 512, 32)
    scales[0::3] *= 2.0 ** -100
    scales[1::3] *= 2.0 ** 90
    assert_within(_run(gpu, codes, scales, z, g, x), *int4(codes, scales, z, g, x), "scales")


def test_outputs_next_door_are_left_alone(gpu):
    codes, scales, z, g, x = _case(31, 5, 100, 640, 64)
    y = torch.full((8, 100), 7.0, device=DEV)
    gpu.int4_gemv(codes.to(DEV), scales.to(DEV), z.to(DEV), g, x.to(DEV), y[1:6])
    torch.cuda.synchronize()
    assert (y[0] == 7).all() and (y[6:] == 7).all()
    assert torch.equal(y[1:6], _run(gpu, codes, scales, z, g, x))


def test_codes_past_32_bit_offsets(gpu):
    """163840 rows of 65536 columns: 5.4 GB of codes, more than 2^32 groups' worth of columns."""
    rows, cols, g = 163840, 65536, 128
    codes = torch.full((rows, cols // 2), 0x88, dtype=torch.uint8, device=DEV)
    scales = torch.ones((rows, cols // g), dtype=torch.bfloat16, device=DEV)
    c, s, _, _, x = _case(37, 2, 3, cols, g, zeros=False)
    at = torch.tensor([0, 140000, rows - 1], device=DEV)
    codes[at], scales[at] = c.to(DEV), s.to(DEV)
    y = torch.empty((2, rows), device=DEV)
    gpu.int4_gemv(codes, scales, None, g, x.to(DEV), y)
    torch.cuda.synchronize()
    assert_within(y[:, at], *int4(c, s, None, g, x), "rows past 2^32")
    y[:, at] = 0
    assert (y == 0).all()


@pytest.mark.parametrize("rows", [40, 9001])
@pytest.mark.parametrize("cols,group", [(128, 128), (384, 128), (416, 32), (320, 64), (2176, 128)])
def test_large_last_columns(gpu, rows, cols, group):
    """The last 8 columns near the end of the range, the same for few and for
    many rows: no column counts twice."""
    codes, scales, z, g, x = _case(41, 3, rows, cols, group)
    codes[:, -4:] = 0xFF
    x[:, -8:] = 2e36  # 15 sum |x| = 2.4e38
    c = codes, scales.abs(), z, g, x
    assert_within(_run(gpu, *c), *int4(*c), f"{rows}x{cols} in groups of {group}")


@pytest.mark.parametrize("rows,cols,group", [(33, 384, 128), (9001, 416, 32)])
def test_largest_values_beside_any_zero_point(gpu, rows, cols, group):
    """Zero points up to 255, with sums of max(15, z) |x| over a group just in f32's range."""
    codes, scales, z, g, x = _case(43, 3, rows, cols, group)
    z = torch.from_numpy(np.random.default_rng(43).integers(0, 256, z.shape, dtype=np.uint8))
    z[0] = 255
    x = (x.sign() * 1.2e38 / (128 * 255) * 2.5).bfloat16()  # 255 sum |x| is at most 3e38
    x[:, ::2] = x[:, ::2].abs()
    c = codes, (scales * 2.0 ** -20), z, g, x
    assert_within(_run(gpu, *c), *int4(*c), f"{rows}x{cols} in groups of {group}")


@pytest.mark.parametrize("rows,cols,group", [(130, 2176, 128), (4096, 4096, 64), (9001, 1056, 32)])
def test_activations_with_an_offset(gpu, rows, cols, group):
    """Activations that share an offset, and zero points far above the codes:
    both sums are large beside their difference, and the bound counts them."""
    codes, scales, z, g, x = _case(47, 4, rows, cols, group)
    z = z + 200
    c = codes, scales, z, g, (x.float() + 30).bfloat16()
    assert_within(_run(gpu, *c), *int4(*c), f"{rows}x{cols} in groups of {group}")
