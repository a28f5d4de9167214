"""The definitions that the softmax layers' GPU tests compare with, against each other,
against values worked by hand and against differences (CPU)."""
import math

import torch

from layer_oracle import rotary64
from softmax_oracle import (CODES, cache_values, fp4_group, fp4_nearest, fp4_values, norm_rotary64, rotary_leaf)


def test_scales_and_codes_by_hand():
    # largest 6: the exponent of 6 is 2, less two: units of 1
    codes, byte = fp4_group([6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -5.0, 5.5, -0.0] + [0.0] * 21)
    assert byte == 127 and codes[:11] == [7, 6, 6, 4, 4, 2, 2, 0, 14, 7, 8]
    # 7 is cut to 6; above it the unit doubles
    assert fp4_group([7.0] + [0.0] * 31) == ([7] + [0] * 31, 127)
    codes, byte = fp4_group([7.001] + [1.0] * 31)
    assert byte == 128 and codes[0] == 6 and codes[1] == 1  # 3.5005 and 1/2 units
    assert fp4_group([0.0] * 32) == ([0] * 32, 1)
    assert fp4_group([2.0 ** 127] + [0.0] * 31)[1] == 252 and fp4_group([1e300] + [0.0] * 31) == ([7] + [0] * 31, 252)
    for bad in (math.inf, -math.inf, math.nan):
        assert fp4_group([1.0, bad] + [0.0] * 30) == (None, 255)


def test_steps_equal_search():
    g = torch.Generator().manual_seed(1)
    x = torch.randn(200, 64, generator=g, dtype=torch.float64) * torch.exp2(torch.randint(-140, 126, (200, 1), generator=g))
    x[3, 5], x[4, 40], x[5] = math.nan, -math.inf, 0.0
    x[6] = torch.tensor(CODES).repeat(8) * 2.0 ** -3 + 2.0 ** -5  # halfway and near it
    a, b = fp4_values(x), fp4_nearest(x)
    assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(), b.nan_to_num())


def test_values_of_codes():
    codes = torch.zeros(1, 1, 2, 16, dtype=torch.uint8)
    scales = torch.full((1, 1, 1, 2), 127, dtype=torch.uint8)
    codes[0, 0, 0, 0], codes[0, 0, 1, 15] = 0x97, 0x2F
    scales[0, 0, 0, 1] = 130
    v = cache_values(codes, scales)
    assert v[0, 0, 0, 0] == 6 and v[0, 0, 0, 1] == -0.5 and v[0, 0, 1, 30] == -48 and v[0, 0, 1, 31] == 8


def test_no_value_is_off_by_more_than_half_a_step():
    """Half a step of the codes next to it: 1/4 unit below 2, 1/2 below 4, 1 above."""
    g = torch.Generator().manual_seed(2)
    x = torch.randn(3000, 32, generator=g, dtype=torch.float64)
    v = fp4_nearest(x)
    for row, got in zip(x, v):
        _, byte = fp4_group(row.tolist())
        z = (row.abs() * 2.0 ** (127 - byte))
        half = torch.where(z < 2, 0.25, torch.where(z < 4, 0.5, 1.0))
        assert ((row - got).abs() * 2.0 ** (127 - byte) <= half).all()


def test_rotation_and_differences():
    g = torch.Generator().manual_seed(3)
    x = torch.randn(5, 2, 12, generator=g, dtype=torch.float64)
    w = 1 + 0.1 * torch.randn(12, generator=g, dtype=torch.float64)
    pos, freqs = torch.tensor([0, 1, 7, 100, 4000]), torch.tensor([1.0, 0.3, 0.01], dtype=torch.float64)
    for inter in (False, True):
        assert (rotary_leaf(x, pos, freqs, inter, 1.3) - rotary64(x, pos, freqs, inter, 1.3)).abs().max() < 1e-12
        f = lambda x, w: norm_rotary64(x, w, pos, freqs, inter, 1.3, 1e-6)  # noqa: E731
        assert torch.autograd.gradcheck(f, (x.clone().requires_grad_(), w.clone().requires_grad_()))
