"""The reference of the 8-bit operators against other definitions of the same: torch's
own conversions for every code and for roundings, exact fractions for the scales."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import fp8_reference as F


@pytest.mark.parametrize("fmt", F.FORMATS)
def test_table_is_torchs(fmt):
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8)
    want = codes.view(F.FORMATS[fmt]).float().double().numpy()
    np.testing.assert_array_equal(F.table(fmt), want)


@pytest.mark.parametrize("fmt", F.FORMATS)
def test_encode_rounds_as_torch_does(fmt):
    gen = torch.Generator().manual_seed(0)
    top = F.LARGEST[fmt]
    v = torch.cat([torch.randn(20000, generator=gen) * 2.0 ** k for k in range(-16, 4, 3)])
    values = np.unique(np.abs(F.table(fmt)[np.isfinite(F.table(fmt))]))
    ties = torch.from_numpy((values[1:] + values[:-1]) / 2).float()
    v = torch.cat([v, ties, -ties, torch.tensor([0.0, -0.0, top, -top, float("nan")])])
    v = v[~(v.abs() > top)]
    want = v.to(F.FORMATS[fmt]).view(torch.uint8).numpy()
    got = F.encode(v.double().numpy(), fmt)
    nan = torch.isnan(v).numpy()
    np.testing.assert_array_equal(got[~nan], want[~nan])
    assert np.isnan(F.table(fmt)[got[nan]]).all()


@pytest.mark.parametrize("fmt", F.FORMATS)
def test_scale_is_the_least_power_of_two(fmt):
    top = Fraction(F.LARGEST[fmt])
    rng = np.random.default_rng(0)
    amax = np.concatenate([2.0 ** rng.uniform(-110, 127, 500), F.LARGEST[fmt] * 2.0 ** np.arange(-100.0, 100, 7)])
    amax = np.concatenate([amax, np.nextafter(amax, 0), np.nextafter(amax, np.inf)])
    for a in amax:
        s = Fraction(F.scale_of(float(a), fmt))
        assert Fraction(float(a)) <= top * s and Fraction(float(a)) > top * s / 2
    assert F.scale_of(0.0, fmt) == 1.0 and F.scale_of(2.0 ** -140, fmt) == 2.0 ** -126


def test_rounding_to_16_bits_is_one_rounding():
    rng = np.random.default_rng(1)
    v = rng.standard_normal(4000)
    half = 1 + 2.0 ** -8  # a tie of bfloat16 that binary32 would reach from above
    v = np.concatenate([v, [half + 2.0 ** -40, half, 1 + 3 * 2.0 ** -8 - 2.0 ** -40, 70000.0, np.inf, np.nan]])
    got = F.rounded(v, torch.bfloat16)
    assert float(got[4000]) == 1 + 2.0 ** -7 and float(got[4001]) == 1.0 and float(got[4002]) == 1 + 2.0 ** -7
    assert float(F.rounded(v, torch.float16)[4003]) == 65504.0
    assert torch.isinf(got[4004]) and torch.isnan(got[4005])
    assert (np.abs(got[:4000].double().numpy() - v[:4000]) <= np.abs(v[:4000]) * 2.0 ** -8).all()


@pytest.mark.parametrize("rows,cols,blocks,parts", [(5, 300, False, 1), (4, 260, False, 2), (300, 140, True, 1),
                                                    (258, 40, True, 2)])
def test_pack_and_values_are_inverse_on_codes(rows, cols, blocks, parts):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((rows, cols))
    codes, scales = F.pack(x, "e4m3", blocks, parts)
    v = F.values(codes, scales, "e4m3", blocks, parts)
    # half a unit of four digits, or half the smallest step
    step = np.repeat(scales, 1, 0).max() * 2.0 ** -10
    assert (np.abs(v - x) <= np.abs(x) * 2.0 ** -4 + step).all()
    again, scales2 = F.pack(v, "e4m3", blocks, parts)
    np.testing.assert_array_equal(F.values(again, scales2, "e4m3", blocks, parts), v)
