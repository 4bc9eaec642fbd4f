"""Pins of the microscaled 4-bit floating point oracle (oracle/fp4.py): none
restates its formulas."""

import numpy as np
import pytest
import torch

from oracle import fp4


def test_e2m1_grid_and_ties():
    grid = fp4.MAGNITUDES
    assert fp4.e2m1_codes(grid).tolist() == list(range(8))
    assert fp4.e2m1_codes(-grid).tolist() == list(range(8, 16))
    # midpoints go to the even code; just beside them to the nearer one
    mid = (grid[1:] + grid[:-1]) / 2
    assert fp4.e2m1_codes(mid).tolist() == [0, 2, 2, 4, 4, 6, 6]
    assert fp4.e2m1_codes(mid * (1 + 1e-12)).tolist() == [1, 2, 3, 4, 5, 6, 7]
    assert fp4.e2m1_codes(mid * (1 - 1e-12)).tolist() == [0, 1, 2, 3, 4, 5, 6]
    assert fp4.e2m1_codes(np.array([7.0, 1e30, -9.0])).tolist() == [7, 7, 15]


def test_e4m3_against_torch():
    v = fp4.e4m3_values()
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, t)
    x = np.concatenate([np.linspace(0, 448, 5001), (v[1:] + v[:-1]) / 2, np.exp(np.linspace(-9, 6.1, 3000))])
    x = x.astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(fp4.e4m3_codes(x), want)
    assert fp4.e4m3_codes(np.array([449.0, 1e9])).tolist() == [126, 126]


def test_mxfp4_hand_example():
    # max 5.0 = 1.25 * 2^2: scale 2^(2 - 2) = 1, so values are their own codes
    x = np.zeros((1, 32), np.float32)
    x[0, :6] = [5.0, -0.5, 3.0, 2.5, 0.3, -4.0]
    codes, s, r = fp4.quantize(x, "mxfp4")
    assert s.tolist() == [[127]] and r is None
    assert codes[0, :6].tolist() == [6, 9, 5, 4, 1, 14]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_power_of_two_scaling(fmt):
    x = np.random.default_rng(3).standard_normal((5, 96)).astype(np.float32)
    c, s, r = fp4.quantize(x, fmt)
    c2, s2, r2 = fp4.quantize(x * 1024, fmt)
    assert np.array_equal(c, c2)
    if fmt == "mxfp4":
        assert np.array_equal(s.astype(int) + 10, s2.astype(int))
    else:
        assert np.array_equal(s, s2) and np.array_equal(r * 1024, r2)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_values_near_the_input(fmt):
    # E2M1's widest relative gap is 4..6: half of it, 1, over the scaled
    # magnitude; mxfp4 also saturates values of up to 8 scales at 6
    x = np.random.default_rng(4).standard_normal((20, 320)).astype(np.float32)
    v = fp4.dequantize(*fp4.quantize(x, fmt), fmt)
    B = fp4.BLOCK[fmt]
    top = np.repeat(np.abs(x).reshape(20, -1, B).max(-1), B, axis=1)
    worst = 2 / 8 if fmt == "mxfp4" else 1 / 6 + 2**-3
    assert (np.abs(v - x) <= worst * top).all()
    assert np.corrcoef(v.ravel(), x.ravel())[0, 1] > 0.98


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_zeros_infinities_nan(fmt):
    x = np.ones((4, 64), np.float32)
    x[0] = 0
    x[1, 40], x[2, 3] = np.inf, np.nan
    v = fp4.dequantize(*fp4.quantize(x, fmt), fmt)
    assert (v[0] == 0).all() and (v[3] == v[3][0]).all() and abs(v[3, 0] - 1) < 0.1
    if fmt == "mxfp4":  # the block alone
        assert np.isnan(v[1, 32:]).all() and np.isfinite(v[1, :32]).all()
        assert np.isnan(v[2, :32]).all() and np.isfinite(v[2, 32:]).all()
    else:  # the row
        assert np.isnan(v[1:3]).all()


def test_pack_bytes():
    codes = np.arange(34, dtype=np.uint8)[None] % 16
    scales = np.array([[1, 2]], np.uint8)
    c, s = fp4.pack(codes, scales, "mxfp4")
    assert c.shape == (1, 32) and s.shape == (1, 16)
    assert c[0, :2].tolist() == [0x10, 0x32] and c[0, 16] == 0x10 and not c[0, 17:].any()
    assert s[0, :2].tolist() == [1, 2] and not s[0, 2:].any()
