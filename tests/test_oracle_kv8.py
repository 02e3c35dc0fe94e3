"""The 8-bit cache's oracle against torch's e4m3 conversion and its own definition (CPU)."""

import numpy as np
import pytest
import torch

from oracle import kv8 as K


def test_codes_are_torchs():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(K.decode(codes), want)


def test_rounding_is_torchs():
    g = np.random.default_rng(0)
    x = np.concatenate([np.linspace(-2 ** -5, 2 ** -5, 4097), g.standard_normal(20000) * 100, np.linspace(-448, 448, 3585)])
    x = np.clip(x, -448, 448).astype(np.float32)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(K.encode(x), want)
    np.testing.assert_array_equal(K.encode([np.nan, np.inf, -np.inf]), [127] * 3)


@pytest.mark.parametrize("amax,e", [(448, 0), (np.nextafter(448, 500), 1), (224, -1), (0, -110), (1e-45, -110), (1, -8),
                                    (1.75, -8), (1.7500001, -7), (3.4e38, 120), (2.0 ** -102 * 1.75, -110)])
def test_least_exponent(amax, e):
    assert K.least_exponent(float(amax)) == e


def test_scales_grow_and_begin_anew():
    codes, scales = np.zeros((1, 16, 1, 1), np.uint8), np.zeros((1, 1, 1), np.uint8)
    K.write(codes, scales, 16, np.full((1, 1, 1), 3.0), 0, [0])
    assert scales[0, 0, 0] == 127 - 7 and K.decode(codes[0, 0, 0, 0]) == 3 * 128
    K.write(codes, scales, 16, np.full((1, 1, 1), 1000.0), 1, [0])
    assert scales[0, 0, 0] == 127 + 2 and K.decode(codes[0, 0, 0, 0]) == 0.75
    np.testing.assert_array_equal(K.read(codes, scales, 16, 0, 2, [0])[:, 0, 0], [3, 1024])
    K.write(codes, scales, 16, np.full((1, 1, 1), 1e-3), 2, [0])
    assert scales[0, 0, 0] == 127 + 2
    K.write(codes, scales, 16, np.full((1, 1, 1), 1e-3), 0, [0])
    assert scales[0, 0, 0] == 127 - 18


def test_visible():
    assert K.visible(2, 3, 0, 0).tolist() == [[1, 1, 1, 1, 0], [1] * 5]
    assert K.visible(2, 3, 2, 1).tolist() == [[1, 0, 1, 1, 0], [1, 0, 0, 1, 1]]


@pytest.mark.parametrize("old", [0, 3])
def test_largest_values_stay_finite(old):
    """Every finite float32 is written as something finite in float32 and within e4m3's half step of it."""
    codes, scales = np.zeros((1, 16, 1, 8), np.uint8), np.zeros((1, 1, 1), np.uint8)
    K.write(codes, scales, 16, np.ones((max(old, 1), 1, 8)), 0, [0])
    top = float(np.finfo(np.float32).max)
    x = np.array([top, -top, 3.2965e38, 3.2962e38, 3.19e38, 3.1e38, np.inf, np.nan]).reshape(1, 1, 8)
    K.write(codes, scales, 16, x, old, [0])
    y = K.read(codes, scales, 16, old, old + 1, [0])[0, 0]
    assert scales[0, 0, 0] == 247 and np.isfinite(y[:6].astype(np.float32)).all() and np.isnan(y[6:]).all()
    assert (np.abs(y[:6] - x[0, 0, :6]) <= 2.0 ** -4 * np.abs(x[0, 0, :6])).all()
    assert y[0] == 240 * 2.0 ** 120 == -y[1]
