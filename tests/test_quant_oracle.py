"""The fp64 reference of the 8-bit caches, pinned on the CPU."""
import numpy as np
import torch

from oracle import serving_oracle as so


def test_the_values_of_e4m3():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(so.e4m3_values(), want)
    assert so.e4m3_values()[0x7e] == 448 and so.e4m3_values()[1] == 2.0 ** -9 and np.isnan(so.e4m3_values()[0xff])


def test_a_row_by_hand():
    # largest 896: scale 2. 3 / 2 is a value; 2 * 1.0625 is half way between 1 and 1.125: to the even code, 1
    codes, scale = so.quantise(np.array([-896.0, 3.0, 2.125, 2.375, 0.0, 2.0 ** -9, 1.5 * 2.0 ** -8]))
    assert scale == 2
    got = so.dequantise(codes, scale)
    np.testing.assert_array_equal(got, [-896, 3, 2, 2.5, 0, 0, 2 * 2.0 ** -8])


def test_codes_are_the_nearest():
    g = np.random.default_rng(1)
    y = g.standard_normal((50, 64)) * np.exp(3 * g.standard_normal((50, 64)))
    codes, scale = so.quantise(y)
    z = y / scale[:, None]
    off = np.abs(so.e4m3_values()[codes] - z)
    best = np.abs(so.e4m3_values()[None, None, :127] * np.sign(z)[..., None] - z[..., None]).min(axis=-1)
    np.testing.assert_array_equal(off, best)
    assert (off <= np.maximum(2.0 ** -4 * np.abs(z), 2.0 ** -10)).all()
    # torch's conversion rounds the same way
    t = torch.from_numpy(z).to(torch.float32)
    np.testing.assert_array_equal(codes, t.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_empty_and_small_rows():
    codes, scale = so.quantise(np.zeros((2, 4)))
    assert not codes.any() and (scale == 2.0 ** -126).all()
    codes, scale = so.quantise(np.array([2.0 ** -130, -2.0 ** -126]))
    np.testing.assert_array_equal(so.dequantise(codes, scale), [2.0 ** -130, -2.0 ** -126])
