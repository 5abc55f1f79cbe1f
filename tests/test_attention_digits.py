"""How closely attention over the cache holds q, step by step in fp32 as the kernel forms its digits (no GPU)."""
import numpy as np

f32 = np.float32
MOST = f32(8355711.0)


def held(x):
    """q as its three digits stand for it, relative to the row's largest."""
    big = np.abs(x).max(1, keepdims=True)
    scaled = np.clip(x * (MOST / big), -MOST, MOST)  # two roundings to fp32
    total = scaled.astype(np.float64) + 8421504.0
    digits = np.trunc(total.astype(f32)) - 8421504.0
    return digits / np.float64(MOST), x.astype(np.float64) / big


def test_query_digits_are_within_the_documented_bound():
    rng = np.random.default_rng(1)
    x = (rng.standard_normal((20000, 128)) * np.exp(rng.standard_normal((20000, 1)) * 5)).astype(f32)
    got, want = held(x)
    off = np.abs(got - want).max()
    assert 2.0 ** -23 < off < 2.0 ** -22  # closer than the stated 2^-22, not as close as 2^-23


def test_digits_of_weights_are_closer():
    """p * 8355711 + 8421504 is 2^23 or more: one rounding to an integer, by at most a half."""
    rng = np.random.default_rng(2)
    p = rng.random(1 << 18).astype(f32)
    total = (p.astype(np.float64) * np.float64(MOST) + 8421504.0).astype(f32)
    assert (total >= 2.0 ** 23).all() and (total == np.trunc(total)).all()
    assert np.abs((total.astype(np.float64) - 8421504.0) / np.float64(MOST) - p).max() <= 0.5 / np.float64(MOST) < 2.0 ** -23
