"""NaN through the backward pass's FMA-pipe 2^x: its float32 steps replayed in
numpy (the reduction to n + f, the polynomial times 2^n), with the constants of
the CUDA source, which does not add n into the polynomial's bits."""
import numpy as np
import pytest

from test_exp2_floor_poly import SRC, coeffs, replay

SHIFT = np.float32(12582912.0)


def steps(x, degree):
    x = x.astype(np.float32)
    x = np.where(np.isnan(x), x, np.maximum(x, np.float32(-127.0)))
    # x + shift rounded down: exact in 64 bits, then to the float32 below.
    wide = np.floor(x.astype(np.float64)) + float(SHIFT)
    t = wide.astype(np.float32)
    n = t - SHIFT
    f = (x - n).astype(np.float32)
    c = coeffs(degree)
    p = np.full_like(f, c[degree])
    for a in c[-2:0:-1]:
        p = (p.astype(np.float64) * f + a).astype(np.float32)
    # A NaN made by an addition has all exponent and mantissa bits set.
    bits = np.where(np.isnan(t), 0x7fffffff, t.view(np.int32).astype(np.int64))
    two_n = (((bits << 23) + 0x3f800000) & 0xffffffff).astype(np.uint32).view(np.float32)
    with np.errstate(invalid="ignore"):
        return (p.astype(np.float64) * (f * two_n) + two_n).astype(np.float32)


@pytest.mark.parametrize("degree", [4, 5])
def test_nan_stays_nan(degree):
    got = steps(np.array([np.nan, 0.0, -3.5], np.float32), degree)
    assert np.isnan(got[0]) and np.isfinite(got[1:]).all()


@pytest.mark.parametrize("degree", [4, 5])
def test_same_values_as_with_the_exponent_added(degree):
    x = np.linspace(-125.9, 20.0, 100_001).astype(np.float32)
    assert np.array_equal(steps(x, degree), replay(x, degree))
    dead = steps(np.array([-np.inf, -1e9, -127.0, -126.5], np.float32), degree)
    assert (dead == 0).all() and not np.signbit(dead).any()


def test_source_multiplies():
    src = open(SRC).read()
    body = src[src.index("void ex2_floor_x2"):src.index("void bulk_load")]
    assert "mul_x2(fa, fb, na, nb)" in body and "__float_as_int(pa)" not in body
