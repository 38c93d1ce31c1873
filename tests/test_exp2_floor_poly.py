"""The backward pass's FMA-pipe 2^x (floor reduction, polynomial with p(0) = 1):
its float32 steps replayed in numpy with the constants of the CUDA source.

Tolerances: the fit's error (2.9e-6 and 8.3e-8, from gen_exp2_poly) plus one
rounding, 2^-24, of each of the degree's Horner steps and of the value."""
import os
import re

import numpy as np
import pytest

from masked_attention_fa_b200.csrc import gen_exp2_poly

SRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                   "masked_attention_fa_b200", "csrc", "fa_bwd_sm100.cu")


def coeffs(degree):
    src = open(SRC).read()
    body = src[src.index("constexpr float kC[2][6]"):]
    rows = re.findall(r"\{([^{}]*)\}", body[:body.index("};")])
    return [np.float32(x.strip().rstrip("f")) for x in rows[degree - 4].split(",")][:degree + 1]


def replay(x, degree):
    x = np.maximum(x.astype(np.float32), np.float32(-127.0))
    n = np.floor(x.astype(np.float64))
    f = (x - n.astype(np.float32)).astype(np.float32)
    c = coeffs(degree)
    p = np.full_like(f, c[degree])
    for a in c[-2::-1]:
        p = (p.astype(np.float64) * f + a).astype(np.float32)
    bits = p.view(np.int32) + (n.astype(np.int64) << 23).astype(np.int32)
    return bits.astype(np.int32).view(np.float32)


@pytest.mark.parametrize("degree", [4, 5])
def test_relative_error(degree):
    _, fit = gen_exp2_poly.remez_from_one(degree)
    x = np.linspace(-125.9, 20.0, 1_000_001).astype(np.float32)
    want = np.exp2(x.astype(np.float64))
    rel = np.abs(replay(x, degree) - want) / want
    assert rel.max() <= fit + (degree + 1) * 2.0 ** -24


@pytest.mark.parametrize("degree", [4, 5])
def test_source_holds_the_fit(degree):
    c, _ = gen_exp2_poly.remez_from_one(degree)
    assert [np.float32(x) for x in c] == coeffs(degree)


@pytest.mark.parametrize("degree", [4, 5])
def test_masked_is_zero(degree):
    got = replay(np.array([-np.inf, -1e9, -127.0], np.float32), degree)
    assert (got == 0).all() and not np.signbit(got).any()
