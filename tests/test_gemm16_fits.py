"""The polynomials of GELU and of its slope against 64 bits, on the CPU: the coefficients are read from the kernels' source and
evaluated step by step in FP32, each operation rounded once.  (The GPU's exponential and reciprocal are a unit or two
off; here they are rounded to nearest, and the reciprocal also taken a unit to either side.)  The bounds are those
that the source's comments give."""

import os
import re

import numpy as np
import pytest
import torch

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "dense_fp32_gemm_sm_gb300", "csrc")
f32, f64 = np.float32, np.float64


def coefficients(name):
    with open(os.path.join(CSRC, "gemm16_device.cuh")) as f:
        text = re.search(r"constexpr float %s\[\] = \{(.*?)\};" % name, f.read(), flags=re.S).group(1)
    return [f32(x.strip().rstrip("f")) for x in text.split(",")]


def fma(a, b, c):
    return (np.asarray(a, f64) * np.asarray(b, f64) + np.asarray(c, f64)).astype(f32)


def mul(a, b):
    return (np.asarray(a, f64) * np.asarray(b, f64)).astype(f32)


def polynomial(c, x):
    h = np.full_like(x, c[0])
    for k in c[1:]:
        h = fma(h, x, k)
    return h


def special(name, x):
    return getattr(torch.special, name)(torch.from_numpy(np.asarray(x, f64))).numpy()


def bell(x):
    return np.exp2(mul(mul(f32(-0.721347520444482), x), x).astype(f64)).astype(f32)


def slope(z):
    z = z.astype(f64)
    return special("ndtr", z) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)


def test_distribution():
    """Phi = 1/2 + c P(2 c^2 / 5.5^2 - 1), held in 0 .. 1."""
    c = np.linspace(-5.5, 5.5, 200001).astype(f32)
    p = polynomial(coefficients("CDF"), fma(mul(c, c), f32(2 / 5.5**2), f32(-1)))
    got = np.clip(fma(c, p, f32(0.5)), 0, 1)
    off = np.abs(got - special("ndtr", c))
    assert off.max() < 9.1e-8 and off.mean() < 1.65e-8
    assert got[0] == 0 and got[-1] == 1  # where the arguments beyond are held
    assert abs(sum(map(abs, map(float, coefficients("CDF")))) - 0.4) < 0.005


def test_tail():
    """Phi(-a) = exp(-a^2/2) g(a), g = t times the polynomial in t = 1 / (1 + 0.31 a)."""
    a = np.linspace(0, 20, 200001).astype(f32)
    g, tail = 0.5 * special("erfcx", a.astype(f64) / np.sqrt(2)), coefficients("TAIL")
    t = 1 / (1 + f64(f32(0.31)) * a.astype(f64))
    h = np.zeros_like(t)
    for k in tail:
        h = h * t + f64(k)
    assert np.abs(h * t / g - 1).max() < 1.9e-7


@pytest.mark.parametrize("unit,bound", [(0, 5e-7), (-1, 6.5e-7), (1, 6.5e-7)])
def test_tail_as_evaluated(unit, bound):
    a = np.linspace(0, 20, 200001).astype(f32)
    t = (1 / fma(a, f32(0.31), f32(1)).astype(f64)).astype(f32)
    t = np.nextafter(t, f32(2 * unit)) if unit else t
    g, h = 0.5 * special("erfcx", a.astype(f64) / np.sqrt(2)), polynomial(coefficients("TAIL"), t)
    assert np.abs(mul(h, t) / g - 1).max() < bound
    s = mul(bell(a), fma(h, t, mul(f32(-0.398942280401433), a)))
    for sign in (1, -1):
        got = (f32(0.5) + f32(sign) * (f32(0.5) - s)).astype(f32)
        assert np.abs(got - slope(sign * a)).max() < 3.3e-7


def test_slope():
    """Phi's 9.1e-8, half a unit of a sum up to 1.13 (6e-8), and two units or so of z phi, 0.25 at most (3e-8)."""
    z = np.linspace(-12, 12, 200001).astype(f32)
    c = np.clip(z, f32(-5.5), f32(5.5))
    p = polynomial(coefficients("CDF"), fma(mul(c, c), f32(2 / 5.5**2), f32(-1)))
    got = fma(c, mul(f32(0.398942280401433), bell(z)), np.clip(fma(c, p, f32(0.5)), 0, 1))
    assert np.abs(got - slope(z)).max() < 1.8e-7
    assert (np.abs(got)[z < -10] < 1e-20).all() and (got[z > 6] == 1).all()


def test_slope_by_definition():
    z = np.linspace(-20, 20, 200001).astype(f32)
    cdf = mul(f32(0.5), special("erfc", mul(-z, f32(0.707106781186548))).astype(f32))
    e = np.exp(mul(mul(f32(-0.5), z), z).astype(f64)).astype(f32)
    got = (cdf + mul(mul(z, e), f32(0.398942280401433))).astype(f32)
    assert np.abs(got - slope(z)).max() < 1.3e-7


def test_silu_slope():
    """s (1 + z (1 - s)), in the fast order and in the definition's: (1 + |z|) 1.1e-7."""
    z = np.linspace(-80, 80, 200001).astype(f32)
    s64 = 1 / (1 + np.exp(-z.astype(f64)))
    want = s64 * (1 + z * (1 - s64))
    fast = (1 / (f32(1) + np.exp2(mul(f32(-1.44269504088896), z).astype(f64)).astype(f32)).astype(f64)).astype(f32)
    by_definition = (1 / (f32(1) + np.exp(-z.astype(f64)).astype(f32)).astype(f64)).astype(f32)
    for got in (mul(fast, fma(z, f32(1) - fast, f32(1))),
                mul(by_definition, (f32(1) + mul(z, f32(1) - by_definition)).astype(f32))):
        assert (np.abs(got - want) / (1 + np.abs(z.astype(f64)))).max() < 1.1e-7
