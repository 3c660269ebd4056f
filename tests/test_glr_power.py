"""2^l and 2^l - 1 of the gated linear recurrence's decay, on the CPU: the
polynomial with the coefficients that the kernel source holds, and the kernel's
fp32 steps after it.

Bounds: 2^f - 1 = f p(f) in fp32 on top of the polynomial's own 2.2e-8 carries
the rounding of the last sum and of the product by f (u = 2^-24 each, relative)
and what earlier steps leave, each scaled by |f| <= 1/2 and by its share of the
sum (0.24 / 0.69 and less): below u.  So q is good to 3 u + 2.2e-8 <= 3.4 u.
2^n + 2^n q with |q| <= 0.42 adds a rounding: 2^l to (0.42 / 0.70 * 3.4 + 1) u <=
3.1 u (2^f is 0.70 at least where q = -0.30, and 1.41 where q is 0.42).
2^l - 1 = (2^n - 1) + 2^n q: q itself at n = 0; else the first sum is at least as
large as the result's 0.29 and exact to n = -24 and within u beyond: 3.1 u of
2^l <= 0.71 is at most 3.1 * 0.71 / 0.29 u, and two roundings: 10 u.
"""
import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bidirectional_mamba_denoiser_b200",
                      "csrc", "glr.cuh")
U = 2.0 ** -24


def _coefficients():
    with open(SOURCE) as f:
        body = re.search(r"float2 glr_ex2m1\(.*?\n}\n", f.read(), re.S).group(0)
    c = [float(v) for v in re.findall(r"(\d\.\d{6,})f", body)]
    assert len(c) == 6
    assert all(float(np.float32(v)) == v for v in c), "coefficients that fp32 does not hold"
    return c


def test_polynomial_is_as_good_as_its_comment_says():
    f = np.linspace(-0.5, 0.5, 2000001)
    f = f[np.abs(f) > 1e-9]
    p = np.zeros_like(f)
    for c in _coefficients():
        p = p * f + c
    want = np.expm1(f * np.log(2.0)) / f
    with open(SOURCE) as src:
        stated = float(re.search(r"relative error by Remez exchange,[^)]*?([\d.]+e-\d+)", src.read()).group(1))
    worst = np.max(np.abs(p / want - 1))
    assert worst <= stated <= 2.2e-8


def _power(l):
    """The kernel's steps with a rounding to fp32 after each (a product and sum in one, as its fma has)."""
    f32, wide = np.float32, np.float64
    fma = lambda a, b, c: (a.astype(wide) * b + wide(c) if np.isscalar(c) else a.astype(wide) * b + c.astype(wide)).astype(f32)  # noqa: E731
    l = np.maximum(l.astype(f32), f32(-127))
    m = l + f32(12582912)
    f = l - (m - f32(12582912))
    c = _coefficients()
    q = fma(f, f32(c[0]), c[1])
    for v in c[2:]:
        q = fma(f, q, v)
    q = (f * q).astype(f32)
    s = ((m.view(np.uint32) << np.uint32(23)) + np.uint32(0x3F800000)).view(f32)
    return fma(q, s, s), fma(q, s, s - f32(1))


def test_power_and_power_less_one_are_relatively_accurate():
    rng = np.random.default_rng(0)
    l = np.concatenate([-np.exp(rng.uniform(np.log(1e-30), np.log(125.9), 400000)), -rng.uniform(0, 3, 400000),
                        [0.0, -0.5, -1.0, -1.5, -125.5]]).astype(np.float32)
    pow_, less = _power(l)
    want = np.exp2(l.astype(np.float64))
    assert np.all(np.abs(pow_ - want) <= 3.1 * U * want)
    want = np.expm1(l.astype(np.float64) * np.log(2.0))
    assert np.all(np.abs(less - want) <= 10 * U * np.abs(want))


def test_power_ends_in_zero():
    pow_, less = _power(np.array([-126.75, -127.0, -1e4, -3.4e38, -np.inf], np.float32))
    assert np.all(pow_ == 0) and np.all(less == -1)
    pow_, less = _power(np.zeros(1, np.float32))
    assert pow_[0] == 1 and less[0] == 0
