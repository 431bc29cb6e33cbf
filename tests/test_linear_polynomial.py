"""The polynomial q(u) = (1 - e^-u) / u in the linear scan, with the coefficients as the kernel holds them."""
import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_chunked_delta_gb300", "csrc", "gdr_linear.cu")


def coefficients():
    with open(SOURCE) as f:
        found = re.search(r"const float poly\[4\] = \{([^}]*)\}", f.read()).group(1)
    c = [np.float32(v.strip().rstrip("f")) for v in found.split(",")]
    assert len(c) == 4
    return c


def test_coefficients_are_those_of_the_function():
    """In 64 bits: off by at most 3.1e-9 of it on [0, 1/4]."""
    u = np.linspace(0, 0.25, 200001)[1:]
    q = np.zeros_like(u)
    for c in reversed(coefficients()):
        q = q * u + float(c)
    q = q * u + 1
    assert np.abs(q * u / -np.expm1(-u) - 1).max() <= 3.1e-9


def test_evaluation_in_32_bits():
    """As the kernel evaluates it, each step a fused multiply-add.  w = u q is off by the last step's rounding (2^-24 of q >= 0.88), the
    product's (2^-24), and at most an eighth of the steps' before (u |c| <= 1/8): 2^-22.5 of it with room; a = 1 - w by half a step of
    numbers below 1 (2^-25) and w's error, which have no mean; 1 - a^2 = w + w a by 2^-22 of it."""
    u = np.random.default_rng(5).uniform(0, 0.25, 400000).astype(np.float32)
    c = coefficients()
    fma = lambda x, y, z: (x.astype(np.float64) * y.astype(np.float64) + z).astype(np.float32)  # noqa: E731  (products of fp32 are exact in 64 bits)
    q = fma(u, np.full_like(u, c[3]), np.float64(c[2]))
    for k in (c[1], c[0], np.float32(1)):
        q = fma(u, q, np.float64(k))
    w = u * q
    a = np.float32(1) - w
    rest = fma(w, a, w.astype(np.float64))
    exact = -np.expm1(-u.astype(np.float64))
    assert np.abs(w / exact - 1).max() <= 2.0 ** -22.5
    assert np.abs(a - (1 - exact)).max() <= 2.0 ** -25 + 0.25 * 2.0 ** -22.5
    assert np.abs(rest / -np.expm1(-2 * u.astype(np.float64)) - 1).max() <= 2.0 ** -22
    assert w.dtype == a.dtype == rest.dtype == np.float32
    # errors of half a step (2^-25 / sqrt(3) rms) and w's, over 400000 arguments: a mean below five times what they leave by chance
    assert abs((a / (1 - exact) - 1).mean()) <= 5 * (2.0 ** -25 + 0.25 * 2.0 ** -22.5) / np.sqrt(len(u)) + 3.1e-9 * 0.125
