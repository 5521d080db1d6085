"""The error bound by which the large 8-bit write decides whether its fp32 rotation can be trusted, on the CPU: the
kernel's operations, each rounded as the device rounds it."""
import os
import re

import numpy as np

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _bound() -> float:
    src = open(os.path.join(ROOT, "position_agnostic_paged_b200", "csrc", "write_q8.cu")).read()
    return float(re.search(r"kErrLarge = ([0-9.e-]+)f;", src).group(1))


def _error(a, b, angle):
    """|x in fp32 - x| / (|x0| + |x1|), the larger of the pair's two: cos and sin rounded from fp64, a product, an fma."""
    f = np.float32
    c, s = np.cos(angle), np.sin(angle)
    cf, sf = c.astype(f).astype(np.float64), s.astype(f).astype(np.float64)
    x0 = ((a * cf).astype(f) - b * sf).astype(f).astype(np.float64)          # (the fp64 sum is exact to 2^-53)
    x1 = ((b * cf).astype(f) + a * sf).astype(f).astype(np.float64)
    return np.maximum(np.abs(x0 - (a * c - b * s)), np.abs(x1 - (b * c + a * s))) / (np.abs(x0) + np.abs(x1))


def test_rotation_error_bound():
    bound = _bound()
    # found by searching 1.2e8 pairs near 1 and small angles
    worst = np.array([(1.0546875, 0.031494140625, -0.02824645625338179), (1.0078125, 0.042236328125, -0.04687101831959606),
                      (1.015625, -0.04638671875, 0.04863783615400019), (1.015625, -0.0185546875, 0.017248086708582022)])
    assert _error(*worst.T).max() > 1.45e-7
    assert (_error(*worst.T) < bound).all()
    rng = np.random.default_rng(1)
    n = 1 << 20
    a = (1 + rng.integers(0, 128, n) / 128) * 2.0 ** rng.integers(-3, 3, n)
    b = (1 + rng.integers(0, 128, n) / 128) * 2.0 ** rng.integers(-8, 3, n) * rng.choice([-1, 1], n)
    assert (_error(a, b, rng.uniform(-4, 4, n)) < bound).all()
    # cos and sin: half an ulp of numbers below 1, |a| + |b| <= sqrt(2) r; a product and a sum of at most r
    assert bound > (np.sqrt(2) / 2 + 2) * 2.0 ** -24
