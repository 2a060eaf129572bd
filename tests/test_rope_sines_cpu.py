"""The sines' polynomials, with the coefficients as they stand in csrc/rope.cuh: how far they are from cos and sin on half
a turn, by themselves and in the order and roundings of the kernels."""
import os
import re

import numpy as np

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "causal_scaled_dot_gb300", "csrc", "rope.cuh")


def coefficients():
    """cos's and sin's, highest power first, as fp32 numbers."""
    with open(SOURCE) as f:
        body = re.search(r"void rope_wave2\(.*?\n}", f.read(), re.S).group(0)
    steps = re.findall(r"\b([cs]) = ptx::fma2\(y, (?:both\(([-\d.e]+)f\)|[cs]), both\(([-\d.e]+)f\)\)", body)
    out = {"c": [], "s": []}
    for name, first, then in steps:
        out[name] += [np.float32(x) for x in (first, then) if x]
    return out["c"], out["s"]


def horner(c, y, round_to=np.float64):
    r = round_to(c[0])
    for x in c[1:]:  # a product and a sum with one rounding
        r = round_to(np.float64(r) * np.float64(y) + np.float64(x))
    return r


def test_the_polynomials_by_themselves():
    c, s = coefficients()
    assert len(c) == 5 and len(s) == 5
    x = np.linspace(-0.5, 0.5, 200_001)
    assert np.abs(horner(c, x * x) - np.cos(np.pi * x)).max() <= 7.8e-8
    assert np.abs(x * horner(s, x * x) - np.sin(np.pi * x)).max() <= 4.8e-8


def test_with_the_kernels_roundings():
    """Two million angles as 32-bit fractions of a turn: under 2^-22."""
    c, s = coefficients()
    t = np.random.default_rng(1).integers(0, 2 ** 32, 2_000_000, dtype=np.uint64)
    twice = ((t << np.uint64(1)) & np.uint64(0xFFFFFFFF)).astype(np.uint32).view(np.int32)
    x = (twice.astype(np.float32) * np.float32(2.0 ** -32)).astype(np.float32)
    y = (x * x).astype(np.float32)
    cos, sin = horner(c, y, np.float32), (horner(s, y, np.float32) * x).astype(np.float32)
    flip = np.where(((t ^ (t << np.uint64(1))) & np.uint64(0x80000000)) != 0, -1.0, 1.0)
    angle = 2 * np.pi * t.astype(np.float64) / 2.0 ** 32
    assert np.abs(cos * flip - np.cos(angle)).max() < 2.0 ** -22
    assert np.abs(sin * flip - np.sin(angle)).max() < 2.0 ** -22
