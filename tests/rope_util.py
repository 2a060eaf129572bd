"""Rotary positions and norms of heads from their definitions, in float64 on the CPU, with the error bounds that the
library's arithmetic keeps.  Nothing here calls the library.

Bounds.  The library computes in fp32 and rounds once to bf16 (half a step: 2^-8 of the value).  Its sines come from an
angle held to 2^-25 half turns (the fraction of a turn as an fp32 number) and polynomials: 2^-22 each; the two
products and the sum add three roundings of 2^-24; r = 1 / sqrt(mean x^2 + eps) sums D <= 128 squares in chains of at most
8 + 3 additions, half of whose relative error counts, and rsqrt (2 ulp): under 2^-21, and two products after it.  In
all, under 2^-19 of the magnitudes that meet in an element."""
from __future__ import annotations

import numpy as np

HALF_BF16 = 2.0 ** -8
FP32 = 2.0 ** -19


def pairs(rot, interleaved):
    """Indices (a, b) of the elements of each pair."""
    i = np.arange(rot // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)


def turn(x, positions, rotary, back=False, magnitude=False):
    """x [B, H, S, D] with its pairs turned by positions [B, S] (back: the transposed rotation); magnitude: sums of
    magnitudes instead, for the bounds."""
    f = np.array(rotary.frequencies, np.float64)
    out = np.abs(x) if magnitude else x.copy()
    if len(f) == 0:
        return out
    angle = np.asarray(positions, np.float64)[:, None, :, None] * f
    a, b = pairs(rotary.rotary_dim, rotary.interleaved)
    m = rotary.factor
    if magnitude:
        both = abs(m) * (np.abs(x[..., a]) + np.abs(x[..., b]))
        out[..., a], out[..., b] = both, both
        return out
    c, s = m * np.cos(angle), m * np.sin(angle) * (-1 if back else 1)
    out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., b] * c + x[..., a] * s
    return out


def norm(x, weight, eps):
    """(u, r) of rows x."""
    if weight is None:
        return x, None
    with np.errstate(invalid="ignore", over="ignore"):
        r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
        return x * r * weight, r


def forward(x, positions, rotary, weight=None, eps=1e-6):
    """(y, tolerance of a bf16 y, tolerance of an fp32 y) for float64 rows x [B, H, S, D]."""
    u, _ = norm(x, weight, eps)
    y = turn(u, positions, rotary)
    fp32 = FP32 * turn(u, positions, rotary, magnitude=True)
    return y, HALF_BF16 * np.abs(y) + fp32 + 2.0 ** -133, fp32


def backward(dy, x, positions, rotary, weight=None, eps=1e-6):
    """(dx, its tolerance, dw, its tolerance as fp32) for upstream gradients dy.  dw sums its rows in chains of at most
    8 + 5 + 8 + 64 additions: 2^-17 of the sum of magnitudes, the terms' own errors included."""
    g, big = turn(dy, positions, rotary, back=True), turn(dy, positions, rotary, magnitude=True)
    if weight is None:
        return g, HALF_BF16 * np.abs(g) + FP32 * big + 2.0 ** -133, None, None
    u, r = norm(x, np.ones_like(weight), eps)
    c = (g * weight * u).mean(-1, keepdims=True)
    dx = r * (g * weight - u * c)
    near = r * (big * np.abs(weight) + np.abs(u) * (big * np.abs(weight * u)).mean(-1, keepdims=True))
    axes = (0, 1, 2)
    return dx, HALF_BF16 * np.abs(dx) + 4 * FP32 * near + 2.0 ** -133, (g * u).sum(axes), 2.0 ** -17 * (big * np.abs(u)).sum(axes)


def to_f64(t):
    return t.detach().double().cpu().numpy()
