"""Float64 oracle of rotary positions and of their frequencies.

Pair i of a head turns by position times freq[i]; the calls of the same names in the library
are checked against these, and these against complex products, inverses and the
dependence of scores on distances alone.
"""
from fractions import Fraction

import numpy as np


def _cos_sin(position, freq):
    """Cosine and sine of position times freq: the product needs up to 55 bits, so what the double
    leaves out comes back as a first-order term."""
    a = float(position) * float(freq)
    rest = float(Fraction(int(position)) * Fraction(float(freq)) - Fraction(a))
    return np.cos(a) - rest * np.sin(a), np.sin(a) + rest * np.cos(a)


def rotate(x, position, freq, interleaved=False, transposed=False, magnitude=1.0):
    """x [n, heads, D] rotated; rows of a negative position become NaN (the library leaves them)."""
    rot = 2 * len(freq)
    y = x.astype(np.float64).copy()
    for n in range(len(x)):
        for i, f in enumerate(freq):
            c, s = _cos_sin(position[n], f)
            s = -s if transposed else s
            j1, j2 = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
            x1, x2 = x[n, :, j1].astype(np.float64), x[n, :, j2].astype(np.float64)
            y[n, :, j1] = magnitude * (x1 * c - x2 * s)
            y[n, :, j2] = magnitude * (x2 * c + x1 * s)
        if position[n] < 0:
            y[n] = np.nan
    return y


def frequencies(rot, base, scaling="plain", factor=1.0, original=0.0, low=1.0, high=32.0):
    """(freq [rot / 2], magnitude) of each way of scaling for long contexts, in float64."""
    i = np.arange(rot // 2)
    f = base ** (-2.0 * i / rot)
    turns = original * f / (2 * np.pi)                    # over the original length
    if scaling == "plain":
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "base":
        return (base * factor ** (rot / (rot - 2.0))) ** (-2.0 * i / rot), 1.0
    if scaling == "bands":
        keep = np.clip((turns - low) / (high - low), 0, 1)
        return f * keep + f / factor * (1 - keep), 1.0
    d = lambda t: rot * np.log(original / (2 * np.pi * t)) / (2 * np.log(base))  # noqa: E731
    a, b = max(0.0, np.floor(d(high))), min(rot - 1.0, np.ceil(d(low)))
    keep = 1 - np.clip((i - a) / (b - a if b > a else 0.001), 0, 1)
    return f * keep + f / factor * (1 - keep), 0.1 * np.log(factor) + 1.0
