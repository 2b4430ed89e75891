"""The rotated append in 64 bits and plain loops: norm, angles, slots. Shares no code with
the library."""
import math

import numpy as np

EPS = {"f32": 2.0 ** -23, "f16": 2.0 ** -10, "bf16": 2.0 ** -7}
TINY = {"f32": 2.0 ** -149, "f16": 2.0 ** -24, "bf16": 2.0 ** -133}   # least step


def normed(x, weight, eps, offset=0.0):
    """x [T, H, D] float64; weight [D], [H, D] or None."""
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    return y if weight is None else y * (offset + weight)


def rotated(y, positions, inv_freq, axes, interleaved, factor=1.0):
    """positions [axes, T] whole numbers, inv_freq [rot / 2] float64. Returns z and, per
    element, the sizes of what was added: |y_a| + |y_b|."""
    z, mag = y.copy(), np.abs(y)
    half = len(inv_freq)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        for t in range(y.shape[0]):
            # (whole turns are taken off in extended precision)
            angle = math.fmod(float(positions[axes[i]][t]) * float(inv_freq[i]), 2 * math.pi)
            c, s = factor * math.cos(angle), factor * math.sin(angle)
            z[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            z[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
            mag[t, :, a] = mag[t, :, b] = factor * (np.abs(y[t, :, a]) + np.abs(y[t, :, b]))
    return z, mag


def bound(z, mag, dtype):
    """What an element may be off by. In f32: the sum of squares is 8 products and 5 joins, halved
    by the root, and root, quotient and two products follow: at most 11 half steps; cosine and
    sine are off by 2 half steps each and the angle by 2^-25; two products and a sum: 3. In
    all at most 20 half steps of 2^-24 of |y_a| + |y_b|. Then one rounding."""
    err = 20 * 2.0 ** -24 * mag
    return err + np.maximum((np.abs(z) + err) * EPS[dtype] / 2, TINY[dtype] / 2)
