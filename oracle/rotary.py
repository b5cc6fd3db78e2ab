"""Rotary positions in NumPy, 64 bits throughout: frequencies with their long-sequence scalings, tables,
and the turned heads [host contract, section 4; gizai:dit, prepOf]."""

import math

import numpy as np


def rotary_frequencies(widths, theta=10000.0, scaling="none", factor=1.0, original=0, beta_fast=32.0, beta_slow=1.0):
    """(radians per position of each pair, axis of each pair, amplitude)."""
    freq, axis, amp = [], [], 1.0
    for a, w in enumerate(widths):
        base = theta
        if scaling == "ntk" and w > 2:
            base = theta * factor ** (w / (w - 2.0))
        for k in range(w // 2):
            f = base ** (-2.0 * k / w)
            if scaling == "linear":
                f /= factor
            elif scaling == "yarn":
                def at(turns):
                    return w * math.log(original / (2 * math.pi * turns)) / (2 * math.log(theta))
                lo, hi = max(0.0, math.floor(at(beta_fast))), min(w - 1.0, math.ceil(at(beta_slow)))
                r = min(1.0, max(0.0, (k - lo) / max(hi - lo, 1e-3)))
                f = f * (1 - r) + f / factor * r
            freq.append(f)
            axis.append(a)
    if scaling == "yarn":
        amp = 0.1 * math.log(factor) + 1.0
    return np.array(freq), np.array(axis), amp


def rotary_tables(pos, freq, axis, amp=1.0):
    """cos, sin [..., pairs] for pos [..., axes]."""
    angle = np.asarray(pos, np.float64)[..., axis] * freq
    return amp * np.cos(angle), amp * np.sin(angle)


def rotary_apply(x, cos, sin, halves, inverse=False):
    """x [..., rows, heads, d], cos / sin [..., rows, pairs]."""
    x = np.asarray(x, np.float64)
    n = cos.shape[-1]
    c, s = cos[..., None, :], (-sin if inverse else sin)[..., None, :]
    i = np.arange(n)
    a, b = (i, i + n) if halves else (2 * i, 2 * i + 1)
    out = x.copy()
    out[..., a] = x[..., a] * c - x[..., b] * s
    out[..., b] = x[..., a] * s + x[..., b] * c
    return out
