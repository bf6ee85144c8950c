"""Rotary positions, the quantised cache rows and attention over them (oracle).

TEST INFRASTRUCTURE (see the package header).

Everything in float64 from the given values; the steps that are fp32 by
definition (a cached row's scale, and the quotient before its rounding) are
rounded to fp32 where the definition says so.
"""
from __future__ import annotations

import math

import numpy as np


def rope_frequencies(rot, base, scaling="none", factor=1.0, orig_len=0, fast=32.0, slow=1.0):
    """Radians per position of each pair."""
    out = []
    for i in range(rot // 2):
        f = base ** (-2.0 * i / rot)
        if scaling == "linear":
            f /= factor
        elif scaling == "parts":
            turns = orig_len * f / (2 * math.pi)
            g = min(max((turns - slow) / (fast - slow), 0.0), 1.0)
            f = g * f + (1 - g) * f / factor
        out.append(f)
    return np.array(out)


def rope(x, positions, freq, layout="half", amp=1.0):
    """x [n][heads][d] with the leading 2*len(freq) elements of each head rotated."""
    x = np.array(x, np.float64)
    half = len(freq)
    angle = np.asarray(positions, np.float64)[:, None, None] * freq
    c, s = amp * np.cos(angle), amp * np.sin(angle)
    ia = np.arange(half) if layout == "half" else 2 * np.arange(half)
    ib = ia + (half if layout == "half" else 1)
    a, b = x[..., ia].copy(), x[..., ib].copy()
    x[..., ia] = a * c - b * s
    x[..., ib] = a * s + b * c
    return x


def quantise_rows(x, kind):
    """Codes (as the numbers they are) and fp32 scales of rows x[..., d]: scale = amax / T, code = x / scale
    rounded to nearest even, a row of zeros or a quotient that is no number giving 0."""
    x = np.asarray(x, np.float32)
    top = np.float32(127.0 if kind == "i8" else 448.0)
    with np.errstate(all="ignore"):
        amax = np.nanmax(np.where(np.isnan(x), np.float32(0), np.abs(x)), axis=-1)
        scale = (amax / top).astype(np.float32)
        y = np.where(scale[..., None] == 0, np.float32(0), x / np.where(scale == 0, np.float32(1), scale)[..., None])
        y = np.where(np.isnan(y), np.float32(0), y).astype(np.float64)
    y = np.clip(y, -float(top), float(top))
    if kind == "i8":
        return np.rint(y), scale
    _, e = np.frexp(y)
    step = np.exp2(np.maximum(e - 1, -6) - 3.0)
    return np.rint(y / step) * step, scale


def attend(q, k, v, visible, scale):
    """q [m][hq][d], k and v [n][hkv][d], visible bool [m][n] -> o [m][hq][d] and sum_j p_j |v_j| of the same shape.

    What a row does not see does not enter its sums, whatever its value; a row that sees nothing is zero."""
    m, hq, d = q.shape
    hkv = k.shape[1]
    o, spread = np.zeros((m, hq, d)), np.zeros((m, hq, d))
    for h in range(hq):
        g = h // (hq // hkv)
        for i in range(m):
            see = np.flatnonzero(visible[i])
            if not len(see):
                continue
            s = scale * (k[see, g].astype(np.float64) @ q[i, h].astype(np.float64))
            p = np.exp(s - s.max())
            p /= p.sum()
            o[i, h] = p @ v[see, g].astype(np.float64)
            spread[i, h] = p @ np.abs(v[see, g].astype(np.float64))
    return o, spread
