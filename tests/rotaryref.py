"""Plain 64-bit definition of the rows' norm and rotation (numpy), its
tolerances, and the tests' inputs."""
from __future__ import annotations

import math

import numpy as np
import torch

from cacheref import F32, HALF_STEP

# rounding of the smallest numbers of a type
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def turns(rot, base=10000.0, scaling="none", factor=1.0, original=0, low=1.0,
          high=4.0):
    """Turns per position of each pair."""
    out = []
    for i in range(rot // 2):
        if scaling == "base":
            b = base * factor ** (rot / (rot - 2))
        else:
            b = base
        f = b ** (-2 * i / rot) / (2 * math.pi)
        w = 1.0
        if scaling == "linear":
            w = 0.0
        elif scaling == "ramp":
            def pair(t):
                return (rot / 2 * math.log(original / (2 * math.pi * t))
                        / math.log(base))
            lo = max(math.floor(pair(high)), 0)
            hi = min(math.ceil(pair(low)), rot - 1)
            w = 1.0 - (i - lo) / max(hi - lo, 1e-3)
        elif scaling == "bands":
            w = (original * f - low) / (high - low)
        w = min(max(w, 0.0), 1.0)
        out.append(f if scaling in ("none", "base") else
                   f * w + f / factor * (1.0 - w))
    return np.array(out)


def rotate(x, pos, table, rot, layout, amplitude=1.0, weight=None, eps=0.0):
    """x [..., heads, D] float64 at positions pos [...]; table: turns per
    position in units of 2^-64 (Python integers).  Returns the result and the
    magnitude that its fp32 rounding is relative to."""
    x = x.astype(np.float64)
    D = x.shape[-1]
    if weight is not None:
        x = x / np.sqrt((x * x).sum(-1, keepdims=True) / D + eps) * weight
    y, mag = x.copy(), np.abs(x)
    for i, f in enumerate(table):
        # exact: whole turns drop out of the integers
        phase = np.array([int(p) * f % (1 << 64) for p in pos.reshape(-1)],
                         dtype=np.float64).reshape(pos.shape) / 2.0 ** 64
        c = np.cos(2 * math.pi * phase)[..., None] * amplitude
        s = np.sin(2 * math.pi * phase)[..., None] * amplitude
        a, b = (i, i + rot // 2) if layout == "half" else (2 * i, 2 * i + 1)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        m = abs(amplitude) * (np.abs(x[..., a]) + np.abs(x[..., b]))
        mag[..., a] = mag[..., b] = m
    return y, mag


def tolerance(y, mag, dtype):
    """One rounding to the type, and of fp32: the norm's sum of 256 squares
    in 8 steps of a lane and 5 over lanes (half of 13 of the root), mean, eps,
    root, reciprocal and two products (6), cosine and sine (the angle 3, the
    series 2, the amplitude 1, the phase's 32 bits 1), the two products and
    their sum (2): under 24 half steps of 2^-24."""
    t = HALF_STEP[dtype]
    return t * np.abs(y) + 24 * F32 * mag * (1 + t) + TINY[dtype]
