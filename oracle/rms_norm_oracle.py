"""Float64 NumPy oracle of the RMS norm with the residual's addition: TEST
INFRASTRUCTURE ONLY (see ``oracle/__init__.py``); it shares no code with the
HIP path.

y = s / sqrt(mean(s^2) + eps) * weight over the last axis; the gradients of
sum(dy y) + sum(dresidual s).
"""

from __future__ import annotations

import numpy as np

__all__ = ["rms_norm", "rms_norm_bwd", "e4m3_nearest"]


def rms_norm(s, weight=None, eps=1e-5):
    s = np.asarray(s, np.float64)
    n = s / np.sqrt((s ** 2).mean(-1, keepdims=True) + eps)
    return n if weight is None else n * np.asarray(weight, np.float64)


def rms_norm_bwd(s, weight, dy, dresidual=None, eps=1e-5):
    s, dy = np.asarray(s, np.float64), np.asarray(dy, np.float64)
    d = s.shape[-1]
    r = 1.0 / np.sqrt((s ** 2).mean(-1, keepdims=True) + eps)
    u = dy if weight is None else dy * np.asarray(weight, np.float64)
    ds = r * u - s * r ** 3 * (u * s).sum(-1, keepdims=True) / d
    if dresidual is not None:
        ds = ds + np.asarray(dresidual, np.float64)
    return ds, (dy * s * r).reshape(-1, d).sum(0)


def e4m3_nearest(x):
    """x (|x| <= 448) to the nearest e4m3 value (3 mantissa bits, least normal
    exponent -6, subnormal step 2^-9), ties to even."""
    x = np.asarray(x, np.float64)
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
    step = 2.0 ** (e - 3)
    return np.round(x / step) * step
