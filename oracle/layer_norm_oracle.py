"""Float64 NumPy oracle of the layer norm: TEST INFRASTRUCTURE ONLY (see
``oracle/__init__.py``); it shares no code with the HIP path.

y = (s - mean(s)) / sqrt(mean((s - mean(s))^2) + eps) * weight + bias over the
last axis; the gradients of sum(dy y) + sum(dresidual s).
"""

from __future__ import annotations

import numpy as np

__all__ = ["layer_norm", "layer_norm_bwd"]


def _normal(s, eps):
    d = s - s.mean(-1, keepdims=True)
    return d / np.sqrt((d ** 2).mean(-1, keepdims=True) + eps)


def layer_norm(s, weight=None, bias=None, eps=1e-5):
    y = _normal(np.asarray(s, np.float64), eps)
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    return y if bias is None else y + np.asarray(bias, np.float64)


def layer_norm_bwd(s, weight, dy, dresidual=None, eps=1e-5):
    """(ds, dweight, dbias). ds from the Jacobian of n = d r: with r' = -r^3 d / width a row's."""
    s, dy = np.asarray(s, np.float64), np.asarray(dy, np.float64)
    width = s.shape[-1]
    d = s - s.mean(-1, keepdims=True)
    r = 1.0 / np.sqrt((d ** 2).mean(-1, keepdims=True) + eps)
    u = dy if weight is None else dy * np.asarray(weight, np.float64)
    dd = u * r - d * r ** 3 * (u * d).sum(-1, keepdims=True) / width
    ds = dd - dd.mean(-1, keepdims=True)
    if dresidual is not None:
        ds = ds + np.asarray(dresidual, np.float64)
    return ds, (dy * d * r).reshape(-1, width).sum(0), dy.reshape(-1, width).sum(0)
