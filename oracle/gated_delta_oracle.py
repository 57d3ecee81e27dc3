"""Float64 NumPy oracle of the gated delta rule: TEST INFRASTRUCTURE ONLY (see
``oracle/__init__.py``); it shares no code with the HIP path.

Per batch row, value head h (query/key head h // (H / G)) and step t, with the
state S [N, P] and the log decay g = max(dt A, -200):

    S <- exp(g) S;   e = v - k^T S;   S <- S + k (beta e)^T;   y = scale q^T S

dt = softplus(dt_raw + dt_bias) or dt_raw + dt_bias; beta = sigmoid(beta_raw)
or beta_raw; with ``l2norm``, q and k are divided by sqrt(|.|^2 + 1e-6).
``seqlens``: steps of each batch row; y (and gradients) behind them are 0.

Shapes: q, k [B, L, G, N]; v, y [B, L, H, P]; dt, beta [B, L, H]; A, dt_bias
[H]; h0, h_final [B, H, P, N].
"""

from __future__ import annotations

import numpy as np

__all__ = ["gated_delta", "gated_delta_bwd"]

L2_EPS = 1e-6


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def _sigmoid(x):
    return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


class _Steps:
    """The per-step quantities of one problem, heads expanded: q, k [B, L, H, N]."""

    def __init__(self, q, k, v, dt, A, beta, dt_bias, softplus, sigmoid, l2norm, seqlens):
        self.qr, self.kr, self.v = _f64(q), _f64(k), _f64(v)
        self.B, self.L, self.G, self.N = self.qr.shape
        self.H, self.P = self.v.shape[2:]
        self.r = self.H // self.G
        self.A = _f64(A)
        self.x = _f64(dt) + (0.0 if dt_bias is None else _f64(dt_bias))
        self.dt = np.logaddexp(0.0, self.x) if softplus else self.x
        with np.errstate(invalid="ignore"):
            self.g = np.maximum(self.dt * self.A, -200.0)
        self.beta = _sigmoid(_f64(beta)) if sigmoid else _f64(beta)
        self.nq = 1.0 / np.sqrt((self.qr ** 2).sum(-1, keepdims=True) + L2_EPS) if l2norm else np.ones(1)
        self.nk = 1.0 / np.sqrt((self.kr ** 2).sum(-1, keepdims=True) + L2_EPS) if l2norm else np.ones(1)
        self.q = np.repeat(self.qr * self.nq, self.r, 2)
        self.k = np.repeat(self.kr * self.nk, self.r, 2)
        n = np.full(self.B, self.L) if seqlens is None else np.clip(np.asarray(seqlens), 0, self.L)
        self.on = np.arange(self.L)[None, :] < n[:, None]       # [B, L]

    def at(self, t):
        """q, k, v, exp(g), beta of step t; a step that is not there has q = k = v = 0, decay 1, beta 0."""
        on = self.on[:, t][:, None]
        z = lambda a: np.where(on[..., None], a[:, t], 0.0)  # noqa: E731
        return (z(self.q), z(self.k), z(self.v), np.where(on, np.exp(self.g[:, t]), 1.0),
                np.where(on, self.beta[:, t], 0.0))


def gated_delta(q, k, v, dt, A, beta, dt_bias=None, softplus=False, sigmoid=False, l2norm=False, scale=1.0,
                h0=None, seqlens=None):
    """y [B, L, H, P] and h_final [B, H, P, N]."""
    s = _Steps(q, k, v, dt, A, beta, dt_bias, softplus, sigmoid, l2norm, seqlens)
    S = np.zeros((s.B, s.H, s.P, s.N)) if h0 is None else _f64(h0).copy()
    y = np.zeros((s.B, s.L, s.H, s.P))
    for t in range(s.L):
        qt, kt, vt, a, b = s.at(t)
        S = S * a[..., None, None]
        e = vt - np.einsum("bhpn,bhn->bhp", S, kt)
        S = S + (b[..., None] * e)[..., None] * kt[:, :, None, :]
        y[:, t] = scale * np.einsum("bhpn,bhn->bhp", S, qt)
    return y, S


def gated_delta_bwd(q, k, v, dt, A, beta, dy, dt_bias=None, softplus=False, sigmoid=False, l2norm=False, scale=1.0,
                    h0=None, dh_final=None, seqlens=None):
    """Gradients of sum(dy y) + sum(dh_final h_final) by the reversed recurrence:
    a dict of dq, dk, dv, ddt, dA, dbeta, ddt_bias, dh0, and under "mag" the
    sums of absolute values behind dA and ddt_bias, and of the two terms that
    the norms' gradients subtract behind dq and dk."""
    s = _Steps(q, k, v, dt, A, beta, dt_bias, softplus, sigmoid, l2norm, seqlens)
    dy = _f64(dy)
    S = np.zeros((s.B, s.H, s.P, s.N)) if h0 is None else _f64(h0).copy()
    decayed, errs, states = [], [], []
    for t in range(s.L):
        qt, kt, vt, a, b = s.at(t)
        S1 = S * a[..., None, None]
        e = vt - np.einsum("bhpn,bhn->bhp", S1, kt)
        S = S1 + (b[..., None] * e)[..., None] * kt[:, :, None, :]
        decayed.append(S1)
        errs.append(e)
        states.append(S)
    X = np.zeros_like(S) if dh_final is None else _f64(dh_final).copy()
    dq, dk = np.zeros((s.B, s.L, s.H, s.N)), np.zeros((s.B, s.L, s.H, s.N))
    dv, dg, db = np.zeros_like(s.v), np.zeros((s.B, s.L, s.H)), np.zeros((s.B, s.L, s.H))
    for t in reversed(range(s.L)):
        qt, kt, vt, a, b = s.at(t)
        dyt = scale * np.where(s.on[:, t][:, None, None], dy[:, t], 0.0)
        dq[:, t] = np.einsum("bhpn,bhp->bhn", states[t], dyt)
        X = X + dyt[..., None] * qt[:, :, None, :]
        u = np.einsum("bhpn,bhn->bhp", X, kt)
        db[:, t] = (u * errs[t]).sum(-1)
        de = b[..., None] * u
        dv[:, t] = de
        dk[:, t] = np.einsum("bhpn,bhp->bhn", X, b[..., None] * errs[t]) - np.einsum("bhpn,bhp->bhn", decayed[t], de)
        X = X - de[..., None] * kt[:, :, None, :]
        dg[:, t] = (X * decayed[t]).sum((-1, -2))
        X = X * a[..., None, None]
    on = s.on[:, :, None]
    dg, db = dg * on, db * on
    out = {"dv": dv * on[..., None], "dh0": X}
    mag = {}
    for name, d, raw, nr in (("dq", dq, s.qr, s.nq), ("dk", dk, s.kr, s.nk)):
        d = (d * on[..., None]).reshape(s.B, s.L, s.G, s.r, s.N).sum(3)
        if l2norm:
            unit = raw * nr
            mag[name] = nr * (np.abs(d) + np.abs(unit * (unit * d).sum(-1, keepdims=True)))
            d = nr * (d - unit * (unit * d).sum(-1, keepdims=True))
        out[name] = d
    with np.errstate(invalid="ignore"):
        dg = np.where(s.dt * s.A < -200.0, 0.0, dg)            # the clamp's own gradient
        dx = dg * s.A * (_sigmoid(s.x) if softplus else 1.0)
        along = np.where(on & (dg != 0.0), dg * s.dt, 0.0)     # a cut-off step: 0, whatever dt
    out["dA"] = along.sum((0, 1))
    out["ddt"], out["ddt_bias"] = dx, dx.sum((0, 1))
    out["dbeta"] = db * s.beta * (1.0 - s.beta) if sigmoid else db
    out["mag"] = dict(mag, dA=np.abs(along).sum((0, 1)), ddt_bias=np.abs(dx).sum((0, 1)))
    return out
