"""Float64 NumPy oracle of the gated linear recurrence: TEST INFRASTRUCTURE ONLY
(see ``oracle/__init__.py``); it shares no code with the HIP path.

Per batch row, channel and step: u = gate + gate_bias; g = u, softplus(u) or
sigmoid(u); a = exp(A g); w = 1, sqrt(1 - a^2) or 1 - a; v = x sigmoid(input_gate
+ input_bias) (or x); h <- a h + w v; y = h. A step behind a row's length leaves
the state, its y is 0.

With the results come their rooms: how far a float32 evaluation may be off, by
counting roundings (E = 2^-24 relative each) through the same recurrences on
magnitudes. A gate is off by (16 + |u|) E of itself: the sum u is off by E |u|, which
is as much of e^-u; an exponential, a logarithm, a reciprocal and sums are 16 E. la = A g
is off by one E more, a by |la| times that and 3 E more, w by the gate's and 24 E (what 1
- a cancels is at most 5-fold), v by 12 E and its gate's |u| E. A state takes these, and
one rounding a step; joins of tiles, a second
evaluation and another order of the sums are covered by twice that and 16 E of
the magnitude. bfloat16 outputs are the caller's to add.
"""

from __future__ import annotations

import numpy as np

__all__ = ["gated_linear", "gated_linear_bwd"]

E = 2.0 ** -24


def _f64(x):
    return None if x is None else np.asarray(x, np.float64)


def _sigmoid(u):
    e = np.exp(-np.abs(u))
    return np.where(u < 0, e, 1.0) / (1.0 + e)


class _Parts:
    """What every step's inputs make: arrays [B, L, D]."""

    def __init__(self, x, gate, A, input_gate, gate_bias, input_bias, act, scale):
        x, gate, A, ig = _f64(x), _f64(gate), _f64(A), _f64(input_gate)
        u = gate if gate_bias is None else gate + _f64(gate_bias)
        if act == "sigmoid":
            g, slope, curve = _sigmoid(u), _sigmoid(u) * _sigmoid(-u), 1.0
        elif act == "softplus":
            g, slope, curve = np.logaddexp(u, 0.0), _sigmoid(u), 1.0
        else:
            g, slope, curve = u, np.ones_like(u), 0.0
        la = A * g
        a, rest = np.exp(la), -np.expm1(la)
        if scale == "norm":
            w = np.sqrt(-np.expm1(2 * la))
            with np.errstate(divide="ignore", invalid="ignore"):
                dw = np.where(w > 0, -a * a / w, 0.0)
        elif scale == "complement":
            w, dw = rest, -a
        else:
            w, dw = np.ones_like(a), np.zeros_like(a)
        if ig is None:
            s, t, ui = np.ones_like(x), np.zeros_like(x), np.zeros_like(x)
        else:
            ui = ig if input_bias is None else ig + _f64(input_bias)
            s, t = _sigmoid(ui), _sigmoid(ui) * _sigmoid(-ui)
        self.A, self.g, self.slope, self.la, self.a, self.w, self.dw, self.x, self.s, self.t = (
            A, g, slope, la, a, w, dw, x, s, t)
        self.v = x * s
        # relative errors
        self.rg = ((16 + np.abs(u)) * curve + 1) * E
        self.ra = np.abs(la) * (self.rg + 4 * E) + 3 * E
        self.rw = self.rg + 24 * E if scale is not None else 0 * a
        self.rv = (12 + np.abs(ui)) * E
        self.rdw = 2 * self.ra + self.rw + 8 * E


def _lengths(B, L, seqlens):
    if seqlens is None:
        return np.full(B, L)
    return np.clip(np.asarray(seqlens, np.int64), 0, L)


def gated_linear(x, gate, A, input_gate=None, gate_bias=None, input_bias=None, act=None, scale=None, h0=None,
                 seqlens=None):
    """(y [B, L, D], h_final [B, D], room of y, room of h_final)."""
    p = _Parts(x, gate, A, input_gate, gate_bias, input_bias, act, scale)
    y, h, room_y, room_h, _, _ = _forward(p, _f64(h0), seqlens)
    return y, h, room_y, room_h


def _forward(p, h0, seqlens):
    B, L, D = p.a.shape
    lens = _lengths(B, L, seqlens)
    h = np.zeros((B, D)) if h0 is None else h0.copy()
    m, r = np.abs(h), np.zeros((B, D))
    y, room = np.zeros((B, L, D)), np.zeros((B, L, D))
    before, mag_before, room_before = (np.zeros((B, L, D)) for _ in range(3))
    for t in range(L):
        on = (lens > t)[:, None]
        before[:, t], mag_before[:, t], room_before[:, t] = h, m, 2 * r + 16 * E * m
        a, b = p.a[:, t], p.w[:, t] * p.v[:, t]
        r = np.where(on, a * r + a * m * p.ra[:, t] + np.abs(b) * (p.rw[:, t] + p.rv[:, t] + 2 * E), r)
        h, m = np.where(on, a * h + b, h), np.where(on, a * m + np.abs(b), m)
        r = np.where(on, r + E * m, r)
        y[:, t], room[:, t] = h * on, (2 * r + 16 * E * m) * on
    return y, h, room, 2 * r + 16 * E * m, (before, mag_before), room_before


def gated_linear_bwd(x, gate, A, dy, input_gate=None, gate_bias=None, input_bias=None, act=None, scale=None, h0=None,
                     dh_final=None, seqlens=None):
    """Gradients of sum(dy y) + sum(dh_final h_final): two dicts, the values and
    their rooms, of dx, dgate, dinput_gate, dA, dgate_bias, dinput_bias, dh0."""
    p = _Parts(x, gate, A, input_gate, gate_bias, input_bias, act, scale)
    B, L, D = p.a.shape
    lens = _lengths(B, L, seqlens)
    _, _, _, _, (before, mag_before), room_before = _forward(p, _f64(h0), seqlens)
    dy = _f64(dy)
    d = np.zeros((B, D)) if dh_final is None else _f64(dh_final).copy()
    m, r = np.abs(d), np.zeros((B, D))
    out = {k: np.zeros((B, L, D)) for k in ("dx", "dgate", "dinput_gate", "dla")}
    room = {k: np.zeros((B, L, D)) for k in out}
    mag = {k: np.zeros((B, L, D)) for k in out}
    for t in reversed(range(L)):
        on = (lens > t)[:, None]
        a, w, v, dw = p.a[:, t], p.w[:, t], p.v[:, t], p.dw[:, t]
        d, m = np.where(on, d + dy[:, t], d), np.where(on, m + np.abs(dy[:, t]), m)
        r = np.where(on, r + E * m, r)
        rd = 2 * r + 16 * E * m  # of d here
        rel = p.rw[:, t] + p.rv[:, t] + 8 * E
        for name, f in (("dx", w * p.s[:, t]), ("dinput_gate", w * p.x[:, t] * p.t[:, t])):
            out[name][:, t] = d * f * on
            room[name][:, t] = (rd + m * rel) * np.abs(f) * on
            mag[name][:, t] = m * np.abs(f) * on
        hb, hm, hr = before[:, t], mag_before[:, t], room_before[:, t]
        out["dla"][:, t] = d * (a * hb + dw * v) * on
        mag["dla"][:, t] = m * (a * hm + np.abs(dw * v)) * on
        room["dla"][:, t] = (rd * (a * np.abs(hb) + np.abs(dw * v)) + m * (a * hr + a * hm * (p.ra[:, t] + 4 * E)
                             + np.abs(dw * v) * (p.rdw[:, t] + p.rv[:, t] + 4 * E))) * on
        f = p.A * p.slope[:, t]
        out["dgate"][:, t] = out["dla"][:, t] * f
        mag["dgate"][:, t] = mag["dla"][:, t] * np.abs(f)
        room["dgate"][:, t] = (room["dla"][:, t] + mag["dla"][:, t] * (p.rg[:, t] + 8 * E)) * np.abs(f)
        r = np.where(on, a * r + a * m * p.ra[:, t], r)
        d, m = np.where(on, a * d, d), np.where(on, a * m, m)
    out["dh0"], room["dh0"] = d, 2 * r + 16 * E * m
    g, rg = np.abs(p.g), p.rg + 2 * E
    out["dA"] = (out["dla"] * p.g).sum((0, 1))
    # sums: 64 roundings of the terms' magnitudes (partial sums in float32, joined in double)
    room["dA"] = ((room["dla"] + mag["dla"] * (rg + 64 * E)) * g).sum((0, 1))
    for name, of in (("dgate_bias", "dgate"), ("dinput_bias", "dinput_gate")):
        out[name] = out[of].sum((0, 1))
        room[name] = (room[of] + 64 * E * mag[of]).sum((0, 1))
    del out["dla"], room["dla"]
    return out, room
