"""Pins of the gated linear recurrence's oracle by something other than itself:
closed forms, the scan's oracle, differences, automatic differentiation."""

import numpy as np
import pytest
import torch

import oracle

FORMS = [(act, scale) for act in (None, "softplus", "sigmoid") for scale in (None, "norm", "complement")]


def inputs(B, L, D, seed, act):
    rng = np.random.default_rng(seed)
    t = dict(x=rng.standard_normal((B, L, D)), gate=rng.standard_normal((B, L, D)), A=-np.exp(rng.standard_normal(D)),
             input_gate=rng.standard_normal((B, L, D)), gate_bias=rng.standard_normal(D),
             input_bias=rng.standard_normal(D), h0=rng.standard_normal((B, D)))
    if act is None:  # (steps themselves: not negative)
        t["gate"], t["gate_bias"] = np.abs(t["gate"]), np.abs(t["gate_bias"])
    return t


def test_constant_gates_are_a_geometric_sum():
    L, a = 30, 0.9
    one = np.ones((1, L, 1))
    y, h, _, _ = oracle.gated_linear(one, one, np.array([np.log(a)]), h0=np.array([[2.0]]))
    n = np.arange(1, L + 1)
    assert np.allclose(y[0, :, 0], (1 - a ** n) / (1 - a) + 2 * a ** n) and np.isclose(h, y[0, -1])
    y, _, _, _ = oracle.gated_linear(one, one, np.array([np.log(a)]), scale="complement")
    assert np.allclose(y[0, :, 0], 1 - a ** n)
    y, _, _, _ = oracle.gated_linear(one, one, np.array([np.log(a)]), scale="norm")
    assert np.allclose(y[0, :, 0], np.sqrt(1 - a * a) * (1 - a ** n) / (1 - a))


def test_softplus_with_the_complement_is_a_sigmoid_gate():
    t = inputs(2, 9, 3, 1, "softplus")
    t.update(A=-np.ones(3), input_gate=None, input_bias=None)
    y, _, _, _ = oracle.gated_linear(**t, act="softplus", scale="complement")
    z = 1 / (1 + np.exp(-(t["gate"] + t["gate_bias"])))
    h = t["h0"]
    for i in range(9):
        h = (1 - z[:, i]) * h + z[:, i] * t["x"][:, i]
        assert np.allclose(y[:, i], h)


def test_norm_keeps_a_unit_variance():
    rng = np.random.default_rng(2)
    y, _, _, _ = oracle.gated_linear(rng.standard_normal((1, 400, 300)), rng.standard_normal((1, 400, 300)),
                                     np.full(300, -1.0), act="sigmoid", scale="norm")
    assert abs((y[:, 50:] ** 2).mean() - 1) < 0.02


def test_against_the_scans_oracle():
    # one state a channel, B = C = 1, u = x / dt: the selective scan's recurrence
    t = inputs(2, 12, 5, 3, "softplus")
    y, h, _, _ = oracle.gated_linear(t["x"], t["gate"], t["A"], None, t["gate_bias"], None, "softplus", None, t["h0"])
    dt = oracle.softplus(t["gate"] + t["gate_bias"])
    one = np.ones((2, 12, 1))
    ref = oracle.selective_scan(t["x"] / dt, t["gate"], t["A"][:, None], one, one, delta_bias=t["gate_bias"],
                                delta_softplus=True, h0=t["h0"][..., None])
    assert np.allclose(y, ref[0]) and np.allclose(h, ref[1][..., 0])


def test_lengths_and_a_decay_of_one():
    t = inputs(3, 8, 4, 4, "sigmoid")
    y, h, _, _ = oracle.gated_linear(**t, act="sigmoid", scale="norm", seqlens=[0, 5, 99])
    assert (y[0] == 0).all() and (h[0] == t["h0"][0]).all() and (y[1, 5:] == 0).all() and (h[1] == y[1, 4]).all()
    t["A"][:] = 0
    y, h, _, _ = oracle.gated_linear(**t, act="sigmoid", scale="norm")
    assert (y == t["h0"][:, None]).all()


@pytest.mark.parametrize("act,scale", FORMS)
def test_gradients_by_differences(act, scale):
    t = inputs(2, 5, 3, 5, act)
    lens = [5, 3]
    rng = np.random.default_rng(6)
    dy, dh = rng.standard_normal((2, 5, 3)), rng.standard_normal((2, 3))

    def loss():
        y, h, _, _ = oracle.gated_linear(**t, act=act, scale=scale, seqlens=lens)
        return (y * dy).sum() + (h * dh).sum()

    got, room = oracle.gated_linear_bwd(**t, dy=dy, act=act, scale=scale, dh_final=dh, seqlens=lens)
    for name, v in t.items():
        assert got["d" + name].shape == room["d" + name].shape == v.shape
        for i in np.ndindex(v.shape):
            keep = v[i]
            v[i] = keep + 1e-6
            up = loss()
            v[i] = keep - 1e-6
            down = loss()
            v[i] = keep
            assert abs((up - down) / 2e-6 - got["d" + name][i]) < 2e-7, (name, i)


def test_rooms_hold_a_float32_evaluation():
    t = inputs(2, 300, 8, 7, "sigmoid")
    t["A"] *= 0.02
    f = {k: torch.tensor(v, dtype=torch.float32) for k, v in t.items()}
    t = {k: v.double().numpy() for k, v in f.items()}
    y, _, room, _ = oracle.gated_linear(**t, act="sigmoid", scale="norm")
    g = torch.sigmoid(f["gate"] + f["gate_bias"])
    la = f["A"] * g
    b = torch.sqrt(-torch.expm1(2 * la)) * f["x"] * torch.sigmoid(f["input_gate"] + f["input_bias"])
    h, a = f["h0"], torch.exp(la)
    for i in range(300):
        h = a[:, i] * h + b[:, i]
        err = np.abs(h.double().numpy() - y[:, i]) / room[:, i]
        assert err.max() < 1
    # and are no wider than 300 steps' 20 roundings of magnitudes below 30 add up to
    assert room.max() < 300 * 20 * 2.0 ** -24 * 30
