"""CPU pins of the gated delta rule's and the RMS norm's float64 oracles:
hand-worked steps, limits in which they become something simpler, and the
gradients against central differences."""

import numpy as np
import pytest

import oracle


def problem(B, L, G, H, N, P, seed, **over):
    r = np.random.default_rng(seed)
    p = dict(q=r.standard_normal((B, L, G, N)), k=r.standard_normal((B, L, G, N)), v=r.standard_normal((B, L, H, P)),
             dt=r.standard_normal((B, L, H)), A=-np.exp(r.standard_normal(H)), beta=r.standard_normal((B, L, H)))
    p.update(over)
    return p


def test_one_step_by_hand():
    # S = [[1, 2]] (P = 1, N = 2), decay 1/2, k = (1, 0), q = (1, 1), v = 3, beta = 1/2:
    # S' = (0.5, 1), e = 3 - 0.5 = 2.5, S = (0.5 + 1.25, 1), y = 2.75
    y, S = oracle.gated_delta(np.array([1.0, 1.0]).reshape(1, 1, 1, 2), np.array([1.0, 0.0]).reshape(1, 1, 1, 2),
                              np.full((1, 1, 1, 1), 3.0), np.full((1, 1, 1), np.log(2.0)), np.array([-1.0]),
                              np.full((1, 1, 1), 0.5), h0=np.array([1.0, 2.0]).reshape(1, 1, 1, 2))
    assert np.allclose(y, 2.75) and np.allclose(S.ravel(), [1.75, 1.0])


def test_full_write_makes_the_key_answer_the_value():
    p = problem(1, 6, 1, 1, 8, 5, 1, beta=np.ones((1, 6, 1)))
    _, S = oracle.gated_delta(**p, l2norm=True)
    k = p["k"][0, -1, 0]
    k = k / np.sqrt((k ** 2).sum() + 1e-6)
    assert np.allclose(S[0, 0] @ k, p["v"][0, -1, 0], atol=1e-5)


def test_zero_writes_leave_a_decayed_state():
    p = problem(2, 5, 1, 2, 4, 3, 2, beta=np.zeros((2, 5, 2)))
    h0 = np.random.default_rng(3).standard_normal((2, 2, 3, 4))
    _, S = oracle.gated_delta(**p, h0=h0)
    a = np.exp(np.maximum(p["dt"] * p["A"], -200.0)).prod(1)
    assert np.allclose(S, h0 * a[..., None, None])


def test_orthogonal_keys_write_as_plain_sums():
    # with orthonormal keys and no decay nothing is taken off: S = sum k v^T
    L = N = 4
    p = problem(1, L, 1, 1, N, 3, 4, k=np.eye(4).reshape(1, 4, 1, 4), dt=np.zeros((1, 4, 1)), beta=np.ones((1, 4, 1)))
    _, S = oracle.gated_delta(**p)
    assert np.allclose(S[0, 0], np.einsum("lp,ln->pn", p["v"][0, :, 0], p["k"][0, :, 0]))


def test_steps_behind_a_row_change_nothing():
    p = problem(2, 7, 1, 2, 4, 3, 5)
    n = np.array([3, 7])
    y, S = oracle.gated_delta(**p, seqlens=n, softplus=True, sigmoid=True)
    cut = {x: (a[:1, :3] if a.ndim > 1 else a) for x, a in p.items()}
    y3, S3 = oracle.gated_delta(**cut, softplus=True, sigmoid=True)
    assert np.allclose(y[0, :3], y3[0]) and not y[0, 3:].any() and np.allclose(S[0], S3[0])


@pytest.mark.parametrize("l2norm,gates,lens", [(True, True, None), (False, False, None), (True, True, [2, 5])])
def test_gradients_against_differences(l2norm, gates, lens):
    p = problem(2, 5, 2, 4, 3, 2, 6)
    if not gates:
        p["dt"], p["beta"] = np.abs(p["dt"]), 0.3 + 0.1 * p["beta"]
    r = np.random.default_rng(7)
    p["dt_bias"], p["h0"] = 0.1 * r.standard_normal(4), r.standard_normal((2, 4, 2, 3))
    dy, dh = r.standard_normal((2, 5, 4, 2)), r.standard_normal((2, 4, 2, 3))
    kw = dict(softplus=gates, sigmoid=gates, l2norm=l2norm, scale=0.7, seqlens=lens)

    def loss(**q):
        y, S = oracle.gated_delta(**q, **kw)
        return (dy * y).sum() + (dh * S).sum()

    g = oracle.gated_delta_bwd(**{x: a for x, a in p.items()}, dy=dy, dh_final=dh, **kw)
    for name in ("q", "k", "v", "dt", "A", "beta", "dt_bias", "h0"):
        got = g["d" + name]
        assert got.shape == p[name].shape
        for i in r.choice(p[name].size, min(6, p[name].size), replace=False):
            d = []
            for h in (1e-5, -1e-5):
                a = p[name].copy()
                a.ravel()[i] += h
                d.append(loss(**dict(p, **{name: a})))
            # a central difference is off by its third-order term (h^2) and by
            # the loss's rounding over 2h: about 1e-9 relative here
            assert np.isclose(got.ravel()[i], (d[0] - d[1]) / 2e-5, rtol=1e-6, atol=1e-7), name


def test_norm_by_hand_and_gradients():
    assert np.allclose(oracle.rms_norm(np.array([[3.0, 4.0]]), eps=0.0), np.array([[3.0, 4.0]]) / np.sqrt(12.5))
    r = np.random.default_rng(8)
    s, w, dy, dr = r.standard_normal((3, 5)), r.standard_normal(5), r.standard_normal((3, 5)), r.standard_normal((3, 5))
    ds, dw = oracle.rms_norm_bwd(s, w, dy, dr)
    f = lambda s, w: (dy * oracle.rms_norm(s, w)).sum() + (dr * s).sum()  # noqa: E731
    for i in range(15):
        d = np.zeros(15)
        d[i] = 1e-5
        d = d.reshape(3, 5)
        assert np.isclose(ds.ravel()[i], (f(s + d, w) - f(s - d, w)) / 2e-5, rtol=1e-6, atol=1e-8)
    for i in range(5):
        d = np.zeros(5)
        d[i] = 1e-5
        assert np.isclose(dw[i], (f(s, w + d) - f(s, w - d)) / 2e-5, rtol=1e-6, atol=1e-8)


def test_e4m3_values():
    x = np.array([0.0, 448.0, -448.0, 1.0625, 1.1875, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -10, 17.0])
    assert np.array_equal(oracle.e4m3_nearest(x), [0.0, 448.0, -448.0, 1.0, 1.25, 2.0 ** -9, 0.0, 2.0 ** -8, 16.0])
