"""Pins of the layer norm's and the dropout's oracles by something other than
themselves: published values, closed forms, differences, moments."""

import numpy as np
import pytest

import oracle


def test_generator_gives_its_published_values():
    # the known answers published with the generator
    full = 2 ** 32 - 1
    for counter, key, want in (([0] * 4, (0, 0), "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
                               ([full] * 4, (full, full), "408f276d 41c83b0e a20bc7c6 6d5451fd")):
        got = oracle.philox4x32(np.array(counter, np.uint64), key)
        assert " ".join(f"{int(w):08x}" for w in got) == want


def test_bits_do_not_depend_on_where_a_piece_starts():
    whole = oracle.dropout_bits(0, 100, 7, 8, 9)
    for first in (0, 1, 5, 8, 13):
        assert (oracle.dropout_bits(first, 60, 7, 8, 9) == whole[first:first + 60]).all()
    far = oracle.dropout_bits(2 ** 36 + 3, 4, 7, 8, 9)  # the counter's second word
    assert (far != oracle.dropout_bits(3, 4, 7, 8, 9)).any()
    for other in ((8, 8, 9), (7, 9, 9), (7, 8, 10), (7 + 2 ** 32, 8, 9)):
        assert (oracle.dropout_bits(0, 100, *other) != whole).sum() > 90


@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 1.0])
def test_shares(p):
    n = 1 << 17
    x = oracle.dropout(np.ones(n, np.float32), p, 3, 4, 5)
    share = oracle.dropout_threshold(p) / 65536
    # six standard deviations of a binomial share
    assert abs((x == 0).mean() - share) <= 6 * np.sqrt(share * (1 - share) / n)
    if p < 1:
        assert set(np.unique(x)) <= {0.0, np.float32(1 / (1 - share))}


def test_halves_of_words_are_not_alike():
    b = oracle.dropout_bits(0, 1 << 15, 1, 2, 3).reshape(-1, 8) / 65536 - 0.5
    c = b.T @ b / len(b) * 12
    assert np.abs(c - np.eye(8)).max() < 6 / np.sqrt(len(b))


def test_layer_norm_closed_forms():
    rng = np.random.default_rng(1)
    s = rng.standard_normal((5, 40))
    y = oracle.layer_norm(s, eps=0.0)
    assert np.allclose(y.mean(-1), 0, atol=1e-14) and np.allclose((y ** 2).mean(-1), 1)
    assert np.allclose(oracle.layer_norm(3 * s + 7, eps=0.0), y)          # shift and scale leave it
    w, b = rng.standard_normal(40), rng.standard_normal(40)
    assert np.allclose(oracle.layer_norm(s, w, b, eps=0.0), y * w + b)
    assert np.allclose(oracle.layer_norm(np.array([[1.0, 3.0]]), eps=3.0), [[-0.5, 0.5]])
    assert np.allclose(oracle.layer_norm(s[:, :1], eps=1e-5), 0)
    centred = s - s.mean(-1, keepdims=True)
    assert np.allclose(oracle.layer_norm(s, w), oracle.rms_norm(centred, w))


def test_layer_norm_gradients_by_differences():
    rng = np.random.default_rng(2)
    s, dy, dr, w = (rng.standard_normal(x) for x in ((3, 7), (3, 7), (3, 7), 7))
    b = rng.standard_normal(7)

    def loss(s, w, b):
        return (oracle.layer_norm(s, w, b, 1e-2) * dy).sum() + (s * dr).sum()

    ds, dw, db = oracle.layer_norm_bwd(s, w, dy, dr, 1e-2)
    for x, d in ((s, ds), (w, dw), (b, db)):
        for i in np.ndindex(x.shape):
            keep = x[i]
            x[i] = keep + 1e-6
            up = loss(s, w, b)
            x[i] = keep - 1e-6
            down = loss(s, w, b)
            x[i] = keep
            assert abs((up - down) / 2e-6 - d[i]) < 1e-7
