"""Pins of the convolution's gradients in the oracle: differences of the
forward oracle, torch's automatic differentiation of its own convolution."""

import numpy as np
import pytest
import torch

import oracle


@pytest.mark.parametrize("K,L,silu,carried", [(1, 4, True, False), (3, 5, True, True), (4, 2, True, True),
                                              (4, 6, False, False), (8, 3, True, True), (2, 1, False, True),
                                              (4, 0, True, True)])
def test_against_differences(K, L, silu, carried):
    rng = np.random.default_rng(K * 10 + L)
    B, d = 2, 3
    x, w, b = rng.standard_normal((B, L, d)), rng.standard_normal((d, K)), rng.standard_normal(d)
    st = rng.standard_normal((B, d, K - 1)) if carried else None
    dy, dst = rng.standard_normal((B, L, d)), rng.standard_normal((B, d, K - 1))

    def loss():
        y, out = oracle.causal_conv1d(x, w, b, silu, st)
        return (y * dy).sum() + (out * dst).sum()

    got = oracle.causal_conv1d_bwd(x, w, dy, b, silu, st, dst)
    for name, v in (("dx", x), ("dweight", w), ("dbias", b), ("dstate_in", st)):
        if v is None:
            continue
        for i in np.ndindex(v.shape):
            keep = v[i]
            v[i] = keep + 1e-6
            up = loss()
            v[i] = keep - 1e-6
            down = loss()
            v[i] = keep
            assert abs((up - down) / 2e-6 - got[name][i]) < 1e-7, (name, i)


def test_against_automatic_differentiation():
    rng = np.random.default_rng(3)
    B, L, d, K = 2, 9, 5, 4
    x, w, b, dy = (torch.tensor(rng.standard_normal(s), requires_grad=True) for s in ((B, L, d), (d, K), (d,), (B, L, d)))
    y = torch.nn.functional.conv1d(x.transpose(1, 2), w[:, None], b, padding=K - 1, groups=d)[..., :L].transpose(1, 2)
    grads = torch.autograd.grad(torch.nn.functional.silu(y), (x, w, b), dy)
    got = oracle.causal_conv1d_bwd(*(t.detach().numpy() for t in (x, w, dy, b)))
    for name, g in zip(("dx", "dweight", "dbias"), grads):
        assert np.allclose(got[name], g.numpy(), rtol=0, atol=1e-13)
