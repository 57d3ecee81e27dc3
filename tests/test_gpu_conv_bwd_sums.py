"""How the convolution's gradients of the filters are added up over the steps.

Small whole numbers, without the activation: a segment's sums (at most 512 steps of
products up to 2^14) stay below 2^24 and are exact in float32 however they are ordered.
Joined in double they stay exact, and each result is the true sum rounded once.
"""

import numpy as np
import pytest
import torch

from selective_state_space_87_amd import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")


@pytest.mark.parametrize("B,L,d,K", [(2, 40000, 5, 4), (1, 300000, 3, 2), (7, 9001, 260, 3), (1, 70000, 1, 8)])
@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
def test_long_sums_are_rounded_once(B, L, d, K, xt):
    g = torch.Generator().manual_seed(L)
    x = torch.randint(0, 16, (B, L, d), generator=g)
    dy = torch.randint(0, 1024, (B, L, d), generator=g)
    xe = torch.cat([torch.zeros(B, K - 1, d, dtype=torch.int64), x], 1)
    dw = torch.stack([(dy * xe[:, k:k + L]).sum((0, 1)) for k in range(K)], -1)
    got = binding.ssm_causal_conv1d_bwd(x.to(xt).cuda(), torch.ones(d, K, device="cuda"), dy.float().cuda(),
                                        bias=torch.zeros(d, device="cuda"), silu_activation=False)
    assert (dw > 2 ** 24).all()
    assert np.array_equal(got["dweight"].cpu().numpy(), dw.numpy().astype(np.float32))
    assert np.array_equal(got["dbias"].cpu().numpy(), dy.sum((0, 1)).numpy().astype(np.float32))


@pytest.mark.parametrize("L,d,K", [(1 << 20, 4, 4), (1 << 20, 3, 1), (1 << 20, 5, 8)])
def test_sums_of_one_sign_do_not_drift(L, d, K):
    """One value at every step, in segments of 512: added step by step in float32 the sum is off by 126 roundings.
    A segment's takes 8 or fewer for a group of steps, as many for what is left of groups, and one for each of at most
    66 groups; the parts are joined in double and rounded once: 76."""
    value = np.float32(1.944)
    x = torch.ones(1, L, d, device="cuda")
    dy = torch.full((1, L, d), float(value), device="cuda")
    got = binding.ssm_causal_conv1d_bwd(x, torch.ones(d, K, device="cuda"), dy, bias=torch.zeros(d, device="cuda"),
                                        silu_activation=False)
    for k in range(K):
        want = float(value) * (L - (K - 1 - k))
        assert float((got["dweight"][:, k].double() - want).abs().max()) <= 76 * 2.0 ** -24 * want
    assert float((got["dbias"].double() - float(value) * L).abs().max()) <= 76 * 2.0 ** -24 * float(value) * L
