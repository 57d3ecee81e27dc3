"""Gradients of the gates: strengths whose sigmoid is saturated."""

import numpy as np
import pytest
import torch

from tests.test_gpu_gated_delta import problem
from tests.test_gpu_gated_delta_bwd import TOL, reference, run, seeds

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_saturated_strengths(sign, dtype):
    """Every raw strength in 8 .. 20 (or -20 .. -8): its derivative b (1 - b) falls
    from 3e-4 to 2e-9, and each element is held to the tolerance of a gradient in
    units of its own. (The factor itself: e^x of |x| <= 20 in base 2 rounds an
    exponent of 29 to 2^-20, e^x to 1e-6 of itself.)"""
    p = problem(2, 150, 1, 2, 64, 48, dtype, 71)
    p["beta"] = (sign * (8.0 + 12.0 * torch.rand(p["beta"].shape, generator=torch.Generator().manual_seed(8)))).to(
        p["beta"].dtype).cuda()
    dy, dh = seeds(p, 72)
    ref = reference(p, dy, dh)["dbeta"]
    got = run(p, dy, dh)["dbeta"].double().cpu().numpy()
    x = np.abs(p["beta"].double().cpu().numpy())
    unit = np.exp(-x) / (1.0 + np.exp(-x)) ** 2
    worst = float(np.abs((got - ref) / unit).max() / (TOL * np.abs(ref / unit).max()))
    print(f"dbeta at {sign:+.0f} x 8 .. 20, {dtype}: {worst:.3f} of the tolerance", flush=True)
    assert worst <= 1.0
