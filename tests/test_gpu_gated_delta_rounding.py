"""A bfloat16 y of the gated delta rule is the float32 y rounded once, however
the walk over the chunks is laid out: the two calls take the same products and
sums, so that nothing but the last rounding may differ. And against the float64
oracle: half a step of the value, 2^-8, beside what a float32 y is allowed on
the scale of the largest element (test_gpu_gated_delta.py), where q^T S and the
chunk's own sum cancel too.
"""

import numpy as np
import pytest
import torch

from tests.test_gpu_gated_delta import TOL, oracle_fwd, problem, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")


# the recurrence; one, two and four pairs of waves a block (a slice is 16 of P's
# columns: 8 of them, 128 heads of 2, 256 heads of 4 and of 5); two walks in segments
SIZES = [(2, 7, 1, 2, 32, 24), (1, 333, 2, 4, 128, 32), (8, 100, 8, 16, 128, 32), (16, 130, 4, 16, 64, 64),
         (16, 70, 16, 16, 128, 80), (1, 4096, 1, 2, 100, 40), (1, 8192, 4, 16, 16, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES)
def test_a_bfloat16_y_is_the_float32_y_rounded(size, dtype):
    B, L = size[:2]
    p = problem(*size, dtype, 61)
    lens = torch.randint(1, L + 1, (B,), generator=torch.Generator().manual_seed(7), dtype=torch.int32)
    lens[0] = L
    full, h = run(p, out_dtype=torch.float32, seqlens=lens.cuda())
    half, h2 = run(p, out_dtype=torch.bfloat16, seqlens=lens.cuda())
    assert torch.equal(h, h2)
    unequal = int((full.bfloat16() != half).sum())
    print(f"{size} {dtype}: {unequal} of {half.numel()} elements", flush=True)
    assert unequal == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_a_bfloat16_y_whose_two_sums_cancel(dtype):
    """Every query and key is one unit row u, every write of full strength, and no
    step forgets: y_t is v_t, while h0 holds 1000 u in every row of the state, so
    that scale q^T S is 1000 and the chunk's own sum takes it out again."""
    p = problem(1, 64, 1, 1, 64, 64, dtype, 62, raw=False)
    u = p["k"][:, :1].clone()
    p["q"], p["k"] = u.expand(-1, 64, -1, -1).contiguous(), u.expand(-1, 64, -1, -1).contiguous()
    p["A"] = torch.zeros(1, device="cuda")
    p["beta"] = torch.ones_like(p["beta"])
    p["h0"] = 1000.0 * u[0, 0].float().expand(64, 64).reshape(1, 1, 64, 64).contiguous()
    ref, _ = oracle_fwd(p, raw=False, scale=1.0)
    y, _ = run(p, raw=False, scale=1.0, out_dtype=torch.bfloat16)
    assert np.abs(ref).max() < 20.0  # (a bfloat16 u has a norm of 1 to 2^-8: what is left of h0 in y_0)
    # float32's allowance, on the scale of what cancels
    room = 2.0**-8 * np.abs(ref) + TOL * 1000.0
    worst = float((np.abs(y.double().cpu().numpy() - ref) / room).max())
    print(f"{dtype}: {worst:.3f} of the tolerance", flush=True)
    assert worst <= 1.0
