"""The gated delta rule where there are heads enough for blocks of two and four
wave pairs (one takes 16 columns of a head), in whole walks, in segments and in
the backward's; rows of different lengths, empty ones among them. Tolerances as
in test_gpu_gated_delta.py and test_gpu_gated_delta_bwd.py.
"""

import numpy as np
import pytest
import torch

from tests.test_gpu_gated_delta import TOL, close, host, oracle_fwd, problem, run
from tests.test_gpu_gated_delta_bwd import compare, reference, seeds
from tests.test_gpu_gated_delta_bwd import run as run_bwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")


# 256 heads of 4 slices (four pairs), 128 of 4 (two), 128 of 5 (four, three of the second
# block's idle), 256 of 2, the second with four columns (two)
SIZES = [(16, 100, 8, 16, 32, 64), (8, 130, 4, 16, 100, 64), (8, 100, 16, 16, 24, 80), (16, 70, 16, 16, 128, 20)]


def lengths(B, L, seed):
    lens = torch.randint(0, L + 1, (B,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)
    lens[1], lens[2], lens[3], lens[4] = 0, L, 64, 65
    return lens


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES)
def test_forward(size, dtype):
    p = problem(*size, dtype, 31)
    lens = lengths(size[0], size[1], 5)
    ref, href = oracle_fwd(p, seqlens=lens.numpy())
    for out in (torch.float32, torch.bfloat16):
        y, h = run(p, out_dtype=out, seqlens=lens.cuda())
        close(f"{size} {dtype} y {out}", y, ref)
        close(f"{size} {dtype} h", h, href)
        for b in range(size[0]):
            assert not y[b, int(lens[b]):].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", SIZES)
def test_gradients(size, dtype):
    p = problem(*size, dtype, 33)
    lens = lengths(size[0], size[1], 6)
    dy, dh = seeds(p, 34)
    ref = reference(p, dy, dh, seqlens=lens.numpy())
    got = run_bwd(p, dy, dh, seqlens=lens.cuda())
    compare(f"{size} {dtype}", got, ref)
    again = run_bwd(p, dy, dh, seqlens=lens.cuda())
    for x in got:
        assert torch.equal(got[x], again[x]), x


def one_half_terms(p):
    """[L, H, P]: what a bfloat16 y's two products sum in absolute value, from
    y_t = scale e^(c_t) q_t . S + sum_s Pm[t,s] e_s with S the state at the start
    of t's 64 steps. In one half an operand is off by at most 2^-12 of itself, a
    product of two by 2^-11 (and 2^-24), their sum by as much of this sum.
    (test_gpu_gated_delta.py allows 2^-11 of the largest y, as errors of random
    sign come to; here 8 million elements, sums of no more than 80 products each,
    reach past that.)"""
    f = host(p)
    L, H, P = f["v"].shape[1:]
    N = f["q"].shape[-1]
    rep = H // f["q"].shape[2]
    unit = lambda a: np.repeat(a / np.sqrt((a * a).sum(-1, keepdims=True) + 1e-6), rep, 1)  # noqa: E731
    q, k, v = unit(f["q"][0]), unit(f["k"][0]), f["v"][0]
    ld = np.logaddexp(0.0, f["dt"][0] + f["dt_bias"]) * f["A"]
    beta = 1 / (1 + np.exp(-f["beta"][0]))
    S, out = f["h0"][0].copy(), np.zeros((L, H, P))  # S [H, P, N]
    for t0 in range(0, L, 64):
        t1 = min(t0 + 64, L)
        first, c, e = np.abs(S), np.cumsum(ld[t0:t1], 0), np.zeros((t1 - t0, H, P))
        for t in range(t0, t1):
            S = S * np.exp(ld[t])[:, None, None]
            e[t - t0] = v[t] - (S * k[t][:, None]).sum(-1)
            S = S + (beta[t][:, None] * e[t - t0])[..., None] * k[t][:, None]
        for h in range(H):
            low = np.tril(np.exp(np.minimum(c[:, None, h] - c[None, :, h], 0)))
            pm = low * np.abs(q[t0:t1, h] @ k[t0:t1, h].T) * beta[None, t0:t1, h]
            out[t0:t1, h] = np.exp(c[:, h])[:, None] * (np.abs(q[t0:t1, h]) @ first[h].T) + pm @ np.abs(e[:, h])
    return N ** -0.5 * out


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_segments_of_several_pairs(dtype):
    p = problem(1, 8192, 4, 16, 16, 64, dtype, 35)
    p["dt_bias"] = torch.full((16,), -7.0, device="cuda")
    ref, href = oracle_fwd(p)
    y, h = run(p, out_dtype=torch.float32)
    close(f"segments {dtype} y", y, ref, tol=2 * TOL)   # the map's products and the walk's
    close(f"segments {dtype} h", h, href, tol=2 * TOL)
    y, h = run(p, out_dtype=torch.bfloat16)
    close(f"segments {dtype} h", h, href, tol=2 * TOL)
    room = 2.0**-8 * np.abs(ref[0]) + 2.0**-11 * (1 + 2.0**-10) * one_half_terms(p) + 2 * TOL * np.abs(ref).max()
    worst = float((np.abs(y[0].double().cpu().numpy() - ref[0]) / room).max())
    print(f"[parity] segments {dtype} y in bfloat16: {worst:.3f} of the tolerance", flush=True)
    assert worst <= 1.0


def test_steps_far_apart():
    """Rows 2^20 elements apart, 4.4e9 elements in all: the same results as from dense arrays, to the bit."""
    L, step = 4200, 1 << 20
    p = problem(1, L, 1, 1, 32, 16, "bf16", 36)
    wide = torch.empty(1, L, step, dtype=torch.bfloat16, device="cuda")
    far = dict(p)
    for x, at in (("q", 8), ("k", step // 2), ("v", step - 16)):
        n = p[x].shape[-1]
        wide[:, :, at:at + n] = p[x][:, :, 0]
        far[x] = wide[:, :, at:at + n].unflatten(-1, (1, n))
    for a, b in zip(run(far), run(p)):
        assert torch.equal(a, b)
    dy, dh = seeds(p, 37)
    dense, strided = run_bwd(p, dy, dh), run_bwd(far, dy, dh)
    for x in dense:
        assert torch.equal(dense[x], strided[x]), x
