"""Long sequences of the gated delta rule: in segments without an initial state and
in a workspace full of NaN, and the gradients of thousands of steps against the
float64 oracle.

Tolerances. The maps of the steps shrink (strengths of a sigmoid, unit keys), so
that errors add over the steps that the state remembers, here about a thousand:
16 chunks of 1.1e-5 each (test_gpu_gated_delta.py), of random sign, 4.4e-5 of the
largest element, and twice that for a gradient, within 5e-5 and 1e-4.
"""

import pytest
import torch

from selective_state_space_87_amd import binding
from tests.test_gpu_gated_delta import close, oracle_fwd, problem, run
from tests.test_gpu_gated_delta_bwd import compare, reference, seeds
from tests.test_gpu_gated_delta_bwd import run as run_bwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")


def slow(B, L, G, H, N, P, dtype, seed):
    p = problem(B, L, G, H, N, P, dtype, seed)
    p["dt_bias"] = torch.full((H,), -7.0, device="cuda")
    return p


def nan_workspace(of, p):
    B, L, G, N = p["q"].shape
    n = of(B, L, G, p["v"].shape[2], p["v"].shape[3], N, p["q"].dtype)
    return torch.full((n,), 255, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("given", [True, False])
@pytest.mark.parametrize("L,G,H,N,P,lens", [(4096, 1, 1, 16, 33, [4096, 2049, 0, 1]), (2304, 1, 2, 64, 40, [2304, 500]),
                                            (4200, 1, 1, 100, 16, [4199])])
def test_segments_with_and_without_a_state(L, G, H, N, P, lens, given, dtype):
    p = slow(len(lens), L, G, H, N, P, dtype, 81)
    if not given:
        p["h0"] = None
    seq = torch.tensor(lens, dtype=torch.int32)
    ref, href = oracle_fwd(p, seqlens=seq.numpy())
    y, h = run(p, out_dtype=torch.float32, seqlens=seq.cuda(),
               workspace=nan_workspace(binding.ssm_gated_delta_workspace_bytes, p))
    close(f"segments {(L, G, H, N, P)} {dtype} y", y, ref, tol=1e-4)   # the map's products and the walk's
    close(f"segments {(L, G, H, N, P)} {dtype} h", h, href, tol=1e-4)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,L,G,H,N,P,lens", [(2, 3000, 1, 2, 32, 16, [3000, 1777]), (1, 4096, 1, 1, 100, 20, None)])
def test_gradients_of_thousands_of_steps(B, L, G, H, N, P, lens, dtype):
    p = slow(B, L, G, H, N, P, dtype, 82)
    dy, dh = seeds(p, 83)
    seq = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    ref = reference(p, dy, dh, seqlens=None if seq is None else seq.numpy())
    got = run_bwd(p, dy, dh, seqlens=None if seq is None else seq.cuda(),
                  workspace=nan_workspace(binding.ssm_gated_delta_bwd_workspace_bytes, p))
    compare(f"{(B, L, G, H, N, P)} {dtype}", got, ref)


def test_captured_gradients():
    """Replayed beside eager work, every replay as the eager call to the bit."""
    p = slow(2, 700, 2, 4, 64, 48, "bf16", 84)
    dy, dh = seeds(p, 85)
    want = run_bwd(p, dy, dh)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run_bwd(p, dy, dh)
    for rep in range(3):
        for x in got.values():
            x.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        for x in want:
            assert torch.equal(got[x], want[x]), (x, rep)
        again = run_bwd(p, dy, dh)
        torch.empty(1 << 24, dtype=torch.uint8, device="cuda").fill_(rep)
        torch.cuda.synchronize()
        assert all(torch.equal(again[x], want[x]) for x in want)
