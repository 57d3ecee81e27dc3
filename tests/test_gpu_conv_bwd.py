"""GPU parity of the causal convolution's gradients with the float64 oracle,
through the C ABI.

Tolerances. The value z before the activation is a float32 sum of K + 1 <= 9 terms:
off by 10 2^-24 m, m = |bias| + sum |w x|. silu' changes by half of that at most, and its
own evaluation (the exponential of z, off by (|z| + 3) 2^-24 of itself, a
reciprocal, four products; |z s (1 - s)| <= 0.28) by 20 2^-24: g is off by
|dy| (20 + 5 m) 2^-24, and by half a rounding of itself more. dx adds K <= 8 products of
it, dstate_out one more: 10 2^-24 of their magnitudes. dweight and dbias add up
to 512 steps one after the other, then parts of sixteen at a time: 600 2^-24 of the
terms' magnitudes.
"""

import numpy as np
import pytest
import torch

import oracle
from selective_state_space_87_amd import binding

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16}
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def inputs(B, L, d, K, xt="f32", seed=0, carried=True, scale=1.0):
    g = torch.Generator().manual_seed(seed + 100 * L + d + K)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    t = dict(x=(scale * rn(B, L, d)).to(T[xt]), weight=rn(d, K) * K ** -0.5, dy=rn(B, L, d), bias=0.3 * rn(d),
             state_in=rn(B, d, K - 1), dstate_out=rn(B, d, K - 1))
    if not carried:
        t["state_in"] = t["dstate_out"] = None
    return {k: None if v is None else v.cuda() for k, v in t.items()}


def check(got, t, silu):
    f = {k: np64(v) for k, v in t.items()}
    ref = oracle.causal_conv1d_bwd(f["x"], f["weight"], f["dy"], f["bias"], silu, f["state_in"], f["dstate_out"])
    a = {k: None if v is None else np.abs(v) for k, v in f.items()}
    m = oracle.causal_conv1d(a["x"], a["weight"], a["bias"], False, a["state_in"])[0]
    off = (a["dy"] * (20 + 5 * m) if silu else 0 * m) * E + E * np.abs(ref["g"])
    zero = np.zeros_like(f["weight"][:, 0])
    # the magnitudes of the sums, and what g's error makes of them
    mag = oracle.causal_conv1d_bwd(a["x"], a["weight"], np.abs(ref["g"]), zero, False, a["state_in"], a["dstate_out"])
    room = oracle.causal_conv1d_bwd(a["x"], a["weight"], off, zero, False, a["state_in"], None)
    for name, v in got.items():
        terms = 600 if name in ("dweight", "dbias") else 10
        err = np.abs(np64(v) - ref[name])
        most = room[name] + terms * E * mag[name] + 1e-30
        assert v.shape == err.shape and (err <= most).all(), (name, float((err / most).max()))


SHAPES = [(1, 1, 1, 1), (2, 1, 5, 4), (1, 2, 4, 4), (2, 3, 8, 4), (1, 31, 7, 3), (3, 32, 64, 4), (2, 33, 65, 2),
          (1, 100, 130, 8), (2, 777, 33, 3), (1, 64, 1028, 4), (4, 129, 300, 5), (1, 40, 12, 6), (2, 50, 9, 7),
          (1, 2100, 16, 4), (700, 70, 8, 4)]


@pytest.mark.parametrize("B,L,d,K", SHAPES)
@pytest.mark.parametrize("xt,silu,carried", [("f32", True, True), ("bf16", True, False), ("bf16", False, True),
                                             ("f32", False, False)])
def test_gradients(B, L, d, K, xt, silu, carried):
    t = inputs(B, L, d, K, xt, carried=carried)
    got = binding.ssm_causal_conv1d_bwd(**t, silu_activation=silu)
    assert set(got) == {"dx", "dweight", "dbias", "dstate_in"}
    check(got, t, silu)
    again = binding.ssm_causal_conv1d_bwd(**t, silu_activation=silu)
    assert all(torch.equal(got[k], again[k]) for k in got)


def test_every_width_at_every_short_length():
    for K in range(1, 9):
        for L in (0, 1, K - 1, K, K + 1, 2 * K, 32 + K):
            for d in (3, 8):
                t = inputs(2, max(L, 0), d, K, seed=7)
                check(binding.ssm_causal_conv1d_bwd(**t), t, True)


def test_wide_values_reach_the_ends_of_the_activation():
    # |z| up to about 300: the exponential overflows on one side, the derivative is 0 or 1
    t = inputs(1, 64, 16, 4, seed=1, scale=100.0)
    check(binding.ssm_causal_conv1d_bwd(**t), t, True)


def test_long_rows_walked_in_segments_of_512():
    t = inputs(2, 5000, 2052, 4, "bf16", seed=2)
    got = binding.ssm_causal_conv1d_bwd(**t)
    some = [0, 1, 1000, 2051]
    part = {k: None if v is None else (v[some] if k in ("weight", "bias") else
                                       v[:, some] if "state" in k else v[..., some]).contiguous() for k, v in t.items()}
    cut = {k: v[some] if k in ("dweight", "dbias") else v[:, some] if k == "dstate_in" else v[..., some]
           for k, v in got.items()}
    check(cut, part, True)


def test_without_a_bias_and_of_nothing():
    t = inputs(2, 40, 12, 4, carried=False)
    t["bias"] = None
    got = binding.ssm_causal_conv1d_bwd(**t)
    assert set(got) == {"dx", "dweight", "dstate_in"}
    t["bias"] = torch.zeros(12, device="cuda")
    want = binding.ssm_causal_conv1d_bwd(**t)
    assert all(torch.equal(got[k], want[k]) for k in got)
    t = inputs(0, 40, 12, 4)
    got = binding.ssm_causal_conv1d_bwd(**t)
    assert got["dx"].shape == (0, 40, 12) and not got["dweight"].any() and not got["dbias"].any()


def test_pieces_of_a_sequence_chain_through_the_state():
    """Gradients of two pieces, the state's gradient carried from the second
    to the first, are those of the whole."""
    B, L, d, K, cut = 2, 90, 20, 4, 41
    t = inputs(B, L, d, K, seed=5)
    whole = binding.ssm_causal_conv1d_bwd(**t)
    one = {**t, "x": t["x"][:, :cut].contiguous(), "dy": t["dy"][:, :cut].contiguous()}
    _, mid = binding.ssm_causal_conv1d_fwd(one["x"], t["weight"], t["bias"], state_in=t["state_in"],
                                           return_final_state=True)
    two = {**t, "x": t["x"][:, cut:].contiguous(), "dy": t["dy"][:, cut:].contiguous(), "state_in": mid}
    g2 = binding.ssm_causal_conv1d_bwd(**two)
    g1 = binding.ssm_causal_conv1d_bwd(**{**one, "dstate_out": g2["dstate_in"]})
    # a term of dx may be added in another order: 20 roundings of sums of some 8 terms below 4
    assert torch.allclose(torch.cat([g1["dx"], g2["dx"]], 1), whole["dx"], rtol=0, atol=20 * E * 32)
    assert torch.allclose(g1["dstate_in"], whole["dstate_in"], rtol=0, atol=20 * E * 32)
    # sums of 180 terms below 16
    for k in ("dweight", "dbias"):
        assert torch.allclose(g1[k] + g2[k], whole[k], rtol=0, atol=180 * 16 * 20 * E)


def test_not_finite_inputs_stay_with_their_window():
    t = inputs(1, 96, 8, 3, seed=6)
    want = binding.ssm_causal_conv1d_bwd(**t)
    t["x"][0, 50, 2] = float("nan")
    t["x"][0, 20, 5] = float("inf")
    got = binding.ssm_causal_conv1d_bwd(**t)
    # out[l] sees x[l-2 .. l]; dx[l] sees g[l .. l+2]
    keep = torch.ones(96, 8, dtype=torch.bool)
    keep[48:53, 2] = False
    keep[18:23, 5] = False
    assert torch.equal(got["dx"][0].cpu()[keep], want["dx"][0].cpu()[keep])
    assert got["dx"][0, 50, 2].isnan()


def test_side_stream_and_captured():
    t = inputs(2, 300, 64, 4, "bf16", seed=8)
    want = binding.ssm_causal_conv1d_bwd(**t)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = binding.ssm_causal_conv1d_bwd(**t, stream=side)
    side.synchronize()
    assert all(torch.equal(got[k], want[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = binding.ssm_causal_conv1d_bwd(**t)
    for i in range(3):
        t["dy"].normal_()
        graph.replay()
        torch.cuda.synchronize()
        want = binding.ssm_causal_conv1d_bwd(**t)
        assert all(torch.equal(got[k], want[k]) for k in want)


def test_refusals():
    t = inputs(2, 16, 8, 4)
    for kw in (dict(weight=t["weight"][:5]), dict(dy=None), dict(dy=t["dy"].bfloat16()), dict(bias=t["bias"][:3]),
               dict(state_in=t["state_in"][:1]), dict(dstate_out=t["dstate_out"][..., :2]),
               dict(dx=t["dy"][:1]), dict(x=t["x"].half()), dict(x=t["x"].cpu()), dict(x=t["x"].transpose(0, 1))):
        with pytest.raises(ValueError):
            binding.ssm_causal_conv1d_bwd(**{**t, **kw})
    for kw, status in ((dict(dx=t["dy"]), 6), (dict(weight=torch.ones(8, 9, device="cuda"), state_in=None,
                                                    dstate_out=None), 7)):
        with pytest.raises(binding.SSMError) as e:
            binding.ssm_causal_conv1d_bwd(**{**t, **kw})
        assert e.value.status == status
