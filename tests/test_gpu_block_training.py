"""The operators together, as a residual block's training step has them:

    s1 = drop(branch) + stream;  n = layer_norm(s1)          (fused)
    proj = n W                                                (x | gate | input gate)
    c = conv1d(x) (SiLU);  h = gated linear recurrence of c, gate, input gate
    out = drop(h) + s1                                        (dropout)

forward and backward, against float64 automatic differentiation of the formulas
with the oracle's random bits; prefill and single tokens; and the step captured.

Tolerances. Everything is float32. A projection of 48 terms is off by some 7 2^-24 of
its largest terms, the norm before it by 3e-6 of an element; the recurrence
gathers its inputs' errors over the memory of its decays (a few steps, A = -1 to -4).
So an output is off by some 30 such errors at most, 1e-4 of the largest element of
its array; gradients pass the chain twice: 3e-4.
"""

import numpy as np
import pytest
import torch

import oracle
from selective_state_space_87_amd import binding

pytestmark = pytest.mark.gpu
D, R, K, P = 48, 40, 4, 0.2
EPS = 1e-5
FORM = dict(gate_sigmoid=True, input_norm=True)


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")


def weights(seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    w = dict(norm=1 + 0.1 * rn(D), shift=0.1 * rn(D), proj=rn(D, 3 * R) * D ** -0.5, conv=rn(R, K) * 0.5,
             conv_bias=0.1 * rn(R), A=-1 - 3 * torch.rand(R, generator=g), gate_bias=rn(R), input_bias=0.5 * rn(R),
             back=rn(R, D) * R ** -0.5)
    return {k: v.cuda() for k, v in w.items()}


def inputs(B, L, seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g).cuda()  # noqa: E731
    return rn(B, L, D), rn(B, L, D), rn(B, L, D), torch.tensor([seed, 7], dtype=torch.int64, device="cuda")


def forward(w, branch, stream, rng, conv_state=None, state=None):
    n = binding.ssm_layer_norm_fwd(branch, w["norm"], w["shift"], residual=stream, eps=EPS, p=P, rng=rng, call=0)
    proj = n["y"] @ w["proj"]
    x = proj[..., :R].contiguous()
    c, conv_out = binding.ssm_causal_conv1d_fwd(x, w["conv"], w["conv_bias"], state_in=conv_state,
                                                return_final_state=True)
    h, last, states = binding.ssm_gated_linear_fwd(c, proj[..., R:2 * R], w["A"], input_gate=proj[..., 2 * R:],
                                                   gate_bias=w["gate_bias"], input_bias=w["input_bias"], h0=state,
                                                   return_final_state=True, states=True, **FORM)
    out = binding.ssm_dropout_fwd(h @ w["back"], P, rng, call=1, residual=n["residual_out"])
    return out, dict(s=n["residual_out"], y=n["y"], proj=proj, x=x, c=c, h=h, states=states, conv_out=conv_out, last=last)


def backward(w, kept, dout, rng):
    d = {}
    dback = binding.ssm_dropout_bwd(dout, P, rng, call=1)
    d["back"] = kept["h"].flatten(0, 1).t() @ dback.flatten(0, 1)
    g = binding.ssm_gated_linear_bwd(kept["c"], kept["proj"][..., R:2 * R], w["A"], dback @ w["back"].t(),
                                     input_gate=kept["proj"][..., 2 * R:], gate_bias=w["gate_bias"],
                                     input_bias=w["input_bias"], states=kept["states"], **FORM)
    d["A"], d["gate_bias"], d["input_bias"] = g["dA"], g["dgate_bias"], g["dinput_bias"]
    cv = binding.ssm_causal_conv1d_bwd(kept["x"], w["conv"], g["dx"], bias=w["conv_bias"])
    d["conv"], d["conv_bias"] = cv["dweight"], cv["dbias"]
    dproj = torch.cat([cv["dx"], g["dgate"], g["dinput_gate"]], -1)
    d["proj"] = kept["y"].flatten(0, 1).t() @ dproj.flatten(0, 1)
    ln = binding.ssm_layer_norm_bwd(kept["s"], w["norm"], dproj @ w["proj"].t(), dresidual=dout, eps=EPS, p=P, rng=rng,
                                    call=0)
    d["norm"], d["shift"], d["stream"], d["branch"] = ln["dweight"], ln["dbias"], ln["ds"], ln["dx"]
    return d


def dropped(x, rng, call):
    """x through the dropout, by the oracle's bits (differentiable)."""
    seed, step = (int(v) for v in rng.cpu())
    t = oracle.dropout_threshold(P)
    keep = torch.from_numpy(oracle.dropout_bits(0, x.numel(), seed, step, call) >= t).view(x.shape)
    return torch.where(keep, x * (65536 / (65536 - t)), torch.zeros((), dtype=x.dtype))


def reference(w, branch, stream, rng):
    """(out, leaves) in float64, on the CPU, from elementary operations."""
    w = {k: v.double().cpu().requires_grad_() for k, v in w.items()}
    w["branch"], w["stream"] = branch.double().cpu().requires_grad_(), stream.double().cpu().requires_grad_()
    s = dropped(w["branch"], rng, 0) + w["stream"]
    d = s - s.mean(-1, keepdim=True)
    y = d / torch.sqrt((d * d).mean(-1, keepdim=True) + EPS) * w["norm"] + w["shift"]
    proj = y @ w["proj"]
    L = s.shape[1]
    x = torch.cat([proj.new_zeros(s.shape[0], K - 1, R), proj[..., :R]], 1)
    z = w["conv_bias"] + sum(x[:, k:k + L] * w["conv"][:, k] for k in range(K))
    c = z * torch.sigmoid(z)
    la = w["A"] * torch.sigmoid(proj[..., R:2 * R] + w["gate_bias"])
    a, weight = torch.exp(la), torch.sqrt(-torch.expm1(2 * la))
    v = c * torch.sigmoid(proj[..., 2 * R:] + w["input_bias"]) * weight
    h, hs = torch.zeros_like(v[:, 0]), []
    for t in range(L):
        h = a[:, t] * h + v[:, t]
        hs.append(h)
    return dropped(torch.stack(hs, 1) @ w["back"], rng, 1) + s, w


@pytest.mark.parametrize("B,L", [(1, 1), (2, 13), (3, 70), (2, 300)])
def test_training_step(B, L):
    w = weights(L)
    branch, stream, dout, rng = inputs(B, L, L + 1)
    out, kept = forward(w, branch, stream, rng)
    ref, leaves = reference(w, branch, stream, rng)
    top = float(ref.detach().abs().max())
    assert float((out.double().cpu() - ref.detach()).abs().max()) <= 1e-4 * top
    ref.backward(dout.double().cpu())
    got = backward(w, kept, dout, rng)
    assert set(got) == set(leaves)
    for k in got:
        g = leaves[k].grad
        err = float((got[k].double().cpu() - g).abs().max())
        assert err <= 3e-4 * float(g.abs().max()), (k, err)


def test_prefill_then_tokens():
    B, L, n = 2, 90, 5
    w = weights(3)
    branch, stream, _, rng = inputs(B, L + n, 4)
    none = lambda t: binding.ssm_layer_norm_fwd(t[0], w["norm"], w["shift"], residual=t[1], eps=EPS)  # noqa: E731
    whole = none((branch, stream))["y"] @ w["proj"]
    x = whole[..., :R].contiguous()
    c = binding.ssm_causal_conv1d_fwd(x, w["conv"], w["conv_bias"])
    gates = dict(gate_bias=w["gate_bias"], input_bias=w["input_bias"], **FORM)
    want = binding.ssm_gated_linear_fwd(c, whole[..., R:2 * R], w["A"], input_gate=whole[..., 2 * R:], **gates)
    head = whole[:, :L]
    c, conv_state = binding.ssm_causal_conv1d_fwd(head[..., :R].contiguous(), w["conv"], w["conv_bias"],
                                                  return_final_state=True)
    h, state = binding.ssm_gated_linear_fwd(c, head[..., R:2 * R].contiguous(), w["A"],
                                            input_gate=head[..., 2 * R:].contiguous(), return_final_state=True, **gates)
    top = float(want.abs().max())
    assert float((h - want[:, :L]).abs().max()) <= 1e-5 * top
    for t in range(L, L + n):
        p = whole[:, t]
        c = binding.ssm_causal_conv1d_update(conv_state, p[:, :R].contiguous(), w["conv"], w["conv_bias"])
        y = binding.ssm_gated_linear_update(state, c, p[:, R:2 * R], w["A"], input_gate=p[:, 2 * R:], **gates)
        assert float((y - want[:, t]).abs().max()) <= 1e-5 * top


def test_captured_step_draws_anew():
    w = weights(5)
    branch, stream, dout, rng = inputs(2, 200, 6)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        kept = forward(w, branch, stream, rng)
        backward(w, kept[1], dout, rng)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        out, kept = forward(w, branch, stream, rng)
        grads = backward(w, kept, dout, rng)
    seen = []
    for step in (7, 8, 9):
        rng[1] = step
        graph.replay()
        torch.cuda.synchronize()
        want, kept2 = forward(w, branch, stream, rng)
        again = backward(w, kept2, dout, rng)
        assert torch.equal(out, want) and all(torch.equal(grads[k], again[k]) for k in grads)
        seen.append(out.clone())
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])
