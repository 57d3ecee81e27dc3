"""The operators together, as a layer has them: RMS norm with the residual's
addition -> projections -> causal convolution over the packed q | k | v ->
gated delta rule on the column ranges -> RMS norm of each head's output.
Prefill and then single tokens, a captured single-token step, and the gradients
of the trained part, against the float64 oracles and float64 automatic
differentiation of the formulas.

Tolerance of the layer's output. All of it is float32 or 22-bit products: an
element of the rule's output is a sum over 32 states and at most 64 steps, of
products off by 2^-21 of themselves with random signs, (3 * 96)^(1/2) 2^-21 = 8e-6
of the largest element at most, half of that in the mean; its inputs carry the
errors of a norm, a projection and a convolution, below 2e-6 of their rows'
size: 1e-5 of the largest element covers both. The norm behind it divides by
the row's root mean square r and moves by at most (1 + |y|) e / r when a row
moves by e: 1e-5 max|o| (1 + |y|) / r, row by row.
"""

import numpy as np
import pytest
import torch

import oracle
from selective_state_space_87_amd import binding

pytestmark = pytest.mark.gpu
FLAGS = dict(dt_softplus=True, beta_sigmoid=True, qk_l2norm=True)
D, G, H, N, P, K = 96, 2, 4, 32, 48, 4
C = 2 * G * N + H * P
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")


def layer(seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return dict(norm=1 + 0.1 * rn(D), proj=rn(D, C) * D ** -0.5, gates=rn(D, 2 * H) * D ** -0.5, conv=rn(C, K) * 0.5,
                conv_bias=0.1 * rn(C), A=-torch.exp(rn(H)), dt_bias=rn(H) - 2, head_norm=1 + 0.1 * rn(P))


def split(c, lead):
    q, k, v = c.split([G * N, G * N, H * P], -1)
    return q.unflatten(-1, (G, N)), k.unflatten(-1, (G, N)), v.unflatten(-1, (H, P))


def prefill(w, x, res, seqlens=None):
    n = binding.ssm_rms_norm_fwd(x, w["norm"], residual=res, eps=EPS)
    gates = n["y"] @ w["gates"]
    c, conv_state = binding.ssm_causal_conv1d_fwd(n["y"] @ w["proj"], w["conv"], w["conv_bias"], return_final_state=True)
    q, k, v = split(c, 2)
    o, state = binding.ssm_gated_delta_fwd(q, k, v, gates[..., :H].contiguous(), w["A"], gates[..., H:].contiguous(),
                                           dt_bias=w["dt_bias"], return_final_state=True, **FLAGS)
    return binding.ssm_rms_norm_fwd(o, w["head_norm"], eps=EPS)["y"], n["residual_out"], conv_state, state


def token(w, x, res, conv_state, state):
    n = binding.ssm_rms_norm_fwd(x, w["norm"], residual=res, eps=EPS)
    gates = n["y"] @ w["gates"]
    c = binding.ssm_causal_conv1d_update(conv_state, n["y"] @ w["proj"], w["conv"], w["conv_bias"])
    q, k, v = split(c, 1)
    o = binding.ssm_gated_delta_update(state, q, k, v, gates[:, :H].contiguous(), w["A"], gates[:, H:].contiguous(),
                                       dt_bias=w["dt_bias"], **FLAGS)
    return binding.ssm_rms_norm_fwd(o, w["head_norm"], eps=EPS)["y"]


def reference(w, x, res):
    """y, and what the head norm's input was, in float64."""
    w = {n: a.double().cpu().numpy() for n, a in w.items()}
    s = x.double().cpu().numpy() + res.double().cpu().numpy()
    y = oracle.rms_norm(s, w["norm"], EPS)
    gates = y @ w["gates"]
    c = oracle.causal_conv1d(y @ w["proj"], w["conv"], w["conv_bias"])
    c = c[0] if isinstance(c, tuple) else c
    B, L = c.shape[:2]
    q, k, v = np.split(c, [G * N, 2 * G * N], -1)
    o = oracle.gated_delta(q.reshape(B, L, G, N), k.reshape(B, L, G, N), v.reshape(B, L, H, P), gates[..., :H], w["A"],
                           gates[..., H:], dt_bias=w["dt_bias"], softplus=True, sigmoid=True, l2norm=True,
                           scale=N ** -0.5)[0]
    return oracle.rms_norm(o, w["head_norm"], EPS), o


def close(name, got, ref, o, top):
    r = np.sqrt((o * o).mean(-1, keepdims=True) + EPS)
    assert tuple(got.shape) == ref.shape == o.shape, name
    room = 1e-5 * top * (1 + np.abs(ref)) / r
    worst = float((np.abs(got.double().cpu().numpy() - ref) / room).max())
    print(f"[layer] {name}: {worst:.3f} of the tolerance", flush=True)
    assert worst <= 1.0, name


@pytest.mark.parametrize("L", [1, 15, 70, 200])
def test_prefill_then_tokens(L):
    B, T = 3, 6
    w = {n: a.cuda() for n, a in layer(L).items()}
    g = torch.Generator().manual_seed(L + 1)
    x, res = torch.randn(B, L + T, D, generator=g).cuda(), torch.randn(B, L + T, D, generator=g).cuda()
    ref, o = reference(w, x, res)
    top = np.abs(o).max()
    y, res_out, conv_state, state = prefill(w, x[:, :L].contiguous(), res[:, :L].contiguous())
    assert torch.equal(res_out, x[:, :L] + res[:, :L])
    close(f"prefill {L}", y, ref[:, :L], o[:, :L], top)
    for t in range(L, L + T):
        y = token(w, x[:, t].contiguous(), res[:, t].contiguous(), conv_state, state)
        close(f"token {t}", y, ref[:, t], o[:, t], top)
    whole, _, conv_end, end = prefill(w, x, res)
    close("the whole at once", whole, ref, o, top)
    assert torch.allclose(end, state, rtol=0, atol=2e-5 * float(end.abs().max()))
    assert torch.allclose(conv_end, conv_state, rtol=0, atol=2e-5 * float(conv_end.abs().max()))


def test_captured_token_step():
    B, L, T = 2, 40, 4
    w = {n: a.cuda() for n, a in layer(9).items()}
    g = torch.Generator().manual_seed(10)
    packed = torch.randn(B, C, generator=g).cuda()
    gates = torch.randn(2, B, H, generator=g).cuda()
    first = (torch.randn(B, C, K - 1, generator=g).cuda(), torch.randn(B, H, P, N, generator=g).cuda())

    def step(conv_state, state):
        c = binding.ssm_causal_conv1d_update(conv_state, packed, w["conv"], w["conv_bias"])
        q, k, v = split(c, 1)
        o = binding.ssm_gated_delta_update(state, q, k, v, gates[0], w["A"], gates[1], dt_bias=w["dt_bias"], **FLAGS)
        return binding.ssm_rms_norm_fwd(o, w["head_norm"], eps=EPS)["y"]

    eager, mine = [a.clone() for a in first], [a.clone() for a in first]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = step(*mine)
    for i in range(4):
        packed.copy_(torch.randn(B, C, generator=g))  # the captured call reads the buffers anew
        gates.copy_(torch.randn(2, B, H, generator=g))
        want = step(*eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(mine[0], eager[0]) and torch.equal(mine[1], eager[1]), i


def test_gradients_through_norms_and_rule():
    """x, residual -> norm -> projections -> rule -> head norm, loss sum(y dy).

    Tolerance: the rule's gradients have twice the forward's sums, 2e-5 of their
    largest; the head norm's gradient is taken at an o that is off by 1e-5 max|o|,
    which moves it by at most three times that over the row's root mean square r,
    relatively.
    """
    B, L = 2, 90
    w = layer(21)
    g = torch.Generator().manual_seed(22)
    x, res = torch.randn(B, L, D, generator=g), torch.randn(B, L, D, generator=g)
    dy, dres = torch.randn(B, L, H, P, generator=g), torch.randn(B, L, D, generator=g)

    # float64, by automatic differentiation of the formulas
    w64 = {n: a.double() for n, a in w.items()}
    for n in ("norm", "proj", "A", "dt_bias", "head_norm"):
        w64[n].requires_grad_(True)
    x64 = x.double().requires_grad_(True)
    s = x64 + res.double()
    norm = lambda a, wt: a * torch.rsqrt((a * a).mean(-1, keepdim=True) + EPS) * wt  # noqa: E731
    y = norm(s, w64["norm"])
    q, k, v = split(y @ w64["proj"], 2)
    unit = lambda a: (a * torch.rsqrt((a * a).sum(-1, keepdim=True) + 1e-6)).repeat_interleave(H // G, 2)  # noqa: E731
    q, k = unit(q), unit(k)
    gates = y @ w64["gates"]
    decay = torch.exp(torch.nn.functional.softplus(gates[..., :H] + w64["dt_bias"]) * w64["A"])
    beta = torch.sigmoid(gates[..., H:])
    S, out = torch.zeros(B, H, P, N, dtype=torch.float64), []
    for t in range(L):
        S = S * decay[:, t, :, None, None]
        e = v[:, t] - (S * k[:, t, :, None]).sum(-1)
        S = S + (beta[:, t, :, None] * e)[..., None] * k[:, t, :, None]
        out.append(N ** -0.5 * (S * q[:, t, :, None]).sum(-1))
    o64 = torch.stack(out, 1)
    loss = (norm(o64, w64["head_norm"]) * dy.double()).sum() + (s * dres.double()).sum()
    loss.backward()

    d = {n: a.cuda() for n, a in w.items()}
    n = binding.ssm_rms_norm_fwd(x.cuda(), d["norm"], residual=res.cuda(), eps=EPS)
    packed = n["y"] @ d["proj"]
    gates = n["y"] @ d["gates"]
    a = dict(dt=gates[..., :H].contiguous(), A=d["A"], beta=gates[..., H:].contiguous(), dt_bias=d["dt_bias"], **FLAGS)
    o = binding.ssm_gated_delta_fwd(*split(packed, 2), **a)
    do, dhead = binding.ssm_rms_norm_bwd(o, d["head_norm"], dy.cuda(), eps=EPS)
    r = binding.ssm_gated_delta_bwd(*split(packed, 2), dy=do, **a)
    dpacked = torch.cat([r["dq"].flatten(2), r["dk"].flatten(2), r["dv"].flatten(2)], -1)
    dn = dpacked @ d["proj"].T + torch.cat([r["ddt"], r["dbeta"]], -1) @ d["gates"].T
    ds, dnorm = binding.ssm_rms_norm_bwd(n["residual_out"], d["norm"], dn, dresidual=dres.cuda(), eps=EPS)

    o_rms = torch.sqrt((o64 * o64).mean(-1) + EPS).min()
    tol = 2e-5 + 3 * 1e-5 * float((o64.abs().max() / o_rms).detach())
    for name, got, ref in (("ds", ds, x64.grad), ("dnorm", dnorm, w64["norm"].grad),
                           ("dproj", n["y"].flatten(0, 1).T @ dpacked.flatten(0, 1), w64["proj"].grad),
                           ("dA", r["dA"], w64["A"].grad), ("ddt_bias", r["ddt_bias"], w64["dt_bias"].grad),
                           ("dhead", dhead, w64["head_norm"].grad)):
        err = float((got.double().cpu() - ref).abs().max() / ref.abs().max())
        print(f"[layer] {name}: {err:.2e}, allowed {tol:.2e}", flush=True)
        assert err <= tol, name
