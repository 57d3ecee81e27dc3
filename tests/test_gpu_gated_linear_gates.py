"""The gates of the gated linear recurrence by themselves: far down the sigmoid and the
softplus, with biases that cancel most of the raw value, and at infinities.

Tolerances, in E = 2^-24. Where a decay is e^-200 = 0 and x is 1, y is the input gate
itself, and with A = -1 and the weight 1 - a, y is 1 - e^-g. Raw values and biases are
multiples of 2^-10 below 2^10, so that u, their sum, is exact in float32. Then e^-|u| is
off by an exponential (2 E), the rounding of what its exponent left (E), ln 2's own in
that (0.05 |u| E, 4 E at 80) and the product (E); a gate by that, a sum (E) and a
reciprocal or a logarithm (2 E), and y by x's product: 12 E, taken as 16. 1 - e^-g adds
A's scaling and the series (24 E in oracle/gated_linear_oracle.py): 40 E. s (1 - s)
takes s twice and e^-u once: 40 E.
"""

import numpy as np
import pytest
import torch

import oracle
from selective_state_space_87_amd import binding

pytestmark = pytest.mark.gpu
E = 2.0 ** -24
LENGTHS = [3, 100, 300]  # step by step, one tile, a chain of tiles
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")


def np64(t):
    return None if t is None else t.double().cpu().numpy()


def raw_and_bias(L, D, seed):
    """raw [1, L, D] and bias [D] whose exact sum u lies within 80 of 0; biases up to 400."""
    g = torch.Generator().manual_seed(seed)
    grid = lambda t: torch.round(t * 1024) / 1024  # noqa: E731
    u = grid(160 * torch.rand(1, L, D, generator=g) - 80)
    bias = grid(800 * torch.rand(D, generator=g) - 400)
    raw = u - bias
    assert torch.equal(raw.double() + bias.double(), u.double())
    return raw.cuda(), bias.cuda(), np64(u)


def sigmoid64(u):
    e = np.exp(-np.abs(u))
    return np.where(u < 0, e, 1.0) / (1.0 + e)


def near(got, want, eps):
    err = np.abs(np64(got) - want)
    room = eps * E * np.abs(want)
    assert (err <= room).all(), float((err / (E * np.abs(want))).max())


def gone(L, D):
    """x = 1 and decays of e^-200: y is the input gate."""
    one = torch.ones(1, L, D, device="cuda")
    return dict(x=one, gate=one.clone(), A=torch.full((D,), -200.0, device="cuda"))


@pytest.mark.parametrize("L", LENGTHS)
@pytest.mark.parametrize("D", [64, 33])
def test_input_gate(L, D):
    raw, bias, u = raw_and_bias(L, D, L + D)
    y = binding.ssm_gated_linear_fwd(**gone(L, D), input_gate=raw, input_bias=bias)
    near(y, sigmoid64(u), 16)


@pytest.mark.parametrize("L", LENGTHS)
@pytest.mark.parametrize("form", ["gate_sigmoid", "gate_softplus"])
def test_decays_gate(L, form):
    # a batch row a step, each from an empty state: y = 1 - e^-g
    raw, bias, u = raw_and_bias(L, 64, L)
    g = sigmoid64(u) if form == "gate_sigmoid" else np.logaddexp(u, 0.0)
    one = torch.ones(L, 1, 64, device="cuda")
    A = torch.full((64,), -1.0, device="cuda")
    y = binding.ssm_gated_linear_fwd(one, raw.reshape(L, 1, 64), A, gate_bias=bias, input_complement=True, **{form: True})
    near(y.reshape(1, L, 64), -np.expm1(-g), 40)
    # the first step of tiles
    wide = raw.reshape(L, 1, 64).expand(L, 130, 64).contiguous()
    y = binding.ssm_gated_linear_fwd(one.expand(L, 130, 64).contiguous(), wide, A, gate_bias=bias, input_complement=True,
                                     **{form: True})
    near(y[:, :1].reshape(1, L, 64), -np.expm1(-g), 40)


@pytest.mark.parametrize("L", LENGTHS)
def test_gradient_of_the_input_gate(L):
    raw, bias, u = raw_and_bias(L, 64, 7 + L)
    t = gone(L, 64)
    dy = torch.randn(1, L, 64, generator=torch.Generator().manual_seed(L)).cuda()
    got = binding.ssm_gated_linear_bwd(**t, dy=dy, input_gate=raw, input_bias=bias)
    near(got["dx"], np64(dy) * sigmoid64(u), 16)
    near(got["dinput_gate"], np64(dy) * sigmoid64(u) * sigmoid64(-u), 40)


@pytest.mark.parametrize("L", [4, 60, 200])
def test_infinite_gates(L):
    """A gate closed by -infinity lets nothing through, in either direction; NaN stays."""
    D = 64
    t = gone(L, D)
    raw = torch.zeros(1, L, D, device="cuda")
    raw[0, 1, 0], raw[0, 1, 1], raw[0, 1, 2] = -INF, INF, float("nan")
    raw[0, 2, 0], raw[0, 2, 1] = -3.0e38, 3.0e38
    y = binding.ssm_gated_linear_fwd(**t, input_gate=raw)
    got = binding.ssm_gated_linear_bwd(**t, dy=torch.ones_like(raw), input_gate=raw)
    for s in (1, 2):
        assert y[0, s, 0] == 0 and y[0, s, 1] == 1
        assert got["dx"][0, s, 0] == 0 and got["dx"][0, s, 1] == 1
        assert got["dinput_gate"][0, s, 0] == 0 and got["dinput_gate"][0, s, 1] == 0
    assert y[0, 1, 2].isnan() and got["dx"][0, 1, 2].isnan() and got["dinput_gate"][0, 1, 2].isnan()
    rest = torch.ones(L, D, dtype=torch.bool, device="cuda")
    rest[1:3, :2] = False
    rest[1:, 2] = False  # (a NaN state stays one: 0 times it is NaN)
    assert (y[0][rest] == 0.5).all() and (got["dinput_gate"][0][rest] == 0.25).all()


@pytest.mark.parametrize("L", [4, 60, 200])
@pytest.mark.parametrize("form", ["gate_sigmoid", "gate_softplus"])
def test_infinite_gates_of_the_decay(L, form):
    """Closed by -infinity: the state passes whole. Open by infinity: e^A of it, or nothing."""
    D = 64
    raw = torch.zeros(1, L, D, device="cuda")
    raw[0, :, 0], raw[0, :, 1] = -INF, INF
    raw[0, 1, 2] = float("nan")
    A = torch.full((D,), -1.0, device="cuda")
    h0 = torch.full((1, D), 3.0, device="cuda")
    kw = dict(input_norm=True, **{form: True})
    y, h = binding.ssm_gated_linear_fwd(torch.ones_like(raw), raw, A, h0=h0, return_final_state=True, **kw)
    assert (y[0, :, 0] == 3).all() and h[0, 0] == 3
    want, first = 3.0, y[0, 0, 1].double().item()
    a, w = (np.exp(-1.0), np.sqrt(-np.expm1(-2.0))) if form == "gate_sigmoid" else (0.0, 1.0)
    assert abs(first - (want * a + w)) <= 64 * E * first
    assert y[0, 0, 2].isfinite() and y[0, 1:, 2].isnan().all()
    assert y[0, :, 3:].isfinite().all()
    got = binding.ssm_gated_linear_bwd(torch.ones_like(raw), raw, A, torch.ones_like(raw), h0=h0, **kw)
    assert (got["dgate"][0, :, 0] == 0).all() and (got["dx"][0, :, 0] == 0).all()
    assert all(got[k][..., 3:].isfinite().all() for k in ("dx", "dgate", "dA", "dh0"))


@pytest.mark.parametrize("B,L,D", [(2, 9, 40), (2, 77, 33), (1, 300, 64)])
@pytest.mark.parametrize("act,scale", [("sigmoid", "norm"), ("softplus", "complement"), ("softplus", None)])
@pytest.mark.parametrize("xt", [torch.float32, torch.bfloat16])
def test_biases_that_cancel(B, L, D, act, scale, xt):
    """Whole calls, within the oracle's rooms, which know nothing of a bias."""
    g = torch.Generator().manual_seed(B + L + D)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    gb, ib = 40 * rn(D), 40 * rn(D)
    t = dict(x=rn(B, L, D).to(xt), gate=(3 * rn(B, L, D) - gb).to(xt), A=-torch.exp(rn(D)),
             input_gate=(3 * rn(B, L, D) - ib).to(xt), gate_bias=gb, input_bias=ib, h0=rn(B, D))
    t = {k: v.cuda() for k, v in t.items()}
    form = dict(gate_sigmoid=act == "sigmoid", gate_softplus=act == "softplus", input_norm=scale == "norm",
                input_complement=scale == "complement")
    ref64 = {k: np64(v) for k, v in t.items()}
    y, h = binding.ssm_gated_linear_fwd(**t, **form, out_dtype=torch.float32, return_final_state=True)
    ry, rh, room_y, room_h = oracle.gated_linear(**ref64, act=act, scale=scale)
    assert (np.abs(np64(y) - ry) <= room_y + 1e-30).all() and (np.abs(np64(h) - rh) <= room_h + 1e-30).all()
    dy, dh = rn(B, L, D).cuda(), rn(B, D).cuda()
    got = binding.ssm_gated_linear_bwd(**t, **form, dy=dy, dh_final=dh)
    want, room = oracle.gated_linear_bwd(**ref64, dy=np64(dy), dh_final=np64(dh), act=act, scale=scale)
    for k in want:
        assert (np.abs(np64(got[k]) - want[k]) <= room[k] + 1e-30).all(), k
