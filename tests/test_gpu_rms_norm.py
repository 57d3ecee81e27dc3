"""GPU parity of the RMS norm (residual's addition, 8-bit output) and its
gradients with the float64 oracle, through the C ABI.

Tolerances. A row's sum of squares in float32 over d elements is off by at most
about (8 + log2 d) 2^-24 of itself (eight in a row, then a tree), the root and
the three products after it by a few 2^-24 more: 3e-6 of the element covers
every d here. Gradients subtract two such terms: 1e-5 of the row's largest.
A bfloat16 output adds 2^-8 of its value, an e4m3 one 2^-4 (or half a
subnormal step of 2^-9) of the value in units of its scale.
"""

import numpy as np
import pytest
import torch

import oracle
from selective_state_space_87_amd import binding

pytestmark = pytest.mark.gpu
T = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no HIP device")


def data(rows, dim, seed, *types):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(rows, dim, generator=g).to(t).cuda() for t in types]


WIDTHS = [(1, 1), (5, 7), (3, 64), (130, 128), (7, 512), (6, 513), (4, 1024), (9, 1025), (5, 1537), (3, 2048),
          (4, 2560), (3, 4096), (2, 4100), (2, 8192), (2, 8193), (1, 16384)]


def np64(t):
    return t.double().cpu().numpy()


@pytest.mark.parametrize("rows,dim", WIDTHS)
@pytest.mark.parametrize("xt,rt,ot", [("f32", None, "f32"), ("bf16", "f32", "bf16"), ("bf16", "bf16", "bf16"),
                                      ("f32", "bf16", "bf16"), ("bf16", None, "e4m3"), ("f32", "f32", "e4m3"),
                                      ("bf16", "bf16", "e4m3")])
def test_forward(rows, dim, xt, rt, ot):
    x, r = data(rows, dim, dim, T[xt], T[rt or "f32"])
    w = 1.0 + 0.1 * torch.randn(dim, generator=torch.Generator().manual_seed(1)).cuda()
    out = binding.ssm_rms_norm_fwd(x, w, residual=r if rt else None, out_dtype=T[ot])
    s = x
    if rt:
        s = (x.float() + r.float()).to(T[rt])
        assert torch.equal(out["residual_out"], s)
    ref = oracle.rms_norm(np64(s), np64(w))
    if ot == "e4m3":
        sc = np64(out["scales"])
        top = np.abs(ref).max(-1)
        assert np.allclose(sc, np.where(top > 0, top / 448, 1.0), rtol=3e-6)
        err = np.abs(np64(out["y"].float()) - ref / sc[:, None])
        room = np.maximum(np.abs(ref / sc[:, None]) * 2.0 ** -4, 2.0 ** -10) + 448 * 6e-6
    else:
        err = np.abs(np64(out["y"]) - ref)
        room = np.abs(ref) * (3e-6 + (2.0 ** -8 if ot == "bf16" else 0.0)) + 1e-30
    assert (err <= room).all(), float((err / room).max())


@pytest.mark.parametrize("rows,dim", WIDTHS + [(2000, 64), (700, 2560), (1500, 100)])
@pytest.mark.parametrize("st", ["f32", "bf16"])
def test_gradients(rows, dim, st):
    s, dy, dr = data(rows, dim, dim + 1, T[st], torch.float32, torch.float32)
    w = 1.0 + 0.1 * torch.randn(dim, generator=torch.Generator().manual_seed(2)).cuda()
    for weight, res in ((w, dr), (None, None)):
        ds, dw = binding.ssm_rms_norm_bwd(s, weight, dy, dresidual=res)
        rs, rw = oracle.rms_norm_bwd(np64(s), None if weight is None else np64(weight), np64(dy),
                                     None if res is None else np64(res))
        r = 1 / np.sqrt((np64(s) ** 2).mean(-1, keepdims=True) + 1e-5)
        room = 1e-5 * ((np.abs(np64(dy)) * r * 1.6).max(-1, keepdims=True) + np.abs(rs))
        assert (np.abs(np64(ds) - rs) <= room).all()
        mag = (np.abs(np64(dy) * np64(s)) * r).sum(0)
        assert (np.abs(np64(dw) - rw) <= 1e-5 * mag + 1e-30).all()
        ds2, dw2 = binding.ssm_rms_norm_bwd(s, weight, dy, dresidual=res)
        assert torch.equal(ds, ds2) and torch.equal(dw, dw2)


def test_zero_rows_of_zeros_and_in_place():
    x = torch.zeros(3, 40, device="cuda")
    out = binding.ssm_rms_norm_fwd(x, out_dtype=T["e4m3"])
    assert not out["y"].float().any() and torch.equal(out["scales"], torch.ones(3, device="cuda"))
    assert binding.ssm_rms_norm_fwd(x[:0])["y"].shape == (0, 40)
    ds, dw = binding.ssm_rms_norm_bwd(x[:0], None, x[:0])
    assert ds.shape == (0, 40) and not dw.any()
    r, x = data(33, 256, 3, torch.float32, torch.bfloat16)
    want = binding.ssm_rms_norm_fwd(x, residual=r)
    got = binding.ssm_rms_norm_fwd(x, residual=r, residual_out=r)
    assert got["residual_out"] is r and torch.equal(r, want["residual_out"]) and torch.equal(got["y"], want["y"])
    s, dy, dr = data(9, 64, 4, torch.float32, torch.float32, torch.float32)
    want = binding.ssm_rms_norm_bwd(s, None, dy, dresidual=dr)
    got = binding.ssm_rms_norm_bwd(s, None, dy, dresidual=dr, ds=dr)
    assert torch.equal(got[0], want[0])


def test_minute_rows_in_eight_bits():
    # largest values 2^-118 (scale below 2^-126 if it were max / 448) and 2^-100, and zeros between
    s = torch.zeros(3, 64, device="cuda")
    s[0, ::3], s[1, ::3], s[2, 5] = 2.0**-118, -(2.0**-100), 2.0**-126
    out = binding.ssm_rms_norm_fwd(s, None, eps=1.0, out_dtype=torch.float8_e4m3fn)
    sc, y = out["scales"], out["y"].float()
    assert float(sc[0]) == 2.0**-126 == float(sc[2]) and abs(float(sc[1]) * 448 / 2.0**-100 - 1) < 3e-6
    assert not y[:, 1].any() and torch.equal(y[0, ::3], torch.full((22,), 256.0, device="cuda"))
    assert torch.equal(y[1, ::3], torch.full((22,), -448.0, device="cuda")) and float(y[2, 5]) == 1.0


def test_more_rows_than_a_launch_takes():
    rows, dim = (1 << 24) + 5, 5
    x = torch.randn(rows, dim, device="cuda", dtype=torch.bfloat16)
    res = torch.randn(rows, dim, device="cuda", dtype=torch.bfloat16)
    out = binding.ssm_rms_norm_fwd(x, None, residual=res, out_dtype=torch.float8_e4m3fn)
    for a in (0, (1 << 23) - 3, (1 << 23), rows - 3):
        part = binding.ssm_rms_norm_fwd(x[a:a + 3].clone(), None, residual=res[a:a + 3].clone(),
                                        out_dtype=torch.float8_e4m3fn)
        assert torch.equal(out["y"][a:a + 3].view(torch.uint8), part["y"].view(torch.uint8))
        assert torch.equal(out["scales"][a:a + 3], part["scales"])
        assert torch.equal(out["residual_out"][a:a + 3], part["residual_out"])


def test_more_elements_than_32_bits_count():
    rows, dim = (1 << 20) + 9, 4096 + 8
    x = torch.empty(rows, dim, device="cuda", dtype=torch.bfloat16)
    w = 1.0 + 0.1 * torch.randn(dim, device="cuda")
    ends = (0, (1 << 20) - 2, rows - 4)
    for a in ends:
        x[a:a + 4] = torch.randn(4, dim, device="cuda")
    y = binding.ssm_rms_norm_fwd(x, w)["y"]
    for a in ends:
        assert torch.equal(y[a:a + 4], binding.ssm_rms_norm_fwd(x[a:a + 4].clone(), w)["y"])


def test_not_finite_rows_stay_their_own():
    x = data(4, 96, 5, torch.float32)[0]
    want = binding.ssm_rms_norm_fwd(x, out_dtype=T["e4m3"])
    x[1, 3], x[2, 5] = float("nan"), float("inf")
    got = binding.ssm_rms_norm_fwd(x, out_dtype=T["e4m3"])
    for row in (0, 3):
        assert torch.equal(got["y"][row].float(), want["y"][row].float()) and got["scales"][row] == want["scales"][row]
    assert got["y"][1].float().isnan().all() and got["y"][2].float().isnan()[5]


def test_unaligned_rows_and_side_stream():
    base = torch.randn(50 * 64 + 1, device="cuda")
    x = base[1:].view(50, 64)                      # 4-byte aligned only
    ref = oracle.rms_norm(np64(x))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    y = binding.ssm_rms_norm_fwd(x, stream=side)["y"]
    side.synchronize()
    assert (np.abs(np64(y) - ref) <= 3e-6 * np.abs(ref) + 1e-30).all()


def test_gradient_against_differences():
    s, dy = data(2, 48, 6, torch.float32, torch.float32)
    ds, _ = binding.ssm_rms_norm_bwd(s, None, dy)
    s64, dy64 = np64(s), np64(dy)
    for i in range(0, 96, 7):
        d = np.zeros(96)
        d[i] = 1e-5
        d = d.reshape(2, 48)
        num = ((oracle.rms_norm(s64 + d) - oracle.rms_norm(s64 - d)) * dy64).sum() / 2e-5
        assert abs(num - np64(ds).ravel()[i]) < 1e-4


def test_refusals():
    x = torch.zeros(2, 8, device="cuda")
    with pytest.raises(binding.SSMError) as e:
        binding.ssm_rms_norm_fwd(torch.zeros(1, 16385, device="cuda"))
    assert e.value.status == 7
    for kw in (dict(weight=torch.ones(7, device="cuda")), dict(residual=x[:1]), dict(out_dtype=torch.float16),
               dict(residual_out=x), dict(scales=torch.ones(2, device="cuda"))):
        with pytest.raises(ValueError):
            binding.ssm_rms_norm_fwd(x, **kw)
    with pytest.raises(ValueError):
        binding.ssm_rms_norm_fwd(x.t())
