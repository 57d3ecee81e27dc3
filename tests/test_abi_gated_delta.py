"""Argument validation of the gated delta rule's and the RMS norm's entry points.

CPU only. Every call here fails validation (or has nothing to do) before the
library touches the device; the fake pointers are never dereferenced.
"""

import ctypes

import pytest
import torch

from selective_state_space_87_amd import binding

OK, E_NULLPTR, E_SHAPE, E_DTYPE, E_ALIGN, E_WORKSPACE, E_ALIAS, E_UNSUPPORTED, E_HIP = range(9)
P = 0x1000000  # fake device addresses, 16 MiB apart, never dereferenced


@pytest.fixture(scope="module")
def lib():
    return binding.library()


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


def fwd(lib, B=2, L=8, G=2, H=4, Pd=8, N=8, ind=0, outd=0, flags=13, scale=1.0, qs=16, ks=16, vs=32, q=P, k=2 * P,
        v=3 * P, dt=4 * P, A=5 * P, beta=6 * P, bias=7 * P, h0=8 * P, lens=9 * P, y=10 * P, hf=11 * P, ws=12 * P,
        wsb=1 << 24):
    return lib.ssm_gated_delta_fwd(B, L, G, H, Pd, N, ind, outd, flags, scale, qs, ks, vs, vp(q), vp(k), vp(v), vp(dt),
                                   vp(A), vp(beta), vp(bias), vp(h0), vp(lens), vp(y), vp(hf), vp(ws), wsb, None)


def upd(lib, B=2, G=2, H=4, Pd=8, N=8, ind=0, outd=0, flags=13, qs=16, ks=16, vs=32, state=P, q=2 * P, k=3 * P,
        v=4 * P, dt=5 * P, A=6 * P, beta=7 * P, bias=8 * P, y=9 * P):
    return lib.ssm_gated_delta_update(B, G, H, Pd, N, ind, outd, flags, 1.0, qs, ks, vs, vp(state), vp(q), vp(k),
                                      vp(v), vp(dt), vp(A), vp(beta), vp(bias), vp(y), None)


def bwd(lib, B=2, L=8, G=2, H=4, Pd=8, N=8, ind=0, flags=13, qs=16, ks=16, vs=32, q=P, k=2 * P, v=3 * P, dt=4 * P,
        A=5 * P, beta=6 * P, bias=7 * P, h0=8 * P, lens=9 * P, dy=10 * P, dh=11 * P, dq=12 * P, dk=13 * P, dv=14 * P,
        ddt=15 * P, dA=16 * P, dbeta=17 * P, dbias=18 * P, dh0=19 * P, ws=20 * P, wsb=1 << 24):
    return lib.ssm_gated_delta_bwd(B, L, G, H, Pd, N, ind, flags, 1.0, qs, ks, vs, vp(q), vp(k), vp(v), vp(dt), vp(A),
                                   vp(beta), vp(bias), vp(h0), vp(lens), vp(dy), vp(dh), vp(dq), vp(dk), vp(dv),
                                   vp(ddt), vp(dA), vp(dbeta), vp(dbias), vp(dh0), vp(ws), wsb, None)


@pytest.mark.parametrize("call", [fwd, bwd, upd])
def test_sizes_types_and_options(lib, call):
    assert call(lib, B=-1) == E_SHAPE
    assert call(lib, Pd=0) == E_SHAPE
    assert call(lib, N=0) == E_SHAPE
    assert call(lib, G=3, qs=99, ks=99) == E_SHAPE      # 4 heads over 3
    assert call(lib, G=0) == E_SHAPE
    assert call(lib, N=129, qs=999, ks=999) == E_UNSUPPORTED
    assert call(lib, Pd=257, vs=9999) == E_UNSUPPORTED
    assert call(lib, ind=2) == E_DTYPE
    assert call(lib, flags=2) == E_UNSUPPORTED          # no zero-order hold here
    assert call(lib, flags=16) == E_UNSUPPORTED
    assert call(lib, qs=15) == E_SHAPE
    assert call(lib, ks=15) == E_SHAPE
    assert call(lib, vs=31) == E_SHAPE
    assert call(lib, vs=1 << 23) == E_UNSUPPORTED
    assert call(lib, B=1 << 45) == E_SHAPE
    assert call(lib, B=1 << 28) == E_UNSUPPORTED


def test_size_limits(lib):
    # at most 2^22 head slices of 16 columns, and as many blocks of 64 steps
    assert fwd(lib, B=1 << 20, L=17, Pd=17, vs=68) == E_UNSUPPORTED
    assert upd(lib, B=(1 << 20) + 1) == E_UNSUPPORTED
    assert bwd(lib, B=1 << 13, L=64 * 128 + 1) == E_UNSUPPORTED
    assert fwd(lib, B=1 << 20, L=17, wsb=0) == E_WORKSPACE  # 2^22 slices: taken
    # products of sizes past 64 bits, though nothing is there
    for call in (fwd, bwd):
        assert call(lib, B=0, G=1 << 61, H=1 << 61, qs=1, ks=1, vs=1) == E_SHAPE
    assert upd(lib, B=0, G=1 << 61, H=1 << 61, qs=1, ks=1, vs=1) == E_SHAPE
    assert lib.ssm_gated_delta_workspace_bytes(0, 8, 1 << 61, 1 << 61, 8, 8, 0) == 0


def test_fwd_pointers(lib):
    for name in ("q", "k", "v", "dt", "A", "beta", "y"):
        assert fwd(lib, **{name: None}) == E_NULLPTR, name
    assert fwd(lib, outd=2) == E_DTYPE
    assert fwd(lib, L=-1) == E_SHAPE
    assert fwd(lib, L=1 << 30) == E_UNSUPPORTED
    assert fwd(lib, q=P + 2) == E_ALIGN
    assert fwd(lib, ind=1, q=P + 1) == E_ALIGN
    assert fwd(lib, lens=9 * P + 2) == E_ALIGN
    assert fwd(lib, hf=11 * P + 2) == E_ALIGN
    for name in ("q", "k", "v", "dt", "A", "beta", "bias", "h0", "lens", "hf"):
        at = dict(q=P, k=2 * P, v=3 * P, dt=4 * P, A=5 * P, beta=6 * P, bias=7 * P, h0=8 * P, lens=9 * P, hf=11 * P)
        assert fwd(lib, y=at[name]) == E_ALIAS, name
        if name not in ("h0", "hf"):
            assert fwd(lib, hf=at[name]) == E_ALIAS, name
    assert fwd(lib, hf=8 * P + 16) == E_ALIAS           # part of h0
    # the last element of a strided q counts, its gaps do too
    assert fwd(lib, qs=64, y=P + 4 * (15 * 64 + 15)) == E_ALIAS
    assert fwd(lib, B=0, q=None, A=None, y=None) == OK
    assert fwd(lib, G=0, H=0, qs=0, ks=0, vs=0, q=None, A=None, y=None) == OK


def test_workspace(lib):
    need = lib.ssm_gated_delta_workspace_bytes(2, 4096, 2, 4, 64, 64, 0)
    big = dict(L=4096, Pd=64, N=64, qs=128, ks=128, vs=256, q=1 << 40, k=2 << 40, v=3 << 40, dt=4 << 40, h0=5 << 40,
               y=6 << 40, hf=7 << 40, beta=8 << 40)
    if need:
        assert fwd(lib, **big, ws=None, wsb=0) == E_WORKSPACE
        assert fwd(lib, **big, ws=9 << 40, wsb=need - 1) == E_WORKSPACE
        assert fwd(lib, **big, ws=(9 << 40) + 8, wsb=need) == E_ALIGN
        assert fwd(lib, **big, ws=1 << 40, wsb=need) == E_ALIAS
    assert lib.ssm_gated_delta_workspace_bytes(2, 8, 2, 3, 8, 8, 0) == 0
    assert lib.ssm_gated_delta_bwd_workspace_bytes(2, 8, 2, 4, 8, 129, 0) == 0


def test_update_pointers(lib):
    for name in ("state", "q", "k", "v", "dt", "A", "beta", "y"):
        assert upd(lib, **{name: None}) == E_NULLPTR, name
    assert upd(lib, state=P + 8) == E_ALIGN
    assert upd(lib, y=P + 16) == E_ALIAS
    assert upd(lib, state=7 * P) == E_ALIAS
    assert upd(lib, y=2 * P) == E_ALIAS
    assert upd(lib, B=0, state=None) == OK


def test_bwd_pointers(lib):
    for name in ("q", "k", "v", "dt", "A", "beta", "dy", "dq", "dk", "dv", "ddt", "dA", "dbeta"):
        assert bwd(lib, **{name: None}) == E_NULLPTR, name
    ins = dict(q=P, k=2 * P, v=3 * P, dt=4 * P, A=5 * P, beta=6 * P, bias=7 * P, h0=8 * P, lens=9 * P, dy=10 * P,
               dh=11 * P)
    outs = dict(dq=12 * P, dk=13 * P, dv=14 * P, ddt=15 * P, dA=16 * P, dbeta=17 * P, dbias=18 * P, dh0=19 * P)
    for o in outs:
        for i in ins:
            assert bwd(lib, **{o: ins[i]}) == E_ALIAS, (o, i)
        for i in outs:
            if i != o:
                assert bwd(lib, **{o: outs[i]}) == E_ALIAS, (o, i)
        assert bwd(lib, **{o: outs[o] + 2}) == E_ALIGN, o


def nf(lib, R=4, d=8, ind=0, rd=0, od=0, eps=1e-5, x=P, res=2 * P, w=3 * P, y=4 * P, ro=5 * P, sc=None):
    return lib.ssm_rms_norm_fwd(R, d, ind, rd, od, eps, vp(x), vp(res), vp(w), vp(y), vp(ro), vp(sc), None)


def test_norm_validation(lib):
    assert nf(lib, R=-1) == E_SHAPE
    assert nf(lib, d=0) == E_SHAPE
    assert nf(lib, d=16385) == E_UNSUPPORTED
    assert nf(lib, eps=-1.0) == E_UNSUPPORTED
    assert nf(lib, eps=float("nan")) == E_UNSUPPORTED
    assert nf(lib, ind=2) == E_DTYPE
    assert nf(lib, rd=2) == E_DTYPE
    assert nf(lib, od=3) == E_DTYPE
    assert nf(lib, x=None) == E_NULLPTR
    assert nf(lib, ro=None) == E_NULLPTR
    assert nf(lib, res=None) == E_NULLPTR
    assert nf(lib, od=2) == E_NULLPTR                   # scales missing
    assert nf(lib, sc=6 * P) == E_NULLPTR               # scales without the 8-bit output
    assert nf(lib, x=P + 2) == E_ALIGN
    assert nf(lib, y=P) == E_ALIAS
    assert nf(lib, y=5 * P) == E_ALIAS
    assert nf(lib, ro=P) == E_ALIAS
    assert nf(lib, ro=2 * P + 4) == E_ALIAS
    assert nf(lib, R=0, x=None) == OK


def nb(lib, R=4, d=8, sd=0, eps=1e-5, s=P, w=2 * P, dy=3 * P, dr=4 * P, ds=5 * P, dw=6 * P, ws=7 * P, wsb=1 << 20):
    return lib.ssm_rms_norm_bwd(R, d, sd, eps, vp(s), vp(w), vp(dy), vp(dr), vp(ds), vp(dw), vp(ws), wsb, None)


def test_norm_bwd_validation(lib):
    assert nb(lib, R=-1) == E_SHAPE
    assert nb(lib, d=16385) == E_UNSUPPORTED
    assert nb(lib, sd=2) == E_DTYPE
    assert nb(lib, s=None) == E_NULLPTR
    assert nb(lib, dy=None) == E_NULLPTR
    assert nb(lib, ds=None) == E_NULLPTR
    assert nb(lib, ws=None, wsb=0) == E_WORKSPACE
    assert nb(lib, wsb=lib.ssm_rms_norm_bwd_workspace_bytes(4, 8) - 1) == E_WORKSPACE
    assert nb(lib, ws=7 * P + 4) == E_ALIGN
    assert nb(lib, ds=P) == E_ALIAS
    assert nb(lib, ds=3 * P + 4) == E_ALIAS
    assert nb(lib, dw=2 * P) == E_ALIAS
    assert nb(lib, dw=5 * P) == E_ALIAS
    assert nb(lib, ws=6 * P) == E_ALIAS


def test_binding_refuses_what_it_cannot_pass_on():
    q = torch.zeros(1, 2, 1, 4)
    v = torch.zeros(1, 2, 1, 3)
    g = torch.zeros(1, 2, 1)
    with pytest.raises(ValueError):
        binding.ssm_gated_delta_fwd(q, q, v, g, torch.zeros(1), g)        # no CPU path
    with pytest.raises(ValueError):
        binding.ssm_gated_delta_fwd(q[0], q, v, g, torch.zeros(1), g)
    with pytest.raises(ValueError):
        binding.ssm_rms_norm_fwd(torch.zeros(2, 4))
    with pytest.raises(ValueError):
        binding.ssm_rms_norm_fwd(torch.zeros(2, 4, dtype=torch.float16))


def test_steps_of_column_ranges():
    wide = torch.zeros(3, 5, 40)
    q = wide[:, :, 8:24].view(3, 5, 4, 4)
    assert binding._step_of("q", q, 2, 16) == 40
    assert binding._step_of("q", q[:1], 2, 16) == 40
    assert binding._step_of("q", q[:, :1], 2, 16) == 200       # batch rows of one step
    assert binding._step_of("q", q[:1, :1], 2, 16) == 16
    with pytest.raises(ValueError):
        binding._step_of("q", q[:, :4], 2, 16)                 # rows cut short: not at one distance
    with pytest.raises(ValueError):
        binding._step_of("q", q[:, :, ::2], 2, 8)
    with pytest.raises(ValueError):
        binding._step_of("q", q[..., ::2], 2, 8)


@pytest.mark.parametrize("call", [fwd, bwd, upd])
def test_key_heads_without_value_heads(lib, call):
    """H = 0 with G > 0 has gradients of q and k that no kernel would write."""
    assert call(lib, H=0, vs=0) == E_SHAPE
    assert call(lib, B=0, H=0, vs=0) == E_SHAPE
    assert call(lib, G=0, H=0, qs=0, ks=0, vs=0) == OK
    assert lib.ssm_gated_delta_workspace_bytes(2, 64, 2, 0, 8, 8, 0) == 0
    assert lib.ssm_gated_delta_bwd_workspace_bytes(2, 64, 2, 0, 8, 8, 0) == 0
