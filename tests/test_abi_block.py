"""Argument validation of the entry points of the layer norm, the dropout and the
causal convolution's gradients.

CPU only. Every call here fails validation (or has nothing to do) before the
library touches the device; the fake pointers are never dereferenced.
"""

import ctypes

import pytest

from selective_state_space_87_amd import binding

OK, E_NULLPTR, E_SHAPE, E_DTYPE, E_ALIGN, E_WORKSPACE, E_ALIAS, E_UNSUPPORTED, E_HIP = range(9)
P = 0x1000000  # fake device addresses, 16 MiB apart, never dereferenced
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    return binding.library()


def vp(x):
    return None if x is None else ctypes.c_void_p(x)


def drop(lib, n=100, ind=0, resd=0, p=0.1, call=0, rng=P, x=2 * P, res=3 * P, y=4 * P):
    return lib.ssm_dropout_fwd(n, ind, resd, p, call, vp(rng), vp(x), vp(res), vp(y), None)


def drop_bwd(lib, n=100, p=0.1, call=0, rng=P, dy=2 * P, dx=3 * P):
    return lib.ssm_dropout_bwd(n, p, call, vp(rng), vp(dy), vp(dx), None)


def norm(lib, rows=4, dim=32, ind=0, resd=0, outd=0, eps=1e-5, p=0.1, call=0, rng=P, x=2 * P, res=3 * P, w=4 * P,
         b=5 * P, y=6 * P, reso=7 * P):
    return lib.ssm_layer_norm_fwd(rows, dim, ind, resd, outd, eps, p, call, vp(rng), vp(x), vp(res), vp(w), vp(b),
                                  vp(y), vp(reso), None)


def norm_bwd(lib, rows=4, dim=32, sd=0, eps=1e-5, p=0.1, call=0, rng=P, s=2 * P, w=3 * P, dy=4 * P, dr=5 * P,
             ds=6 * P, dx=7 * P, dw=8 * P, db=9 * P, ws=10 * P, wsb=1 << 20):
    return lib.ssm_layer_norm_bwd(rows, dim, sd, eps, p, call, vp(rng), vp(s), vp(w), vp(dy), vp(dr), vp(ds), vp(dx),
                                  vp(dw), vp(db), vp(ws), wsb, None)


def conv_bwd(lib, B=2, L=8, d=8, K=4, ind=0, silu=1, x=P, w=2 * P, b=3 * P, st=4 * P, dy=5 * P, dst=6 * P, dx=7 * P,
             dw=8 * P, db=9 * P, dsi=10 * P, ws=11 * P, wsb=1 << 20):
    return lib.ssm_causal_conv1d_bwd(B, L, d, K, ind, silu, vp(x), vp(w), vp(b), vp(st), vp(dy), vp(dst), vp(dx),
                                     vp(dw), vp(db), vp(dsi), vp(ws), wsb, None)


def test_dropout(lib):
    assert drop(lib, n=-1) == E_SHAPE and drop(lib, n=(1 << 52) + 1) == E_SHAPE
    for call in (drop, drop_bwd):
        for p in (-0.1, 1.1, NAN):
            assert call(lib, p=p) == E_UNSUPPORTED
        assert call(lib, n=0, rng=None) == OK
        assert call(lib, rng=None) == E_NULLPTR
        assert call(lib, rng=P + 4) == E_ALIGN
    assert drop(lib, ind=2) == E_DTYPE and drop(lib, resd=2) == E_DTYPE
    for name in ("x", "y"):
        assert drop(lib, **{name: None}) == E_NULLPTR
    assert drop(lib, x=2 * P + 2) == E_ALIGN and drop(lib, ind=1, x=2 * P + 1) == E_ALIGN
    assert drop(lib, res=3 * P + 2) == E_ALIGN and drop(lib, y=4 * P + 2) == E_ALIGN
    # y may be x of the same type or the residual, whole
    assert drop(lib, y=2 * P + 4) == E_ALIAS and drop(lib, y=3 * P + 4) == E_ALIAS
    assert drop(lib, ind=1, y=2 * P) == E_ALIAS          # the types differ: elements of others would be lost
    assert drop(lib, y=P) == E_ALIAS
    assert drop_bwd(lib, dx=2 * P + 4) == E_ALIAS and drop_bwd(lib, dx=P) == E_ALIAS
    assert drop_bwd(lib, dy=None) == E_NULLPTR and drop_bwd(lib, dx=None) == E_NULLPTR


def test_layer_norm(lib):
    assert norm(lib, rows=-1) == E_SHAPE and norm(lib, dim=0) == E_SHAPE and norm(lib, rows=1 << 50) == E_SHAPE
    assert norm(lib, dim=16385) == E_UNSUPPORTED and norm(lib, rows=1 << 31) == E_UNSUPPORTED
    assert norm(lib, eps=-1.0) == E_UNSUPPORTED and norm(lib, eps=NAN) == E_UNSUPPORTED
    for p in (-0.1, 1.1, NAN):
        assert norm(lib, p=p) == E_UNSUPPORTED
    assert norm(lib, res=None, reso=None) == E_UNSUPPORTED   # nothing is dropped but a branch
    assert norm(lib, ind=2) == norm(lib, resd=2) == norm(lib, outd=2) == E_DTYPE
    for name in ("x", "y", "reso", "rng"):
        assert norm(lib, **{name: None}) == E_NULLPTR, name
    assert norm(lib, p=0.0, rng=None, res=None) == E_NULLPTR  # residual_out without a residual
    for name, at in dict(x=2, res=3, w=4, b=5, y=6, reso=7).items():
        assert norm(lib, **{name: at * P + 2}) == E_ALIGN, name
    assert norm(lib, rng=P + 4) == E_ALIGN
    for name, at in dict(rng=1, x=2, res=3, w=4, b=5, reso=7).items():
        assert norm(lib, y=at * P) == E_ALIAS, name
    for name, at in dict(rng=1, x=2, w=4, b=5).items():
        assert norm(lib, reso=at * P) == E_ALIAS, name
    assert norm(lib, reso=3 * P + 16) == E_ALIAS
    assert norm(lib, rows=0, x=None, y=None, res=None) == OK


def test_layer_norm_bwd(lib):
    assert norm_bwd(lib, rows=-1) == E_SHAPE and norm_bwd(lib, dim=0) == E_SHAPE
    assert norm_bwd(lib, dim=16385) == E_UNSUPPORTED and norm_bwd(lib, eps=NAN) == E_UNSUPPORTED
    assert norm_bwd(lib, p=2.0) == E_UNSUPPORTED and norm_bwd(lib, sd=2) == E_DTYPE
    for name in ("s", "dy", "ds", "dx", "rng"):
        assert norm_bwd(lib, **{name: None}) == E_NULLPTR, name
    for name, at in dict(s=2, w=3, dy=4, dr=5, ds=6, dx=7, dw=8, db=9).items():
        assert norm_bwd(lib, **{name: at * P + 2}) == E_ALIGN, name
    need = lib.ssm_layer_norm_bwd_workspace_bytes(4, 32)
    assert need > 0
    assert norm_bwd(lib, ws=None) == E_WORKSPACE and norm_bwd(lib, wsb=need - 1) == E_WORKSPACE
    assert norm_bwd(lib, ws=10 * P + 8) == E_ALIGN
    for out in ("ds", "dx"):
        for at in (1, 2, 3, 8, 9, 10):
            assert norm_bwd(lib, **{out: at * P}) == E_ALIAS, (out, at)
        for at in (4, 5):
            assert norm_bwd(lib, **{out: at * P + 16}) == E_ALIAS, (out, at)
    assert norm_bwd(lib, dx=6 * P) == E_ALIAS
    for out in ("dw", "db", "ws"):
        for at in (1, 2, 3, 4, 5):
            assert norm_bwd(lib, **{out: at * P}) == E_ALIAS, (out, at)
    assert norm_bwd(lib, dw=9 * P) == E_ALIAS and norm_bwd(lib, dw=10 * P) == E_ALIAS
    assert norm_bwd(lib, rows=0, dw=None, db=None) == OK
    assert lib.ssm_layer_norm_bwd_workspace_bytes(0, 32) == lib.ssm_layer_norm_bwd_workspace_bytes(4, 16385) == 0


def test_conv_bwd(lib):
    assert conv_bwd(lib, B=-1) == conv_bwd(lib, L=-1) == conv_bwd(lib, d=-1) == conv_bwd(lib, K=0) == E_SHAPE
    assert conv_bwd(lib, B=60000, L=1 << 20, d=1 << 30) == E_SHAPE
    assert conv_bwd(lib, K=9) == conv_bwd(lib, B=65536) == conv_bwd(lib, L=4194241) == E_UNSUPPORTED
    assert conv_bwd(lib, ind=2) == E_DTYPE
    for name in ("x", "w", "dy", "dx"):
        assert conv_bwd(lib, **{name: None}) == E_NULLPTR, name
    for name, at in dict(x=1, dy=5, dx=7).items():
        assert conv_bwd(lib, **{name: at * P + 8}) == E_ALIGN, name
    for name, at in dict(w=2, b=3, st=4, dst=6, dw=8, db=9, dsi=10).items():
        assert conv_bwd(lib, **{name: at * P + 2}) == E_ALIGN, name
    need = lib.ssm_causal_conv1d_bwd_workspace_bytes(2, 8, 8, 4)
    assert need >= 2 * 5 * 8 * 4
    assert conv_bwd(lib, ws=None) == E_WORKSPACE and conv_bwd(lib, wsb=need - 1) == E_WORKSPACE
    assert conv_bwd(lib, ws=11 * P + 8) == E_ALIGN
    outs = dict(dx=7, dw=8, db=9, dsi=10, ws=11)
    for name, own in outs.items():
        for at in range(1, 12):
            if at != own:
                assert conv_bwd(lib, **{name: at * P}) == E_ALIAS, (name, at)
    assert conv_bwd(lib, d=0, x=None) == OK and conv_bwd(lib, B=0, dw=None, db=None, x=None) == OK
    for bad in ((0, 8, 8, 4), (2, -1, 8, 4), (2, 8, 0, 4), (2, 8, 8, 9), (65536, 8, 8, 4), (2, 8, 1 << 55, 4)):
        assert lib.ssm_causal_conv1d_bwd_workspace_bytes(*bad) == 0
