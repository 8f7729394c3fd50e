"""Host-side refusals of the training-step entry points, before any CUDA call
(no GPU needed)."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def gs():
    import mixed_precision_numerics_gradscaler_gb300 as gs
    return gs


def test_layernorm_arguments(gs):
    lib, p = gs._lib, ctypes.c_void_p(0x1000)   # never dereferenced
    fwd = lambda ldx=64, dt=1, R=8, C=64, w=2, eps=1e-5, ldy=64, x=p, y=p: lib.gs_layernorm_fwd(  # noqa: E731
        x, ldx, dt, R, C, None, None, w, eps, y, ldy, None, None, None)
    assert fwd(dt=3) == gs.GS_ERR_DTYPE and fwd(dt=1, w=0) == gs.GS_ERR_DTYPE
    assert fwd(ldx=63) == fwd(ldy=63) == fwd(R=-1) == fwd(C=-1) == gs.GS_ERR_SHAPE
    assert fwd(R=1 << 40, ldx=1 << 40, C=1) == gs.GS_ERR_SHAPE
    assert fwd(eps=-1.0) == fwd(eps=float("nan")) == fwd(eps=float("inf")) == gs.GS_ERR_ARG
    assert fwd(R=0, x=None, y=None) == fwd(C=0, x=None, y=None) == gs.GS_OK
    assert fwd(x=None) == fwd(y=None) == gs.GS_ERR_NULL
    assert fwd(x=ctypes.c_void_p(0x1001)) == gs.GS_ERR_ARG
    assert gs.gs_layernorm_ws_bytes(-1, 5) == 0 and gs.gs_layernorm_ws_bytes(1 << 40, 1 << 40) == 0
    bwd = lambda dt=1, R=8, C=64, ld=64, w=2, dw=2, ws=p, dy=p, mean=p, dg=p: lib.gs_layernorm_bwd(  # noqa: E731
        dy, ld, p, ld, dt, R, C, None, w, mean, p, p, ld, dg, None, dw, ws, None)
    assert bwd(dt=9) == bwd(dw=3) == bwd(w=0) == gs.GS_ERR_DTYPE
    assert bwd(ld=63) == bwd(R=-1) == gs.GS_ERR_SHAPE
    assert bwd(dy=None) == bwd(mean=None) == bwd(ws=None) == gs.GS_ERR_NULL
    assert bwd(ws=ctypes.c_void_p(0x1008)) == gs.GS_ERR_ARG
    assert bwd(C=0) == gs.GS_OK


def test_token_logprob_arguments(gs):
    lib, p = gs._lib, ctypes.c_void_p(0x1000)
    fwd = lambda ld=100, dt=1, R=4, V=100, t=p, lp=p, k=0, ids=None, tl=None, x=p: lib.gs_token_logprob(  # noqa: E731
        x, ld, dt, R, V, t, lp, None, None, k, ids, tl, None)
    assert fwd(dt=-1) == gs.GS_ERR_DTYPE
    assert fwd(ld=99) == fwd(V=0) == fwd(R=-2) == fwd(V=1 << 31, ld=1 << 31) == gs.GS_ERR_SHAPE
    assert fwd(k=33) == fwd(k=-1) == fwd(V=3, k=4) == gs.GS_ERR_SHAPE
    assert fwd(R=0, x=None) == gs.GS_OK
    assert fwd(x=None) == fwd(t=None) == fwd(lp=None) == fwd(k=2) == fwd(k=2, ids=p) == gs.GS_ERR_NULL
    assert fwd(t=ctypes.c_void_p(0x1004)) == gs.GS_ERR_ARG
    bwd = lambda ld=100, lo=100, dt=1, ot=0, R=4, V=100, lse=p, h=None, dh=None, d=p: lib.gs_token_logprob_bwd(  # noqa: E731
        p, ld, dt, R, V, p, lse, p, h, dh, None, d, lo, ot, None)
    assert bwd(dt=4) == bwd(ot=4) == gs.GS_ERR_DTYPE
    assert bwd(ld=99) == bwd(lo=99) == bwd(V=0) == gs.GS_ERR_SHAPE
    assert bwd(lse=None) == bwd(h=p) == bwd(dh=p) == bwd(d=None) == gs.GS_ERR_NULL
    assert bwd(R=0) == gs.GS_OK
    assert bwd(d=ctypes.c_void_p(0x1001)) == gs.GS_ERR_ARG


def test_adamw_arguments(gs):
    lib, p, out = gs._lib, ctypes.c_void_p(0x1000), ctypes.c_void_p()
    new = lambda n=1, gt=2, mo=0, ms=None, w=p, o=ctypes.byref(out): lib.gs_adamw_list_create(  # noqa: E731
        w, None, p, gt, mo, p, p, ms, ms, None, p, n, o)
    assert new(o=None) == new(w=None) == new(mo=1) == gs.GS_ERR_NULL
    assert new(n=-1) == gs.GS_ERR_SHAPE
    assert new(gt=5) == new(mo=2) == gs.GS_ERR_DTYPE
    assert new(ms=p) == gs.GS_ERR_ARG
    assert lib.gs_adamw_list_destroy(None) == gs.GS_OK
    # the list is looked at after everything else
    step = lambda li=p, lr=1e-3, b1=0.9, b2=0.999, eps=1e-8, wd=0.0, mx=0.0, nrm=None, f=p, s=p: \
        lib.gs_master_update_adamw(li, lr, b1, b2, eps, wd, mx, nrm, f, s, 0, None)  # noqa: E731
    assert step(li=None) == step(f=None) == step(s=None) == step(mx=1.0) == gs.GS_ERR_NULL
    nan, inf = float("nan"), float("inf")
    for bad in (dict(lr=-1.0), dict(lr=nan), dict(b1=1.0), dict(b1=nan), dict(b2=-0.5), dict(eps=-1.0),
                dict(wd=inf), dict(mx=nan), dict(s=ctypes.c_void_p(0x1004)), dict(f=ctypes.c_void_p(0x1002))):
        assert step(**bad) == gs.GS_ERR_ARG, bad


class NoList:
    handle = None       # the library refuses it: no call gets as far as the device


def test_adamw_scalars_have_the_type_the_kernel_reads(gs):
    """The step's number is read and written as 8 bytes: a tensor of another
    type or length is refused before the library sees its address."""
    import torch
    one = lambda dtype, n=1: torch.zeros(n, dtype=dtype)  # noqa: E731
    good = dict(step=one(torch.int64), found_inf=one(torch.int32), grad_norm=one(torch.float32))
    with pytest.raises(gs.GsError):
        gs.gs_master_update_adamw(NoList, lr=1e-3, stream=0, **good)
    with pytest.raises(gs.GsError):
        gs.gs_master_update_adamw(NoList, lr=1e-3, stream=0, **{**good, "grad_norm": None, "step": one(torch.int64)[0]})
    for bad in (dict(step=one(torch.int32)), dict(step=one(torch.float32)), dict(step=one(torch.int64, 2)),
                dict(step=one(torch.int64, 0)), dict(found_inf=one(torch.bool)), dict(found_inf=one(torch.int64)),
                dict(found_inf=one(torch.int32, 3)), dict(grad_norm=one(torch.float64)),
                dict(grad_norm=one(torch.float16)), dict(grad_norm=one(torch.float32, 2))):
        with pytest.raises(ValueError):
            gs.gs_master_update_adamw(NoList, lr=1e-3, stream=0, **{**good, **bad})


def test_layernorm_workspace_is_one_piece(gs):
    """The workspace is written from its first byte on: a view with gaps, whose
    elements would count as enough, is refused, and so is a short one."""
    import torch
    x, mean, rstd, dg = torch.zeros(4, 64), torch.zeros(4), torch.ones(4), torch.zeros(64)
    n = gs.gs_layernorm_ws_bytes(4, 64)
    assert n >= 4 * 2 * 64 * 4
    bwd = lambda ws: gs.gs_layernorm_bwd(x, x, None, mean, rstd, torch.zeros_like(x), dg, None, ws, stream=0)  # noqa: E731
    with pytest.raises(ValueError):
        bwd(torch.zeros(2 * n, dtype=torch.uint8)[::2])
    with pytest.raises(ValueError):
        bwd(torch.zeros(n - 1, dtype=torch.uint8))
    with pytest.raises(gs.GsError):                  # host memory
        bwd(torch.zeros(n, dtype=torch.uint8))
