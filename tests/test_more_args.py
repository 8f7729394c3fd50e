"""Host-side refusals of the 4-bit tensors', the policy loss's and the
orthogonalised momentum's entry points, before any CUDA call (no GPU needed)."""
import ctypes

import pytest
import torch


@pytest.fixture(scope="module")
def gs():
    import mixed_precision_numerics_gradscaler_gb300 as gs
    return gs


P = ctypes.c_void_p(0x1000)   # never dereferenced
ODD = ctypes.c_void_p(0x1002)


def test_fp4_quant_arguments(gs):
    f = lambda x=P, ld=64, dt=1, R=32, C=64, fmt=0, q=P, s=P, qt=None, st=None, ts=None, ws=None: \
        gs._lib.fp4_quant(x, ld, dt, R, C, fmt, q, s, qt, st, ts, ws, None)  # noqa: E731
    assert f(dt=3) == f(fmt=2) == f(fmt=-1) == gs.GS_ERR_DTYPE
    assert f(C=48, ld=48) == f(ld=63) == f(R=-1) == f(C=-32) == f(R=1 << 40, ld=1 << 40) == gs.GS_ERR_SHAPE
    assert f(R=33, qt=P, st=P) == gs.GS_ERR_SHAPE
    assert f(x=None) == f(q=None) == f(s=None) == f(q=None, s=None) == f(qt=P) == f(st=P) == gs.GS_ERR_NULL
    assert f(fmt=1) == gs.GS_ERR_NULL
    assert f(ts=P) == f(ws=P) == f(q=ODD) == f(s=ODD) == f(fmt=1, ts=ODD) == gs.GS_ERR_ARG
    assert gs.fp4_scale_bytes(1, 32, "nvfp4") == 512 and gs.fp4_scale_bytes(129, 96, "nvfp4") == 4 * 512
    assert gs.fp4_scale_bytes(129, 160, "mxfp4") == 4 * 512 and gs.fp4_scale_bytes(0, 64, "mxfp4") == 0
    assert gs._lib.fp4_scale_bytes(-1, 64, 0) == gs._lib.fp4_scale_bytes(64, 64, 2) == 0


def test_fp4_dequant_and_product_arguments(gs):
    f = lambda q=P, s=P, ts=None, R=4, C=64, fmt=0, ot=1, y=P, ld=64: gs._lib.fp4_dequant(  # noqa: E731
        q, s, ts, R, C, fmt, ot, y, ld, None)
    assert f(ot=5) == f(fmt=3) == gs.GS_ERR_DTYPE
    assert f(C=40, ld=40) == f(ld=32) == f(R=-1) == gs.GS_ERR_SHAPE
    assert f(R=0) == f(C=0) == gs.GS_OK
    assert f(q=None) == f(s=None) == f(y=None) == f(fmt=1) == gs.GS_ERR_NULL
    assert f(ts=P) == f(q=ODD) == f(y=ctypes.c_void_p(0x1001)) == gs.GS_ERR_ARG
    f = lambda qa=P, sa=P, ta=None, qb=P, sb=P, tb=None, M=4, N=8, K=64, fmt=0, ot=1, d=P, ld=8: \
        gs._lib.fp4_gemm_block_scaled(qa, sa, ta, qb, sb, tb, M, N, K, fmt, ot, d, ld, None)  # noqa: E731
    assert f(ot=0) == f(fmt=2) == gs.GS_ERR_DTYPE
    assert f(K=48) == f(M=-1) == f(ld=7) == f(M=1 << 31) == f(K=1 << 31) == f(N=1 << 31, ld=1 << 31) == gs.GS_ERR_SHAPE
    assert f(M=1 << 23, N=1 << 23, ld=1 << 23) == f(K=(1 << 24) + 32) == gs.GS_ERR_SHAPE
    assert f(M=0) == f(N=0, ld=0) == gs.GS_OK
    assert f(qa=None) == f(sb=None) == f(d=None) == f(fmt=1, ta=P) == f(fmt=1, tb=P) == gs.GS_ERR_NULL
    assert f(ta=P) == f(tb=P) == f(qa=ODD) == f(sb=ODD) == gs.GS_ERR_ARG


def test_fp4_binding_checks_shapes(gs):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    x = torch.zeros(32, 64)
    with pytest.raises(ValueError):
        gs.fp4_quant(x, "mxfp4", u8(32, 31), u8(512), stream=0)
    with pytest.raises(ValueError):
        gs.fp4_quant(x, "mxfp4", u8(32, 32), u8(511), stream=0)
    with pytest.raises(ValueError):
        gs.fp4_quant(x, "mxfp4", u8(32, 32), None, stream=0)
    with pytest.raises(ValueError):
        gs.fp4_quant(x, "nvfp4", u8(32, 32), u8(512), torch.zeros(2), stream=0)
    with pytest.raises(ValueError):
        gs.fp4_quant(x, "nvfp4", u8(32, 32), u8(512), torch.zeros(1), u8(64), stream=0)
    with pytest.raises(gs.GsError):                      # host memory
        gs.fp4_quant(x, "mxfp4", u8(32, 32), u8(512), stream=0)
    d = torch.zeros(32, 8)
    with pytest.raises(ValueError):
        gs.fp4_gemm_block_scaled(u8(32, 32), u8(512), u8(8, 48), u8(512), "mxfp4", d, stream=0)
    with pytest.raises(ValueError):
        gs.fp4_dequant(u8(32, 32), u8(512), "mxfp4", torch.zeros(32, 128), stream=0)


def test_policy_loss_arguments(gs):
    f = lambda lp=P, old=P, ref=None, adv=P, na=8, tg=None, T=8, off=None, S=1, lo=0.2, hi=0.2, dual=0.0, kl=0.0, \
        red=0, loss=P, ws=P, g=None: gs._lib.gs_policy_loss(lp, old, ref, adv, na, tg, T, off, S, lo, hi, dual,
                                                            kl, red, None, loss, None, g, ws, None)  # noqa: E731
    nan, inf = float("nan"), float("inf")
    assert f(T=-1) == f(S=0) == f(S=2, na=2) == f(na=7) == f(T=(1 << 40) + 1) == gs.GS_ERR_SHAPE
    for bad in (dict(lo=-0.1), dict(lo=nan), dict(hi=nan), dict(hi=-1.0), dict(dual=0.5), dict(dual=nan), dict(dual=-1.0),
                dict(kl=inf), dict(red=3), dict(red=-1), dict(loss=ODD), dict(ws=ctypes.c_void_p(0x1008)),
                dict(tg=ctypes.c_void_p(0x1004)), dict(g=ODD)):
        assert f(**bad) == gs.GS_ERR_ARG, bad
    assert f(lp=None) == f(old=None) == f(adv=None) == f(loss=None) == f(ws=None) == f(kl=0.1) == gs.GS_ERR_NULL
    assert gs._lib.gs_policy_loss_ws_bytes(-1, 1) == 0 and gs.gs_policy_loss_ws_bytes(100, 7) > 56
    v = torch.zeros(8)
    ws = torch.zeros(gs.gs_policy_loss_ws_bytes(8, 1), dtype=torch.uint8)
    with pytest.raises(ValueError):
        gs.gs_policy_loss(v, torch.zeros(7), v, torch.zeros(1), ws, stream=0)
    with pytest.raises(ValueError):
        gs.gs_policy_loss(v, v, v, torch.zeros(1), ws[:-1], stream=0)
    with pytest.raises(ValueError):
        gs.gs_policy_loss(v, v, v, torch.zeros(1), ws, targets=torch.zeros(8, dtype=torch.int32), stream=0)
    with pytest.raises(KeyError):
        gs.gs_policy_loss(v, v, v, torch.zeros(1), ws, reduction="mean", stream=0)
    with pytest.raises(gs.GsError):                      # host memory
        gs.gs_policy_loss(v, v, v, torch.zeros(1), ws, stream=0)


def test_muon_arguments(gs):
    out = ctypes.c_void_p()
    dims = lambda *v: (ctypes.c_int64 * len(v))(*v)  # noqa: E731
    ptr = (ctypes.c_void_p * 1)(0x1000)
    none = (ctypes.c_void_p * 1)(None)
    odd = (ctypes.c_void_p * 1)(0x1002)
    f = lambda w=ptr, g=ptr, gt=2, m=ptr, r=dims(4), c=dims(8), n=1, o=ctypes.byref(out): \
        gs._lib.gs_muon_list_create(w, None, g, gt, m, r, c, n, o)  # noqa: E731
    assert f(o=None) == f(w=None) == f(g=None) == f(m=None) == f(r=None) == f(c=None) == gs.GS_ERR_NULL
    assert f(w=none) == f(g=none) == f(m=none) == gs.GS_ERR_NULL
    assert f(gt=4) == gs.GS_ERR_DTYPE
    assert f(n=-1) == f(r=dims(-1)) == f(r=dims(1 << 20), c=dims(1 << 11)) == f(r=dims(1 << 40)) == gs.GS_ERR_SHAPE
    assert f(r=dims((1 << 18) + 1), c=dims(1)) == f(r=dims(1), c=dims((1 << 18) + 1)) == gs.GS_ERR_SHAPE
    assert f(w=odd) == f(m=odd) == f(g=odd) == gs.GS_ERR_ARG
    assert gs._lib.gs_muon_list_destroy(None) == gs.GS_OK
    g = lambda li=P, lr=1e-3, mu=0.9, wd=0.0, st=5, sc=0, mx=0.0, nrm=None, fi=P: gs._lib.gs_master_update_muon(  # noqa: E731
        li, lr, mu, wd, 1, st, sc, mx, nrm, fi, None)
    nan, inf = float("nan"), float("inf")
    assert g(li=None) == g(fi=None) == g(mx=1.0) == gs.GS_ERR_NULL
    for bad in (dict(lr=-1.0), dict(lr=nan), dict(wd=inf), dict(mu=1.0), dict(mu=nan), dict(mu=-0.1), dict(st=0),
                dict(st=21), dict(sc=2), dict(mx=nan), dict(fi=ODD)):
        assert g(**bad) == gs.GS_ERR_ARG, bad
    w = [torch.zeros(4, 8)]
    for bad in ((w, w, w + w, None), (w, [torch.zeros(8, 4)], w, None), ([torch.zeros(8)],) * 3 + (None,),
                (w, w, w, w), (w, w, [torch.zeros(8, 4).t()], None)):
        with pytest.raises(ValueError):
            gs.gs_muon_list_create(*bad)
    with pytest.raises(gs.GsError):                      # host memory
        gs.gs_muon_list_create(w, [torch.zeros(4, 8)], [torch.zeros(4, 8)])
