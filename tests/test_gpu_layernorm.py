"""Layer norm and its backward pass against 64-bit restatements.

Tolerances.  A sum of n terms added by at least 32 threads has at most
n / 32 + 16 dependent additions, each with relative error 2^-24: a sum is off
by at most c = (n / 32 + 16) 2^-24 of the sum of magnitudes.  From there:
  mean:  c E|x|
  rstd:  relative c + (2 c E|x| + 2^-22 (|mean| + E|x - mean|))
         E|x - mean| rstd^2 + (mean error)^2 rstd^2 + 2^-21
  y:     |gamma| rstd (mean error + 2^-23 (|x| + |mean|)) +
         |gamma xhat| (rstd error + 2^-21) + 2^-22 |beta|, and half an ulp
         of the type
and likewise for the gradients, each term below."""
import numpy as np
import pytest
import torch

import train_refs as tr
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
E = tr.EPS24


@pytest.fixture(scope="module")
def gs():
    import mixed_precision_numerics_gradscaler_gb300 as gs
    torch.cuda.set_device(0)
    return gs


def rounded(want, dtype):
    return want.abs() * HALF_ULP[dtype] + (2.0 ** -25 if dtype == torch.float16 else 0.0)


def check(got, want, tol, what):
    got = got.double()
    ok = (got - want).abs() <= tol
    assert ok.all(), (what, int((~ok).sum()), float(((got - want).abs() - tol)[~ok].max()))


def rows(R, C, pad, dtype, gen, scale=1.0, shift=0.0, offset=0):
    """A [R, C] view with pad elements between rows, starting `offset`
    elements into its buffer; the buffer too."""
    buf = torch.full((offset + R * (C + pad) + 8,), 7.0, dtype=dtype, device=DEV)
    x = buf.as_strided((R, C), (C + pad, 1), offset)
    x.copy_(torch.randn(R, C, device=DEV, generator=gen) * scale + shift)
    return x, buf


def gaps_kept(buf, x, offset, fill=7.0):
    mask = torch.ones_like(buf, dtype=torch.bool)
    mask.as_strided(x.shape, x.stride(), offset).fill_(False)
    return bool((buf[mask] == fill).all())


def fwd_case(gs, R, C, dtype, wt, pad=0, offset=0, scale=1.0, shift=0.3, eps=1e-5, affine=True):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(R * 1000003 + C)
    x, _ = rows(R, C, pad, dtype, gen, scale, shift, offset)
    y, ybuf = rows(R, C, pad, dtype, gen, 0.0, 7.0, offset)
    gamma = (1 + 0.2 * torch.randn(C, device=DEV, generator=gen)).to(wt) if affine else None
    beta = (0.2 * torch.randn(C, device=DEV, generator=gen)).to(wt) if affine else None
    mean, rstd = torch.full((R,), 9.0, device=DEV), torch.full((R,), 9.0, device=DEV)
    gs.gs_layernorm_fwd(x, gamma, beta, y, mean, rstd, eps)
    wy, wm, wr = tr.layernorm(x, gamma, beta, eps)
    c = (C / 32 + 16) * E
    xd = x.double()
    ax, dev = xd.abs().mean(1), (xd - wm[:, None]).abs().mean(1)
    em = c * ax + 2 * E * wm.abs()
    check(mean, wm, em, "mean")
    er = c + (2 * em + 4 * E * (wm.abs() + dev)) * dev * wr ** 2 + em ** 2 * wr ** 2 + 8 * E
    check(rstd, wr, wr * er, "rstd")
    g = gamma.double().abs() if affine else torch.ones(C, device=DEV, dtype=torch.float64)
    b = beta.double().abs() if affine else torch.zeros(C, device=DEV, dtype=torch.float64)
    xh = ((xd - wm[:, None]) * wr[:, None]).abs()
    tol = g * wr[:, None] * (em[:, None] + 2 * E * (xd.abs() + wm.abs()[:, None])) + \
        g * xh * (er[:, None] + 8 * E) + 4 * E * b
    check(y, wy, tol * 1.01 + rounded(wy, dtype), "y")
    assert gaps_kept(ybuf, y, offset), "written between the rows"


@pytest.mark.parametrize("C", [1, 2, 7, 31, 32, 33, 64, 127, 128, 255, 1000, 1023, 1024, 2048, 4096,
                               4097, 8192, 10000, 16384, 20001, 33000, 70000])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_forward_sizes(gs, C, dtype):
    for R in (1, 3, 37):
        fwd_case(gs, R, C, TYPES[dtype], torch.float32)


@pytest.mark.parametrize("dtype,wt", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (0, 1), (3, 5), (8, 8), (24, 16)])
def test_forward_strides_and_alignment(gs, dtype, wt, pad, offset):
    for C in (40, 129, 1024, 4096, 9001):
        fwd_case(gs, 19, C, TYPES[dtype], TYPES[wt], pad, offset)


def test_forward_many_rows(gs):
    fwd_case(gs, 20011, 96, torch.bfloat16, torch.float32)
    fwd_case(gs, 70001, 33, torch.float16, torch.float32)
    fwd_case(gs, 5003, 4096, torch.bfloat16, torch.bfloat16)


def test_forward_without_affine_and_with_offset(gs):
    fwd_case(gs, 64, 1000, torch.float32, torch.float32, affine=False)
    # rows whose mean is a hundred standard deviations from zero
    fwd_case(gs, 64, 4096, torch.float32, torch.float32, shift=100.0)
    # rows of one value: variance zero, y = beta
    x = torch.full((5, 640), 3.25, device=DEV)
    y = torch.empty_like(x)
    beta = torch.randn(640, device=DEV)
    gs.gs_layernorm_fwd(x, None, beta, y, None, None, 1e-5)
    assert torch.equal(y, beta.expand(5, -1))


def test_forward_nonfinite_rows_stay_apart(gs):
    x = torch.randn(6, 2048, device=DEV)
    x[1, 5], x[3, 7], x[4, 2047] = float("nan"), float("inf"), float("-inf")
    y, y2 = torch.empty_like(x), torch.empty_like(x)
    gs.gs_layernorm_fwd(x, None, None, y)
    gs.gs_layernorm_fwd(torch.nan_to_num(x), None, None, y2)
    for r in range(6):
        if r in (1, 3, 4):
            assert torch.isnan(y[r]).any()
        else:
            assert torch.equal(y[r], y2[r])


@pytest.mark.parametrize("R,C", [(6000, 8192), (6003, 520), (20003, 200), (5000, 1001)])
def test_nonfinite_rows_among_many(gs, R, C):
    """Rows with NaN or Inf change no other row, forward or backward, whichever
    rows share a barrier with them."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(C)
    x, dy = (torch.randn(R, C, device=DEV, generator=gen).bfloat16() for _ in range(2))
    bad = torch.arange(0, R, 7, device=DEV)
    xb, dyb = x.clone(), dy.clone()
    xb[bad, bad % C], dyb[bad[::2], 0], xb[bad[::3], C - 1] = float("nan"), float("inf"), float("-inf")
    ys = []
    mean, rstd = x.float().mean(1), x.float().var(1).rsqrt()
    for a, d in ((x, dy), (xb, dyb)):
        y, dx = torch.empty_like(x), torch.empty_like(x)
        dg, db = torch.empty(C, device=DEV), torch.empty(C, device=DEV)
        gs.gs_layernorm_fwd(a, None, None, y)
        ws = torch.empty(gs.gs_layernorm_ws_bytes(R, C), dtype=torch.uint8, device=DEV)
        gs.gs_layernorm_bwd(d, a, None, mean, rstd, dx, dg, db, ws)
        ys.append((y, dx))
    keep = torch.ones(R, dtype=torch.bool, device=DEV)
    keep[bad] = False
    assert torch.equal(ys[0][0][keep], ys[1][0][keep]) and torch.equal(ys[0][1][keep], ys[1][1][keep])
    assert torch.isnan(ys[1][0][bad]).any(1).all()
    # where the infinity stands in the NaN's place the gradient holds infinities only
    xh = (xb[bad].double() - mean[bad, None]) * rstd[bad, None]
    d = dyb[bad].double()
    ref = rstd[bad, None] * (d - d.mean(1, keepdim=True) - xh * (d * xh).mean(1, keepdim=True))
    assert torch.equal(torch.isnan(ys[1][1][bad]).any(1), torch.isnan(ref).any(1))
    assert not torch.isfinite(ys[1][1][bad]).all(1).any()


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("R,C", [(5, 1024), (700, 8192), (5000, 512), (64, 16384), (300, 1023), (300, 4097)])
def test_constant_rows_small_eps(gs, R, C, dtype):
    """Rows of one value with a tiny eps: x - mean is 0 however large 1 / sqrt(eps)
    is.  Sums of C equal small integers are exact in fp32; for a C that is no
    power of two the mean's own rounding counts, so there the backward alone."""
    x = (torch.arange(R, device=DEV) % 13 - 6).to(dtype)[:, None].expand(R, C).contiguous()
    ones = torch.ones(C, device=DEV)
    if C & (C - 1) == 0:
        y, rstd = torch.empty_like(x), torch.empty(R, device=DEV)
        gs.gs_layernorm_fwd(x, ones, 0.25 * ones, y, rstd=rstd, eps=1.1e-12)
        assert (y == 0.25).all() and (rstd > 0.9e6).all()
    mean, rstd = x[:, 0].float().contiguous(), torch.full((R,), 987654.3125, device=DEV)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(R)
    dy, dx = torch.randn(R, C, device=DEV, generator=gen).to(dtype), torch.empty_like(x)
    dg, db = torch.ones(C, device=DEV), torch.empty(C, device=DEV)
    ws = torch.empty(gs.gs_layernorm_ws_bytes(R, C), dtype=torch.uint8, device=DEV)
    gs.gs_layernorm_bwd(dy, x, ones, mean, rstd, dx, dg, db, ws)
    assert (dg == 0).all()
    d = dy.double()
    ref = 987654.3125 * (d - d.mean(1, keepdim=True))
    if dtype != torch.float16:  # (1e6 is beyond it)
        # dx: the mean of dy (sum in fp32 over 2^5 terms a thread and a tree of 2^10)
        # and three roundings, each 2^-24 of what it rounds; then the store's
        tol = 1e6 * 64 * 2**-24 * d.abs().amax() + (2**-8 if dtype == torch.bfloat16 else 2**-22) * ref.abs()
        assert ((dx.double() - ref).abs() <= tol).all()


# many rows whose pitch is no multiple of 16 bytes, or is one and their width not
MANY = [(700, 8177, 0), (640, 8001, 3), (2001, 4097, 1), (3100, 2049, 7), (5003, 1025, 0),
        (2500, 2001, 23), (700, 8001, 7), (12001, 515, 0)]


@pytest.mark.parametrize("dtype,wt", [("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("R,C,pad", MANY)
def test_many_odd_rows_forward(gs, R, C, pad, dtype, wt):
    fwd_case(gs, R, C, TYPES[dtype], TYPES[wt], pad=pad)
    fwd_case(gs, R, C, TYPES[dtype], TYPES[wt], pad=pad, offset=8, shift=30.0)
    fwd_case(gs, R, C, TYPES[dtype], TYPES[wt], pad=pad, affine=False)


@pytest.mark.parametrize("dtype,wt", [("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("R,C,pad", [(1900, 8177, 0), (1830, 6001, 1), (3700, 4001, 3), (5500, 3001, 7),
                                     (7400, 2001, 23), (11003, 1025, 0), (1000, 16383, 0), (930, 9001, 1),
                                     (470, 20001, 2), (200, 40001, 0)])
def test_many_odd_rows_backward(gs, R, C, pad, dtype, wt):
    bwd_case(gs, R, C, TYPES[dtype], TYPES[wt], pad=pad)
    bwd_case(gs, R, C, TYPES[dtype], TYPES[wt], pad=pad, offset=8, dw=torch.float16, sums=(True, False))
    bwd_case(gs, R, C, TYPES[dtype], TYPES[wt], pad=pad, affine=False, sums=(False, False))


@pytest.mark.parametrize("dtype,wt", [("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("R,C,pad", [(400, 16384, 0), (310, 8200, 8), (170, 32768, 0), (80, 65536, 0),
                                     (400, 12001, 1), (200, 16383, 0), (100, 40001, 2)])
def test_wide_rows_forward(gs, R, C, pad, dtype, wt):
    fwd_case(gs, R, C, TYPES[dtype], TYPES[wt], pad=pad)
    fwd_case(gs, R, C, TYPES[dtype], TYPES[wt], pad=pad, offset=8, shift=30.0)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("R,C", [(1, 8200), (3, 65536), (37, 65528), (161, 12000), (600, 16384), (90, 32768), (77, 4100)])
def test_wide_rows_backward(gs, R, C, dtype):
    """Rows that several CTAs share."""
    bwd_case(gs, R, C, TYPES[dtype], torch.float32)
    bwd_case(gs, R, C, TYPES[dtype], torch.float32, pad=8, offset=8, sums=(False, True))
    bwd_case(gs, R, C, TYPES[dtype], TYPES[dtype], affine=False, dw=TYPES[dtype])


@pytest.mark.parametrize("pads", [(1, 1, 1), (1, 9, 17), (7, 2, 0)])
def test_odd_rows_neighbours(gs, pads):
    """What stands between odd rows, and in the rows beside them, is none of a row's
    business: NaN there changes nothing; pitches that agree modulo 8 or do not."""
    R, C = 2000, 8001
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)

    def view(pad, like=None):
        buf = torch.full((R, C + pad), float("nan"), dtype=torch.bfloat16, device=DEV)
        v = buf[:, :C]
        v.copy_(torch.randn(R, C, device=DEV, generator=gen) if like is None else like)
        return v

    x, dy = view(pads[0]), view(pads[1])
    bad = torch.arange(3, R, 5, device=DEV)
    keep = torch.ones(R, dtype=torch.bool, device=DEV)
    keep[bad] = False
    gamma = torch.rand(C, device=DEV, generator=gen) + 0.5
    want = None
    for spoilt in (False, True):
        if spoilt:  # whole rows, their first and last columns beside the others' ends
            x[bad], dy[bad] = float("nan"), float("inf")
        y, dx = view(pads[2], 0.0 * x), view(pads[2], 0.0 * x)
        mean, rstd = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
        gs.gs_layernorm_fwd(x, gamma, None, y, mean, rstd)
        if not spoilt:
            stats = mean.clone(), rstd.clone()
        ws = torch.empty(gs.gs_layernorm_ws_bytes(R, C), dtype=torch.uint8, device=DEV)
        gs.gs_layernorm_bwd(dy, x, gamma, *stats, dx, torch.empty(C, device=DEV),
                            torch.empty(C, device=DEV), ws)
        got = y[keep], dx[keep], mean[keep], rstd[keep]
        assert all(torch.isfinite(t).all() for t in got)
        assert want is None or all(torch.equal(a, b) for a, b in zip(got, want))
        assert torch.isnan(y._base[:, C:]).all() and torch.isnan(dx._base[:, C:]).all()
        want = got


def bwd_case(gs, R, C, dtype, wt, pad=0, offset=0, dw=torch.float32, affine=True, sums=(True, True)):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(R * 7919 + C)
    x, _ = rows(R, C, pad, dtype, gen, 1.5, 0.3, offset)
    dy, _ = rows(R, C, pad, dtype, gen, 0.5, 0.1, offset)
    dx, dxbuf = rows(R, C, pad, dtype, gen, 0.0, 7.0, offset)
    gamma = (1 + 0.2 * torch.randn(C, device=DEV, generator=gen)).to(wt) if affine else None
    _, mean, rstd = tr.layernorm(x, None, None, 1e-5)
    mean, rstd = mean.float(), rstd.float()
    dg = torch.full((C,), 9.0, dtype=dw, device=DEV) if sums[0] else None
    db = torch.full((C,), 9.0, dtype=dw, device=DEV) if sums[1] else None
    nbytes = gs.gs_layernorm_ws_bytes(R, C)
    ws = torch.full((nbytes + 256,), 0xAB, dtype=torch.uint8, device=DEV)
    gs.gs_layernorm_bwd(dy, x, gamma, mean, rstd, dx, dg, db, ws[:nbytes])
    wdx, wdg, wdb = tr.layernorm_bwd(dy, x, gamma, mean, rstd)
    assert (ws[nbytes:] == 0xAB).all()
    assert gaps_kept(dxbuf, dx, offset), "written between the rows"
    md, rs = mean.double()[:, None], rstd.double()[:, None]
    xh = ((x.double() - md) * rs).abs()
    eh = rs * 2 * E * (x.double().abs() + md.abs()) + 2 * E * xh      # error of xhat
    d = (dy.double() * (gamma.double() if affine else 1.0)).abs()
    c = (C / 32 + 16) * E
    e1 = (c + 2 * E) * d.mean(1, keepdim=True)
    s2 = (d * xh).mean(1, keepdim=True)
    e2 = (c + 4 * E) * s2 + (d * eh).mean(1, keepdim=True)
    s1 = d.mean(1, keepdim=True)
    tol = rs * (4 * E * (d + s1 + xh * s2) + e1 + xh * e2 + eh * s2)
    check(dx, wdx, tol * 1.01 + rounded(wdx, dtype), "dx")
    cr = (R + 16) * E      # a column's rows may be added one after another
    if sums[0]:
        tol = cr * (dy.double().abs() * xh).sum(0) + (dy.double().abs() * eh).sum(0)
        check(dg, wdg, tol * 1.01 + rounded(wdg, dw), "dgamma")
    if sums[1]:
        check(db, wdb, cr * dy.double().abs().sum(0) + rounded(wdb, dw), "dbeta")


@pytest.mark.parametrize("C", [1, 2, 7, 31, 32, 33, 64, 127, 128, 255, 1000, 1023, 1024, 2048, 4096,
                               4097, 8192, 10000, 16384, 20001, 33000, 70000])
@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
def test_backward_sizes(gs, C, dtype):
    for R in (1, 3, 37, 700 if C <= 10000 else 160):
        bwd_case(gs, R, C, TYPES[dtype], torch.float32)


@pytest.mark.parametrize("dtype,wt", [("bf16", "bf16"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (0, 1), (3, 5), (8, 8), (24, 16)])
def test_backward_strides_and_alignment(gs, dtype, wt, pad, offset):
    for C in (40, 129, 1024, 4096, 9001):
        bwd_case(gs, 203, C, TYPES[dtype], TYPES[wt], pad, offset)


@pytest.mark.parametrize("dw", ["f16", "bf16", "f32"])
def test_backward_gradient_types_and_absent_outputs(gs, dw):
    bwd_case(gs, 300, 1000, torch.bfloat16, torch.float32, dw=TYPES[dw])
    bwd_case(gs, 300, 1000, torch.bfloat16, torch.float32, dw=TYPES[dw], sums=(True, False))
    bwd_case(gs, 300, 1000, torch.bfloat16, torch.float32, dw=TYPES[dw], sums=(False, True))
    bwd_case(gs, 300, 1000, torch.bfloat16, torch.float32, sums=(False, False), affine=False)


def test_backward_many_rows(gs):
    bwd_case(gs, 20011, 96, torch.bfloat16, torch.float32)
    bwd_case(gs, 70001, 33, torch.float16, torch.float32)
    bwd_case(gs, 5003, 4096, torch.bfloat16, torch.bfloat16)


def test_backward_without_rows_writes_zero_sums(gs):
    x = torch.empty(0, 100, device=DEV)
    none = torch.empty(0, device=DEV)
    dg, db = torch.full((100,), 9.0, device=DEV), torch.full((100,), 9.0, device=DEV)
    gs.gs_layernorm_bwd(x, x, None, none, none, torch.empty(0, 100, device=DEV), dg, db, None)
    assert (dg == 0).all() and (db == 0).all()


def test_backward_is_reproducible(gs):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(5)
    R, C = 3001, 2056
    x, dy = (torch.randn(R, C, device=DEV, generator=gen).bfloat16() for _ in range(2))
    mean, rstd = x.float().mean(1), x.float().var(1).rsqrt()
    got = []
    for _ in range(3):
        dx, dg, db = torch.empty_like(x), torch.empty(C, device=DEV), torch.empty(C, device=DEV)
        ws = torch.randint(0, 255, (gs.gs_layernorm_ws_bytes(R, C),), dtype=torch.uint8, device=DEV)
        gs.gs_layernorm_bwd(dy, x, None, mean, rstd, dx, dg, db, ws)
        got.append((dx, dg, db))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_rows_beyond_32_bit_offsets(gs):
    C, ld = 4096, (1 << 31) + 4104
    for off in (0, 1):
        big = torch.empty(2 * ld + C + 8, dtype=torch.bfloat16, device=DEV)
        out = torch.empty_like(big)
        x, y = (b.as_strided((3, C), (ld, 1), off) for b in (big, out))
        gen = torch.Generator(device=DEV)
        gen.manual_seed(6)
        x.copy_(torch.randn(3, C, device=DEV, generator=gen))
        near, want = x.contiguous(), torch.empty(3, C, dtype=torch.bfloat16, device=DEV)
        gs.gs_layernorm_fwd(x, None, None, y)
        gs.gs_layernorm_fwd(near, None, None, want)
        # bf16 results of sums in another order: one rounding step apart at most
        assert ((y.float() - want.float()).abs() <= want.float().abs() * 2.0 ** -7).all()
        mean, rstd = near.float().mean(1), near.float().var(1).rsqrt()
        wdx, dg, db = torch.empty_like(near), torch.empty(C, device=DEV), torch.empty(C, device=DEV)
        dg2, db2 = torch.empty_like(dg), torch.empty_like(db)
        ws = torch.empty(gs.gs_layernorm_ws_bytes(3, C), dtype=torch.uint8, device=DEV)
        gs.gs_layernorm_bwd(x, x, None, mean, rstd, y, dg, db, ws)
        gs.gs_layernorm_bwd(near, near, None, mean, rstd, wdx, dg2, db2, ws)
        bound = wdx.float().abs() * 2.0 ** -7 + 2.0 ** -16
        assert ((y.float() - wdx.float()).abs() <= bound).all()
        assert torch.allclose(dg, dg2, rtol=1e-5, atol=1e-5) and torch.allclose(db, db2, rtol=1e-5, atol=1e-5)
        del big, out, x, y
        torch.cuda.empty_cache()


def test_runs_on_the_given_stream_and_in_a_graph(gs):
    x = torch.randn(64, 1000, device=DEV)
    y, want = torch.zeros_like(x), torch.empty_like(x)
    gs.gs_layernorm_fwd(x, None, None, want)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    gs.gs_layernorm_fwd(x, None, None, y, stream=side)
    side.synchronize()
    assert torch.equal(y, want)
    mean, rstd = x.mean(1), x.var(1).rsqrt()
    dx, dg, db = torch.empty_like(x), torch.empty(1000, device=DEV), torch.empty(1000, device=DEV)
    ws = torch.empty(gs.gs_layernorm_ws_bytes(64, 1000), dtype=torch.uint8, device=DEV)
    gs.gs_layernorm_bwd(x, x, None, mean, rstd, dx, dg, db, ws)
    wanted = [t.clone() for t in (dx, dg, db)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        gs.gs_layernorm_fwd(x, None, None, y)
        gs.gs_layernorm_bwd(x, x, None, mean, rstd, dx, dg, db, ws)
    for t in (y, dx, dg, db):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and all(torch.equal(a, b) for a, b in zip((dx, dg, db), wanted))


def test_refusals(gs):
    x = torch.randn(8, 64, device=DEV)
    y = torch.empty_like(x)
    with pytest.raises(gs.GsError):
        gs.gs_layernorm_fwd(x, None, None, x)                      # in place
    with pytest.raises(gs.GsError):
        gs.gs_layernorm_fwd(x, None, None, y, eps=-1.0)
    with pytest.raises(gs.GsError):
        gs.gs_layernorm_fwd(x, None, None, y, eps=float("nan"))
    with pytest.raises(gs.GsError):
        gs.gs_layernorm_fwd(x, torch.ones(64, dtype=torch.float16, device=DEV), None, y)
    with pytest.raises(gs.GsError):
        gs.gs_layernorm_fwd(x.cpu(), None, None, y)
    with pytest.raises(ValueError):
        gs.gs_layernorm_fwd(x, torch.ones(63, device=DEV), None, y)
    with pytest.raises(ValueError):
        gs.gs_layernorm_fwd(x, None, None, y.t())
    with pytest.raises(ValueError):
        gs.gs_layernorm_fwd(x, None, None, y.half())
    # columns side by side in one wider buffer do not overlap
    wide = torch.zeros(8, 128, device=DEV)
    wide[:, :64] = x
    gs.gs_layernorm_fwd(wide[:, :64], None, None, wide[:, 64:])
    gs.gs_layernorm_fwd(x, None, None, y)
    assert torch.equal(wide[:, 64:], y) and torch.equal(wide[:, :64], x)
    with pytest.raises(gs.GsError):
        gs.gs_layernorm_fwd(wide[:, :64], None, None, wide[:, 63:127])
    s = torch.ones(8, device=DEV)
    dg = torch.empty(64, device=DEV)
    with pytest.raises(gs.GsError):
        gs.gs_layernorm_bwd(x, x, None, s, s, y, dg, None, None)   # sums without a workspace
    with pytest.raises(ValueError):
        gs.gs_layernorm_bwd(x, x, None, s, s, y, dg, None, torch.empty(4, dtype=torch.uint8, device=DEV))
    ws = torch.empty(gs.gs_layernorm_ws_bytes(8, 64) + 4, dtype=torch.uint8, device=DEV)
    with pytest.raises(gs.GsError):
        gs.gs_layernorm_bwd(x, x, None, s, s, y, dg, None, ws[4:])  # not 16-byte aligned
    with pytest.raises(gs.GsError):
        gs.gs_layernorm_bwd(x, x, None, s, s, y, s[:1].expand(64).clone()[:64], y[0], ws)


# One size at least for every way through the rows: a warp's, a CTA's, the copy
# rings of one and of several CTAs, on and off alignment, element by element,
# rows read again.  (dtype, R, C, pad, offset)
WAYS = [("bf16", 61, 256, 0, 0), ("f32", 61, 512, 0, 0), ("f16", 61, 2048, 0, 0), ("f32", 61, 4096, 0, 0),
        ("bf16", 61, 16384, 0, 0), ("f32", 61, 16384, 0, 0), ("bf16", 61, 40000, 0, 0), ("f32", 61, 20000, 0, 0),
        ("bf16", 5003, 4096, 0, 0), ("f16", 20003, 200, 0, 0), ("f32", 3001, 4096, 0, 0), ("bf16", 1300, 8192, 8, 8),
        ("f16", 5001, 4097, 0, 0), ("bf16", 12001, 1025, 0, 0), ("bf16", 2001, 8001, 3, 8),
        ("bf16", 403, 16384, 0, 0), ("f16", 170, 32768, 0, 0), ("bf16", 83, 65536, 0, 0), ("f32", 100, 16384, 0, 0),
        ("f16", 1003, 12001, 1, 0), ("bf16", 470, 20001, 2, 0), ("bf16", 200, 40001, 0, 0),
        ("bf16", 2003, 100, 1, 1), ("f32", 61, 1001, 0, 1), ("f16", 61, 3001, 0, 1), ("bf16", 61, 5001, 0, 1),
        ("f32", 61, 8001, 0, 1), ("f16", 61, 20001, 0, 1), ("bf16", 152, 8192, 0, 0), ("bf16", 153, 8192, 0, 0),
        ("bf16", 303, 8192, 0, 0), ("bf16", 305, 8192, 0, 0), ("f16", 9001, 264, 0, 0)]


def telling_columns(C):
    """The first and last ones, those about multiples of 256, and some others
    (all of a short row), in no order."""
    rng = np.random.default_rng(C)
    if C <= 2048:
        return rng.permutation(C)
    near = (np.arange(0, C + 1, 256)[:, None] + np.arange(-1, 2)).ravel()
    some = np.concatenate([np.arange(40), np.arange(C - 40, C), near, rng.integers(0, C, 300)])
    return rng.permutation(np.unique(some[(some >= 0) & (some < C)]))


def one_per_row(R, C, columns, first):
    return torch.from_numpy(columns[(np.arange(R) + first) % columns.size]).to(DEV)


@pytest.mark.parametrize("dtype,R,C,pad,offset", WAYS)
def test_forward_every_column_counts_once(gs, dtype, R, C, pad, offset):
    """Rows of zeros but one 1: mean 1 / C, variance (1 - 1 / C) / C.  A column
    left out or read twice makes them 0 or twice that, whatever C is; the
    statistics are allowed 2^-16 of themselves, y two roundings of the type."""
    dt = TYPES[dtype]
    x, _ = rows(R, C, pad, dt, torch.Generator(device=DEV), 0.0, 0.0, offset)
    y, _ = rows(R, C, pad, dt, torch.Generator(device=DEV), 0.0, 7.0, offset)
    mean, rstd = torch.empty(R, device=DEV), torch.empty(R, device=DEV)
    columns, at = telling_columns(C), torch.arange(R, device=DEV)
    wm, wr = 1 / C, C / (1 - 1 / C) ** 0.5 * C ** -0.5
    for first in range(0, columns.size, R):
        c = one_per_row(R, C, columns, first)
        x[at, c] = 1
        gs.gs_layernorm_fwd(x, None, None, y, mean, rstd, 0.0)
        x[at, c] = 0
        assert ((mean.double() / wm - 1).abs() <= 2.0 ** -16).all()
        assert ((rstd.double() / wr - 1).abs() <= 2.0 ** -16).all()
        tol = 2.0 ** -15 + 2 * HALF_ULP[dt]
        peak = y[at, c].double()
        assert ((peak / ((1 - wm) * wr) - 1).abs() <= tol).all()
        y[at, c] = y[at, (c + 1) % C]
        assert ((y.double() / (-wm * wr) - 1).abs().amax() <= tol)


@pytest.mark.parametrize("dtype,R,C,pad,offset", WAYS)
def test_backward_every_column_counts_once(gs, dtype, R, C, pad, offset):
    """xhat = 1 and dy of zeros but one 1 per row: dx = 1[column] - 2 / C, where a
    column left out or read twice makes 2 / C zero or twice that; dgamma and
    dbeta count the rows of each column, exactly."""
    dt = TYPES[dtype]
    x, _ = rows(R, C, pad, dt, torch.Generator(device=DEV), 0.0, 1.0, offset)
    dy, _ = rows(R, C, pad, dt, torch.Generator(device=DEV), 0.0, 0.0, offset)
    dx, _ = rows(R, C, pad, dt, torch.Generator(device=DEV), 0.0, 7.0, offset)
    mean, rstd = torch.zeros(R, device=DEV), torch.ones(R, device=DEV)
    dg, db = torch.empty(C, device=DEV), torch.empty(C, device=DEV)
    ws = torch.empty(gs.gs_layernorm_ws_bytes(R, C), dtype=torch.uint8, device=DEV)
    columns, at = telling_columns(C), torch.arange(R, device=DEV)
    for first in range(0, columns.size, R):
        c = one_per_row(R, C, columns, first)
        dy[at, c] = 1
        gs.gs_layernorm_bwd(dy, x, None, mean, rstd, dx, dg, db, ws)
        dy[at, c] = 0
        count = torch.bincount(c, minlength=C).float()
        assert torch.equal(dg, count) and torch.equal(db, count)
        tol = 2.0 ** -16 + HALF_ULP[dt]
        assert ((dx[at, c].double() - (1 - 2 / C)).abs() <= tol).all()
        dx[at, c] = dx[at, (c + 1) % C]
        assert ((dx.double() * C / -2 - 1).abs().amax() <= tol)


@pytest.mark.parametrize("dtype,R,C,pad,offset", WAYS + [("bf16", 70001, 33, 0, 0), ("f16", 20011, 96, 0, 0),
                                                          ("bf16", 5500, 3001, 7, 0), ("f16", 11003, 1025, 0, 0)])
def test_backward_sums_over_rows_are_exact_for_whole_numbers(gs, dtype, R, C, pad, offset):
    """xhat and dy small whole numbers: every partial sum of dgamma and dbeta is one
    below 2^24, so that any order of addition gives the sums exactly, and a row
    dropped or counted twice shows."""
    r, c = torch.arange(R, device=DEV)[:, None], torch.arange(C, device=DEV)[None, :]
    xi, di = (r * 5 + c * 11) % 9 - 4, 1 + (r * 7 + c * 3 + r // 5) % 3
    x, _ = rows(R, C, pad, TYPES[dtype], torch.Generator(device=DEV), 0.0, 0.0, offset)
    dy, _ = rows(R, C, pad, TYPES[dtype], torch.Generator(device=DEV), 0.0, 0.0, offset)
    x.copy_(xi)
    dy.copy_(di)
    dg, db = torch.empty(C, device=DEV), torch.empty(C, device=DEV)
    ws = torch.full((gs.gs_layernorm_ws_bytes(R, C),), 0xFF, dtype=torch.uint8, device=DEV)
    gs.gs_layernorm_bwd(dy, x, None, torch.zeros(R, device=DEV), torch.ones(R, device=DEV), torch.empty_like(x), dg,
                        db, ws)
    assert torch.equal(db.long(), di.sum(0))
    assert torch.equal(dg.long(), (di * xi).sum(0))
