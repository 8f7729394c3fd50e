"""4-bit tensors on the GPU: codes and scale bytes against the step-by-step
restatement, equal byte for byte; values exact; products exact where the sums
are whole numbers of fp32's, and within the stated bound elsewhere:
2^-23 (K / 16 + 8) times the sum of the terms' magnitudes (an addition's error
for each 16 products), the scale's product and the output's half step besides."""
import numpy as np
import pytest
import torch

import more_refs as mr
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


@pytest.fixture(scope="module")
def gs():
    import mixed_precision_numerics_gradscaler_gb300 as gs
    torch.cuda.set_device(0)
    return gs


def u8(*shape, fill=0xA5):
    return torch.full(shape, fill, dtype=torch.uint8, device=DEV)


def quant(gs, x, fmt, ts=None, given=False, q=True, qt=False):
    """Runs the quantiser; codes and scales as numpy, with guard bytes checked."""
    R, C = x.shape
    out, guard = [], []
    for want, shape in ((q, (R, C)), (qt, (C, R))):
        if not want:
            out += [None, None]
            continue
        for n in (shape[0] * shape[1] // 2, gs.fp4_scale_bytes(*shape, fmt)):
            buf = u8(n + 64)
            guard.append((buf, n))
            out.append(buf[:n])
        out[-2] = out[-2].view(shape[0], shape[1] // 2)
    scale = None
    if fmt == "nvfp4":
        scale = torch.full((1,), float(ts) if given else -7.0, device=DEV)
    ws = torch.empty(gs.gs_ws_bytes(), dtype=torch.uint8, device=DEV) if fmt == "nvfp4" and not given else None
    gs.fp4_quant(x, fmt, out[0], out[1], scale, ws, out[2], out[3])
    torch.cuda.synchronize()
    assert all(bool((b[n:] == 0xA5).all()) for b, n in guard)
    return [None if t is None else t.cpu().numpy() for t in out], scale


def same_quant(gs, x, fmt, qt=False, ts=None, given=False):
    x32 = x.float().cpu().numpy()
    (q, s, q2, s2), scale = quant(gs, x, fmt, ts, given, True, qt)
    if fmt == "nvfp4" and not given:
        ts = mr.tensor_scale(x32)
        got = scale.cpu().numpy()[0]
        assert got == ts or (np.isnan(got) and np.isnan(ts))
    for got, tiles, ref in ((q, s, x32), (q2, s2, x32.T)) if qt else ((q, s, x32),):
        c, sb = mr.quantise(np.ascontiguousarray(ref), fmt, ts)
        assert (got == mr.pack(c)).all()
        assert (tiles == mr.tiles(sb, fmt)).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R,C,pad,qt", [(1, 32, 0, False), (7, 96, 1, False), (32, 32, 0, True), (128, 128, 8, True),
                                         (160, 672, 0, True), (513, 1056, 3, False), (1024, 1536, 16, True),
                                         (32, 8224, 0, True), (4128, 64, 5, True)])
def test_quantise(gs, fmt, dtype, R, C, pad, qt):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(R + C)
    buf = torch.full((R, C + pad), 1e4, dtype=TYPES[dtype], device=DEV)
    x = buf[:, :C]
    x.copy_(torch.randn(R, C, device=DEV, generator=gen) * torch.exp2(12 * torch.rand(R, 1, device=DEV, generator=gen) - 8))
    same_quant(gs, x, fmt, qt)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_ties_zeros_and_extremes(gs, fmt):
    """Halfway values of every code at exact scales, signed zeros, blocks of
    zeros, subnormal and the largest numbers."""
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 0.0, -0.0, 0.5, 1, 2, 3, 4, 6])
    x = torch.zeros(64, 64)
    x[0] = torch.cat([mid, -mid, mid * 2, -mid * 0.5])
    x[1] = mid.repeat(4) * 2.0 ** 100
    x[2] = mid.repeat(4) * 2.0 ** -130
    x[3] = -0.0
    x[4] = 3e38
    x[5, :16] = 1e-45
    x[6] = torch.arange(64) * 2.0 ** -149
    same_quant(gs, x.to(DEV), fmt, True)
    same_quant(gs, (x[:1] if fmt == "nvfp4" else x[:2]).to(DEV), fmt)
    same_quant(gs, torch.zeros(32, 64, device=DEV), fmt, True)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("bad", [float("inf"), -float("inf"), float("nan")])
def test_non_finite_values_are_scales_of_nan(gs, fmt, bad):
    x = torch.randn(64, 128, device=DEV)
    x[33, 70] = bad
    (q, s, q2, s2), _ = quant(gs, x, fmt, qt=True)
    nan = 255 if fmt == "mxfp4" else 127
    _, k = 33, 70 // mr.BLOCK[fmt]
    hit = mr.tiles(np.full((64, 128 // mr.BLOCK[fmt]), 1, np.uint8), fmt) > 0
    if fmt == "nvfp4":                                   # the tensor's scale is none
        assert (s[hit] == nan).all() and (q == 0).all() and (q2 == 0).all()
        same_quant(gs, x, fmt, True, np.float32(0.01), True)
    else:
        assert (s == nan).sum() == 1 and (s2 == nan).sum() == 1
        assert (mr.unpack(q)[33, 32 * k:32 * k + 32] == 0).all()
        same_quant(gs, x, fmt, True)


def test_given_tensor_scales(gs):
    x = torch.randn(96, 160, device=DEV)
    for ts in (np.float32(0.003), np.float32(1e-4), np.float32(2.0 ** -100), np.float32(2.0 ** 120), np.float32(0),
               np.float32("nan"), np.float32(-1), np.float32("inf"), np.float32(2.0 ** -101)):
        same_quant(gs, x, "nvfp4", True, ts, True)


def test_one_direction_alone_and_empty(gs):
    x = torch.randn(64, 96, device=DEV).bfloat16()
    both, _ = quant(gs, x, "nvfp4", qt=True)
    a, _ = quant(gs, x, "nvfp4")
    b, _ = quant(gs, x, "nvfp4", q=False, qt=True)
    assert (a[0] == both[0]).all() and (a[1] == both[1]).all()
    assert (b[2] == both[2]).all() and (b[3] == both[3]).all()
    _, ts = quant(gs, x[:0], "nvfp4")
    assert float(ts) == float(mr.tensor_scale(np.zeros(0, np.float32)))


def test_every_sixteen_bit_value(gs):
    """Every finite bf16 and fp16 number, each in a block of its own with a
    fixed neighbour."""
    for dtype in (torch.bfloat16, torch.float16):
        v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
        v = v[torch.isfinite(v)]
        x = torch.ones(v.numel(), 32, dtype=dtype)
        x[:, 3] = v
        x[:, 16:] = v[:, None]
        same_quant(gs, x.to(DEV), "mxfp4")
        same_quant(gs, x.to(DEV), "nvfp4", False, np.float32(0.01), True)


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("R,C,pad", [(1, 32, 0), (130, 320, 1), (333, 992, 8), (2600, 4128, 0), (256, 256, 16)])
def test_dequantise(gs, fmt, dtype, R, C, pad):
    rng = np.random.default_rng(R)
    c = rng.integers(0, 16, (R, C)).astype(np.uint8)
    s = rng.integers(0, 127 if fmt == "nvfp4" else 250, (R, C // mr.BLOCK[fmt])).astype(np.uint8)
    s[0, 0] = 127 if fmt == "nvfp4" else 255
    ts = np.float32(0.37)
    buf = torch.full((R, C + pad), 9.0, dtype=TYPES[dtype], device=DEV)
    y = buf[:, :C]
    gs.fp4_dequant(torch.from_numpy(mr.pack(c)).to(DEV), torch.from_numpy(mr.tiles(s, fmt)).to(DEV), fmt, y,
                   torch.full((1,), float(ts), device=DEV) if fmt == "nvfp4" else None)
    # code times scale is exact, times the tensor's rounded to fp32, then to the type
    v = mr.values(c, s, fmt, 1.0)
    want = torch.from_numpy((v * float(ts) if fmt == "nvfp4" else v).astype(np.float32)).to(TYPES[dtype])
    got = y.cpu()
    assert bool(((got == want) | (got.isnan() & want.isnan())).all())
    assert bool((buf[:, C:] == 9.0).all())


def operand(rng, rows, K, fmt, whole):
    """Codes, scale bytes and values; whole: products that add up exactly."""
    c = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    n = K // mr.BLOCK[fmt]
    if fmt == "mxfp4":
        s = rng.integers(127, 129, (rows, n)) if whole else rng.integers(110, 140, (rows, n))
    else:
        s = rng.choice([0x30, 0x38, 0x40], (rows, n)) if whole else rng.integers(1, 126, (rows, n))  # 0.5, 1, 2
    return c, s.astype(np.uint8)


SHAPES = [(1, 1, 32), (1, 128, 64), (1, 4096, 8192), (3, 257, 96), (7, 1000, 4128), (32, 5000, 1024), (33, 64, 160),
          (100, 100, 544), (128, 128, 256), (129, 257, 512), (255, 513, 288), (500, 3, 2048), (700, 1500, 320),
          (2048, 2100, 1056), (4096, 4097, 64)]


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
@pytest.mark.parametrize("out", ["f32", "bf16"])
@pytest.mark.parametrize("M,N,K", SHAPES)
def test_product(gs, fmt, out, M, N, K):
    rng = np.random.default_rng(M + N + K)
    for whole, pad in ((True, 0), (False, 3)):
        (ca, sa), (cb, sb) = operand(rng, M, K, fmt, whole), operand(rng, N, K, fmt, whole)
        t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
        ta, tb = (np.float32(0.5), np.float32(0.75)) if fmt == "nvfp4" else (1.0, 1.0)
        dev = lambda v: torch.full((1,), float(v), device=DEV) if fmt == "nvfp4" else None  # noqa: E731
        buf = torch.full((M, N + pad), 77.0, dtype=TYPES[out], device=DEV)
        d = buf[:, :N]
        args = (t(mr.pack(ca)), t(mr.tiles(sa, fmt)), t(mr.pack(cb)), t(mr.tiles(sb, fmt)), fmt, d, dev(ta), dev(tb))
        gs.fp4_gemm_block_scaled(*args)
        first = d.clone()
        a, b = t(mr.values(ca, sa, fmt, 1.0)), t(mr.values(cb, sb, fmt, 1.0))
        want = a @ b.t() * (float(ta) * float(tb))
        terms = a.abs() @ b.abs().t() * (float(ta) * float(tb))
        tol = torch.zeros_like(terms) if whole else terms * 2.0 ** -23 * (K / 16 + 8)
        tol = tol + (want.abs() + tol) * (2.0 ** -24 if out == "f32" else 2.0 ** -8 + 2.0 ** -24)
        assert bool(((first.double() - want).abs() <= tol).all()), float(((first.double() - want).abs() - tol).max())
        if whole and out == "f32":
            assert bool((first.double() == want).all())
        assert bool((buf[:, N:] == 77.0).all())
        d.fill_(0)
        gs.fp4_gemm_block_scaled(*args)                  # the same sums in the same order
        assert torch.equal(d, first)
    assert gs.gs_device_status() == gs.GS_OK


def test_product_of_nothing_and_of_nan(gs):
    d = torch.full((5, 9), 3.0, device=DEV)
    gs.fp4_gemm_block_scaled(u8(5, 0), u8(0), u8(9, 0), u8(0), "mxfp4", d[:, :7] if False else d)
    assert float(d.abs().max()) == 0.0
    # a block whose scale is NaN makes its row of the product NaN and no other
    rng = np.random.default_rng(4)
    (ca, sa), (cb, sb) = operand(rng, 200, 256, "nvfp4", True), operand(rng, 70, 256, "nvfp4", True)
    sa[131, 5] = 0x7F
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    one = torch.ones(1, device=DEV)
    d = torch.zeros(200, 70, device=DEV)
    gs.fp4_gemm_block_scaled(t(mr.pack(ca)), t(mr.tiles(sa, "nvfp4")), t(mr.pack(cb)), t(mr.tiles(sb, "nvfp4")), "nvfp4",
                             d, one, one)
    bad = d.isnan()
    assert bool(bad[131].all()) and int(bad.sum()) == 70


def test_backward_products_from_transposed_codes(gs):
    """dX = dY W and dW = dY^T X of Y = X W^T from fp4_quant's transposes: the
    product of the values that codes and scales stand for."""
    T, K, N = 160, 256, 320
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)
    mk = lambda *s: torch.randn(*s, device=DEV, generator=gen).bfloat16()  # noqa: E731
    x, w, dy = mk(T, K), mk(N, K), mk(T, N)
    for a, b, want in ((dy, w.t(), (T, K)), (dy.t(), x.t(), (N, K))):
        ops, vals = [], []
        for m in (a, b):                                 # operand [rows, sum]
            flip = m.stride(1) != 1
            src = m.t() if flip else m
            (q, s, qt, st), ts = quant(gs, src, "nvfp4", q=not flip, qt=flip)
            q, s = (qt, st) if flip else (q, s)
            ops += [torch.from_numpy(q).to(DEV), torch.from_numpy(s).to(DEV), ts]
            c, sb = mr.quantise(np.ascontiguousarray(m.float().cpu().numpy()), "nvfp4", np.float32(ts.item()))
            vals.append(torch.from_numpy(mr.values(c, sb, "nvfp4", float(ts))).to(DEV))
        d = torch.empty(want, device=DEV)
        gs.fp4_gemm_block_scaled(ops[0], ops[1], ops[3], ops[4], "nvfp4", d, ops[2], ops[5])
        exact, terms = vals[0] @ vals[1].t(), vals[0].abs() @ vals[1].abs().t()
        assert bool(((d.double() - exact).abs() <= terms * 2.0 ** -23 * (vals[0].shape[1] / 16 + 8)).all())
