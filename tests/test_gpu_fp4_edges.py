"""The product of 4-bit tensors at the edges of its numbers: tensor scales whose
product leaves fp32, empty sums with rows apart and with long rows."""
import numpy as np
import pytest
import torch

import more_refs as mr
from gpu_helpers import DEV
from test_gpu_fp4 import operand

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def gs():
    import mixed_precision_numerics_gradscaler_gb300 as gs
    torch.cuda.set_device(0)
    return gs


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("M,N,K,pad", [(5, 200, 96, 0), (200, 70, 256, 0), (200, 70, 256, 3), (40, 8200, 64, 0)])
@pytest.mark.parametrize("ea,eb", [(-70, -70), (-100, -40), (-40, -100), (-100, -100), (75, 70), (50, 100), (100, 50), (-100, 120), (120, 5)])
def test_scales_whose_product_leaves_fp32(gs, out, M, N, K, pad, ea, eb):
    """ta tb sum with ta tb below or above fp32's range and the result inside it:
    one rounding more than the product's bound has (a factor at a time), 2^-24."""
    rng = np.random.default_rng(M + N + K)
    (ca, sa), (cb, sb) = operand(rng, M, K, "nvfp4", False), operand(rng, N, K, "nvfp4", False)
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    ca[0] = 0                                            # a row of zeros stays one
    ta, tb = (float(np.float32(v)) for v in (1.2345678 * 2.0 ** ea, 1.7654321 * 2.0 ** eb))
    d = torch.full((M, N + pad), 77.0, dtype=TYPES[out], device=DEV)[:, :N]
    gs.fp4_gemm_block_scaled(t(mr.pack(ca)), t(mr.tiles(sa, "nvfp4")), t(mr.pack(cb)), t(mr.tiles(sb, "nvfp4")), "nvfp4", d,
                             torch.full((1,), ta, device=DEV), torch.full((1,), tb, device=DEV))
    a, b = t(mr.values(ca, sa, "nvfp4", 1.0)), t(mr.values(cb, sb, "nvfp4", 1.0))
    want = (a @ b.t()) * ta * tb
    terms = (a.abs() @ b.abs().t()) * ta * tb
    tol = terms * 2.0 ** -23 * (K / 16 + 8)
    step = 2.0 ** -24 if out == "f32" else 2.0 ** -8
    low = 2.0 ** -150 if out == "f32" else 2.0 ** -134     # half the smallest subnormal
    tol = tol + (want.abs() + tol) * (step + 2.0 ** -23) + low + 2.0 ** -150
    most = float(torch.finfo(TYPES[out]).max)
    over = (want.abs() + tol) >= most * (1 + step / 2)
    got = d.double()
    assert bool((got[0] == 0.0).all())
    assert bool((((got - want).abs() <= tol) | over).all())
    assert bool((torch.isinf(got) & (got.sign() == want.sign()))[(want.abs() - tol) > most * (1 + step)].all())
    assert gs.gs_device_status() == gs.GS_OK


@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("M,N,ld", [(5, 9, 16), (5, 9, 9), (1, 9, 16), (3, 300, 301), (40, 1, 7)])
def test_an_empty_sum_writes_its_rows_alone(gs, out, M, N, ld):
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    for fmt, ts in (("mxfp4", None), ("nvfp4", torch.ones(1, device=DEV))):
        buf = torch.full((M, ld), 77.0, dtype=TYPES[out], device=DEV)
        gs.fp4_gemm_block_scaled(u8(M, 0), u8(0), u8(N, 0), u8(0), fmt, buf[:, :N], ts, ts)
        assert bool((buf[:, :N] == 0.0).all()) and bool((buf[:, N:] == 77.0).all())


@pytest.mark.parametrize("ld", [(1 << 29) + 8, 1 << 29])
def test_an_empty_sum_of_long_rows(gs, ld):
    """Rows of 2 GiB and more, as they lie together and apart."""
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)  # noqa: E731
    N = 1 << 29
    buf = torch.full((3, ld), 77.0, device=DEV)
    gs.fp4_gemm_block_scaled(u8(3, 0), u8(0), u8(N, 0), u8(0), "mxfp4", buf[:, :N])
    assert int(torch.count_nonzero(buf[:, :N])) == 0 and bool((buf[:, N:] == 77.0).all())
