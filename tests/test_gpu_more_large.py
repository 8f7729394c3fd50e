"""The 4-bit tensors, the policy loss and the orthogonalised momentum past 2^31
and 2^32 elements: what lies at the far end is what the same rows or tokens give
by themselves."""
import pytest
import torch

import more_refs as mr
from gpu_helpers import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gs():
    import mixed_precision_numerics_gradscaler_gb300 as gs
    torch.cuda.set_device(0)
    return gs


def u8(*s):
    return torch.zeros(s, dtype=torch.uint8, device=DEV)


def test_quantise_and_dequantise(gs):
    R, C = 70016, 65536                                  # 4.6e9 elements
    x = torch.randn(1024, C, device=DEV).bfloat16().repeat(69, 1)[:R]
    x[R - 1, C - 1] = 50.0                               # the tensor's largest, at its end
    q, s, ts = u8(R, C // 2), u8(gs.fp4_scale_bytes(R, C, "nvfp4")), torch.zeros(1, device=DEV)
    gs.fp4_quant(x, "nvfp4", q, s, ts, u8(gs.gs_ws_bytes()))
    assert float(ts) == 50.0 / 2688 or abs(float(ts) * 2688 / 50 - 1) < 2.0 ** -23
    a, b = R - 256 - R % 128, R                          # whole scale tiles from a on
    q2, s2 = u8(b - a, C // 2), u8(gs.fp4_scale_bytes(b - a, C, "nvfp4"))
    gs.fp4_quant(x[a:b], "nvfp4", q2, s2, ts)
    assert torch.equal(q[a:], q2) and torch.equal(s[-s2.numel():], s2)
    # the transpose of the same, by its last columns
    qt, st = u8(C, R // 2), u8(gs.fp4_scale_bytes(C, R, "nvfp4"))
    gs.fp4_quant(x, "nvfp4", None, None, ts, None, qt, st)
    cols = x[:, C - 128:].contiguous()
    qt2, st2 = u8(128, R // 2), u8(gs.fp4_scale_bytes(128, R, "nvfp4"))
    gs.fp4_quant(cols, "nvfp4", None, None, ts, None, qt2, st2)
    assert torch.equal(qt[C - 128:], qt2) and torch.equal(st[-st2.numel():], st2)
    del qt, st, x
    y, y2 = torch.empty(R, C, dtype=torch.bfloat16, device=DEV), torch.empty(b - a, C, dtype=torch.bfloat16, device=DEV)
    gs.fp4_dequant(q, s, "nvfp4", y, ts)
    gs.fp4_dequant(q2, s2, "nvfp4", y2, ts)
    assert torch.equal(y[a:], y2)


@pytest.mark.parametrize("M,N,pad", [(49152, 49153, 0), (49152, 49152, 8), (8, 300000001, 0)])
def test_product(gs, M, N, pad):
    K = 64
    gen = torch.Generator(device=DEV)
    gen.manual_seed(1)
    codes = lambda r: torch.randint(0, 256, (r, K // 2), dtype=torch.uint8, device=DEV, generator=gen)  # noqa: E731
    scales = lambda r: torch.full((gs.fp4_scale_bytes(r, K, "mxfp4"),), 127, dtype=torch.uint8, device=DEV)  # noqa: E731
    qa, qb, sa, sb = codes(M), codes(N), scales(M), scales(N)
    d = torch.empty(M, N + pad, dtype=torch.bfloat16, device=DEV)[:, :N]
    gs.fp4_gemm_block_scaled(qa, sa, qb, sb, "mxfp4", d)
    one = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    one = torch.cat([one, -one])
    val = lambda q: torch.stack([one[(q & 15).int()], one[(q >> 4).int()]], 2).flatten(1)  # noqa: E731
    for i, j in ((0, 0), (M - min(M, 300), N - 300), (M // 2, N // 2), (0, N - 300)):
        a, b = val(qa[i:i + 300]), val(qb[j:j + 300])
        want = (a.double() @ b.double().t()).bfloat16()  # whole halves: exact in fp32
        assert torch.equal(d[i:i + 300, j:j + 300], want)
    assert gs.gs_device_status() == gs.GS_OK


def test_policy_loss(gs):
    T, S = (1 << 31) + 1000, 5
    lp, old, adv = (torch.full((T,), v, device=DEV) for v in (-1.0, -1.0, 0.0))
    off = torch.tensor([0, 10, 1 << 20, 1 << 30, (1 << 31) + 300, T], device=DEV)
    at = torch.tensor([5, (1 << 20) + 3, (1 << 31) - 1, (1 << 31) + 299, (1 << 31) + 300, T - 1], device=DEV)
    lp[at] += torch.tensor([0.1, -0.1, 0.5, -0.5, 0.05, 0.2], device=DEV)
    adv[at] = torch.tensor([1.0, -1.0, 2.0, 1.0, -2.0, 3.0], device=DEV)
    grad, loss, stats = torch.zeros(T, device=DEV), torch.zeros(1, device=DEV), torch.zeros(4, device=DEV)
    ws = u8(gs.gs_policy_loss_ws_bytes(T, S))
    gs.gs_policy_loss(lp, old, adv, loss, ws, grad, stats, seq_offsets=off, reduction="sequence")
    w = 1.0 / (off.diff().double() * S)
    seq = torch.searchsorted(off[1:], at, right=True)
    d, a = (lp[at].double() - old[at].double()), adv[at].double()
    rho = d.exp()
    obj = torch.minimum(rho * a, rho.clamp(0.8, 1.2) * a)
    assert abs(float(loss) + float((w[seq] * obj).sum())) <= float((w[seq] * obj.abs()).sum()) * 2.0 ** -20
    want = torch.where(rho * a <= rho.clamp(0.8, 1.2) * a, -rho * a * w[seq], 0.0)
    assert bool(((grad[at].double() - want).abs() <= want.abs() * 2.0 ** -20).all())
    assert int((grad != 0).sum()) == int((want != 0).sum())
    assert float(stats[0]) == float(torch.tensor(float(T)))


@pytest.mark.parametrize("shape", [(8, 1 << 18), (1 << 18, 40), (600, 1 << 18)])
def test_muon_of_the_longest_sums(gs, shape):
    """A sum of n positive products is cut by up to n / 16 2^-24 = 1e-3 of itself,
    half of that in the mean, in G alone, whose part in X's error is at most its own
    (the slope b + 2 c G is below 1 where G is 1): five steps add 2.5e-3 to the
    bounds for short sums."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(2)
    w, m = torch.zeros(shape, device=DEV), torch.zeros(shape, device=DEV)
    g = torch.randn(shape, device=DEV, generator=gen)
    li = gs.gs_muon_list_create([w], [g], [m])
    gs.gs_master_update_muon(li, torch.zeros(1, dtype=torch.int32, device=DEV), 1.0, scale="aspect", nesterov=False)
    f = max(1.0, shape[0] / shape[1]) ** 0.5
    want = -mr.orthogonalise(g, 5) * f
    off = float(torch.linalg.norm(w.double() - want)) / float(torch.linalg.norm(want))
    assert off <= (5.7e-3 if min(shape) < 32 else 3.3e-3) + 2.5e-3, off
    assert gs.gs_device_status() == gs.GS_OK
