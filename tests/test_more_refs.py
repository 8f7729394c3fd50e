"""The restatements behind the GPU tests of the 4-bit tensors, the policy loss
and the orthogonalised momentum, pinned on the CPU: formats against their
definitions, gradients against differences, the polynomial against singular
values."""
import math

import numpy as np
import pytest
import torch

import more_refs as mr


def test_nearest_against_search():
    rng = np.random.default_rng(1)
    t = mr.e4m3_table()
    assert t[-1] == 448 and t[1] == 2.0 ** -9 and t[8] == 2.0 ** -6 and len(t) == 127
    for table in (mr.E2M1, t):
        mid = (table[1:] + table[:-1]) / 2
        v = np.concatenate([table, mid, np.nextafter(mid, 0), np.nextafter(mid, 1e9), rng.random(500) * table[-1] * 1.2])
        got = mr.nearest(table, v)
        for x, c in zip(v, got):
            d = np.abs(table - x)
            best = np.flatnonzero(d == d.min())
            assert c == (best[0] if len(best) == 1 else best[best % 2 == 0][0]), x


def test_torch_agrees_on_e4m3():
    v = torch.rand(4000, dtype=torch.float32) * 500
    want = v.clamp(max=448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert (mr.nearest(mr.e4m3_table(), v.double().numpy()) == want).all()


@pytest.mark.parametrize("fmt", ["nvfp4", "mxfp4"])
def test_quantised_values_are_near(fmt):
    """Half a step of e2m1 is at most a quarter of the value in [1, 6] and 0.25
    below, plus what saturation at 6 cuts off: the largest is at most 8 (MXFP4)
    or 6 (1 + 2^-4) (the scale's rounding) units."""
    x = np.random.default_rng(2).standard_normal((64, 128)).astype(np.float32)
    ts = mr.tensor_scale(x) if fmt == "nvfp4" else None
    c, s = mr.quantise(x, fmt, ts)
    v = mr.values(c, s, fmt, ts)
    unit = np.repeat(mr.values(np.full((64, 128 // mr.BLOCK[fmt]), 2, np.uint8).repeat(mr.BLOCK[fmt], 1), s, fmt, ts)[:, ::mr.BLOCK[fmt]],
                     mr.BLOCK[fmt], 1)
    assert (np.abs(v - x) <= np.maximum(0.25 * unit, np.abs(x) * 0.25) + 1e-6).all()
    assert (mr.unpack(mr.pack(c)) == c).all()


def test_scale_places_are_all_different():
    s = np.arange(300 * 10, dtype=np.int64).reshape(300, 10) % 251 + 1
    out = mr.tiles(s.astype(np.uint8), "nvfp4")
    assert out.size == 3 * 3 * 512 and (out > 0).sum() == s.size


@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
@pytest.mark.parametrize("dual", [0.0, 2.0])
def test_policy_gradient_against_differences(reduction, dual):
    torch.manual_seed(3)
    T = 40
    off = torch.tensor([0, 5, 5, 20, 40])
    lp, old = torch.randn(T, dtype=torch.float64), torch.randn(T, dtype=torch.float64)
    ref, adv = torch.randn(T, dtype=torch.float64), torch.randn(4, dtype=torch.float64)
    tg = torch.where(torch.arange(T) % 3 == 0, -1, 7)
    f = lambda v: mr.policy_loss(v, old, adv, ref, tg, off, 0.2, 0.3, dual, 0.1, reduction)[0]  # noqa: E731
    grad = mr.policy_loss(lp, old, adv, ref, tg, off, 0.2, 0.3, dual, 0.1, reduction)[2]
    h = 1e-6
    for i in range(T):
        e = torch.zeros(T, dtype=torch.float64)
        e[i] = h
        # central differences: h^2 times third derivatives, none of which is above 100 here
        assert abs((f(lp + e) - f(lp - e)) / (2 * h) - float(grad[i])) < 1e-6


def test_policy_loss_against_autograd_of_its_usual_form():
    torch.manual_seed(4)
    T = 200
    lp = torch.randn(T, dtype=torch.float64, requires_grad=True)
    old, ref, adv = (torch.randn(T, dtype=torch.float64) for _ in range(3))
    rho = torch.exp(lp - old)
    obj = torch.minimum(rho * adv, rho.clamp(0.8, 1.3) * adv)
    obj = torch.where(adv < 0, torch.maximum(obj, 2.5 * adv), obj)
    y = ref - lp
    loss = (-obj + 0.1 * (torch.exp(y) - 1 - y)).mean()
    loss.backward()
    got, _, grad, _ = mr.policy_loss(lp.detach(), old, adv, ref, None, None, 0.2, 0.3, 2.5, 0.1)
    assert abs(got - float(loss)) < 1e-12 and torch.allclose(grad, lp.grad, atol=1e-14)


@pytest.mark.parametrize("shape", [(8, 20), (20, 8), (6, 6), (1, 9)])
def test_orthogonalise_moves_singular_values_alone(shape):
    torch.manual_seed(5)
    u = torch.randn(shape, dtype=torch.float64)
    x = mr.orthogonalise(u, 3)
    p, s, q = torch.linalg.svd(u / torch.linalg.norm(u), full_matrices=False)
    a, b, c = mr.QUINTIC
    for _ in range(3):
        s = a * s + b * s ** 3 + c * s ** 5
    assert torch.allclose(x, p @ torch.diag(s) @ q, atol=1e-12)
    # bounds the 16-bit operands' powers of two rely on
    z = torch.linspace(0, 1.21, 10001, dtype=torch.float64)
    assert float((a * z + b * z ** 3 + c * z ** 5).abs().max()) < 1.21
    assert float((a - 1 + b * z ** 2 + c * z ** 4).abs().max()) < 2.45
    assert math.isclose(float(torch.linalg.norm(mr.orthogonalise(torch.zeros(3, 4), 5))), 0.0)
