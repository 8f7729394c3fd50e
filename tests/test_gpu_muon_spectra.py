"""The update by orthogonalised momentum where a few directions are far stronger
than the rest, as a gradient's are, and element by element.

The bound of test_gpu_muon.py, 3.3e-3 sqrt(n / 5) of |X| in the 2-norm, takes every
rounding as relative to what it rounds.  A rounding of X is relative to X's largest
directions and lies in all of them, and five steps raise the smallest ones 3.44^5 =
485 times: the bound holds for such spectra only if X is kept to more than fp16's 11
bits until its last step.  (Products of G's and P's errors with X lie in X's own
directions, which the steps do not raise.)

Element by element: the error's entries have its root mean square in the mean and,
as sums of many independent roundings, a normal distribution; the largest of 2^21 is
5.2 times it.  8 times the bound over the root of the number of elements leaves room,
and is 2.7 % of the update's root mean square: one element in fifty of those left out
would pass.  A row's norm over n elements: the same with sqrt(n) + 8."""
import math

import pytest
import torch

import more_refs as mr
from gpu_helpers import DEV
from test_gpu_muon import make, step, views

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gs():
    import mixed_precision_numerics_gradscaler_gb300 as gs
    torch.cuda.set_device(0)
    return gs


def bound(s, steps):
    return (3.3e-3 if min(s) >= 32 else 5.7e-3) * math.sqrt(max(steps, 5) / 5)


def spiked(shape, rank, ratio, seed):
    """Noise whose largest singular value is 1 and `rank` directions of `ratio`."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    R, C = shape
    rnd = lambda *s: torch.randn(*s, device=DEV, generator=gen, dtype=torch.float64)  # noqa: E731
    a, b = torch.linalg.qr(rnd(R, rank))[0], torch.linalg.qr(rnd(C, rank))[0]
    return ratio * a @ b.t() + rnd(R, C) / (math.sqrt(R) + math.sqrt(C))


def direction(gs, g, steps):
    """X of a gradient alone: masters of zeros, momentum of zeros."""
    w, m = torch.zeros_like(g), torch.zeros_like(g)
    li = gs.gs_muon_list_create([w], [g], [m])
    gs.gs_master_update_muon(li, torch.zeros(1, dtype=torch.int32, device=DEV), 1.0, nesterov=False, ns_steps=steps,
                             scale="aspect")
    f = math.sqrt(max(1.0, g.shape[0] / g.shape[1]))
    return -w.double() / f, mr.orthogonalise(g, steps)


def off(x, want):
    return float(torch.linalg.norm(x - want)) / float(torch.linalg.norm(want))


@pytest.mark.parametrize("steps", [1, 2, 5, 6])
@pytest.mark.parametrize("rank,ratio", [(1, 10.0), (1, 100.0), (1, 1000.0), (1, 1e4), (8, 100.0), (8, 1000.0), (8, 1e5)])
@pytest.mark.parametrize("shape", [(256, 768), (768, 256), (333, 257), (128, 2050)])
def test_strong_directions(gs, shape, rank, ratio, steps):
    x, want = direction(gs, spiked(shape, rank, ratio, rank).float(), steps)
    assert off(x, want) <= bound(shape, steps), off(x, want)
    assert gs.gs_device_status() == gs.GS_OK


def carried(g, steps):
    """Of many steps the quintic no longer raises what is small but moves values
    about near 1, with slopes of up to 3.9 either way: three roundings of 2^-11 /
    sqrt(3) a step, relative to each singular value, times the slopes that its later
    values meet, in quadrature.  Twice that, for errors between two directions, whose
    slope is a difference quotient."""
    a, b, c = mr.QUINTIC
    orbit = [torch.linalg.svdvals(g.double()) / torch.linalg.norm(g.double())]
    for _ in range(steps):
        s = orbit[-1]
        orbit.append(a * s + b * s ** 3 + c * s ** 5)
    total, slope = 0.0, torch.ones_like(orbit[0])
    for k in range(steps - 1, -1, -1):
        total += 2.0 ** -22 * float(((orbit[k + 1] * slope) ** 2).sum())
        s = orbit[k]
        slope = slope * (a + 3 * b * s ** 2 + 5 * c * s ** 4).abs()
    return 2 * math.sqrt(total) / float(torch.linalg.norm(orbit[-1]))


@pytest.mark.parametrize("steps", [10, 20])
@pytest.mark.parametrize("rank,ratio", [(1, 10.0), (1, 1000.0), (1, 1e4), (8, 100.0), (8, 1000.0)])
def test_strong_directions_of_many_steps(gs, rank, ratio, steps):
    g = spiked((256, 768), rank, ratio, 5).float()
    x, want = direction(gs, g, steps)
    assert off(x, want) <= carried(g, steps), (off(x, want), carried(g, steps))


@pytest.mark.parametrize("shape", [(192, 320), (320, 192), (1000, 1500), (2304, 1100)])
@pytest.mark.parametrize("decay", ["1/i", "1/i^2", "exponential"])
def test_decaying_spectra(gs, shape, decay):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(3)
    s = min(shape)
    i = torch.arange(1, s + 1, device=DEV, dtype=torch.float64)
    sv = {"1/i": 1 / i, "1/i^2": 1 / i ** 2, "exponential": 10 ** (-6 * i / s)}[decay]
    rnd = lambda n: torch.linalg.qr(torch.randn(n, s, device=DEV, generator=gen, dtype=torch.float64))[0]  # noqa: E731
    x, want = direction(gs, ((rnd(shape[0]) * sv) @ rnd(shape[1]).t()).float(), 5)
    assert off(x, want) <= bound(shape, 5), off(x, want)


def test_strong_rows_and_elements(gs):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(4)
    g = torch.randn(200, 600, device=DEV, generator=gen)
    rows = g * 10 ** (-3 * torch.arange(200, device=DEV) / 200)[:, None]
    lone = g * 1e-3
    lone[37, 411] = 300.0
    for v in (rows, lone):
        x, want = direction(gs, v, 5)
        assert off(x, want) <= bound((200, 600), 5), off(x, want)


@pytest.mark.parametrize("offset", [0, 1])
@pytest.mark.parametrize("shape", [(64, 64), (65, 63), (100, 1000), (1000, 100), (256, 256), (257, 255), (300, 2000),
                                   (2000, 300), (513, 769), (1024, 2050), (2050, 1030)])
def test_every_element(gs, shape, offset):
    ts = make([shape], "f32", 7, offset)
    w, g, m, _ = views(ts)
    before = w[0].clone(), m[0].clone()
    step(gs, w, g, m, None, 0.02, momentum=0.95, weight_decay=0.1)
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    want, _ = mr.muon(before[0], g[0], before[1], f32(0.02), f32(0.95), f32(0.1))
    moved = want - before[0].double() * (1 - f32(0.02) * f32(0.1))
    unit = bound(shape, 5) * float(torch.linalg.norm(moved)) / math.sqrt(moved.numel())
    err = w[0].double() - want
    assert bool((err.abs() <= 8 * unit + want.abs() * 2.0 ** -22).all()), float(err.abs().max()) / unit
    for dim in (0, 1):
        n = shape[dim]
        e, size = torch.linalg.norm(err, dim=dim), torch.linalg.norm(want, dim=dim)
        assert bool((e <= (math.sqrt(n) + 8) * unit + size * 2.0 ** -22).all())
