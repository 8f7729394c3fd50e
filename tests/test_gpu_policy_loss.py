"""The policy loss and its gradient against a float64 restatement.

Tolerances: a ratio e^d has the relative error of d's rounding, 2^-24 |d|, and of
the exponential, 2^-22; the divergence's terms the same of e^y + 1 (y is at most
two roundings off where it does not cancel).  The gradient multiplies that by
three to four rounded factors, the sums add eight terms in fp32: 2^-20 times the
terms' magnitudes ("size") covers both, and half a step of the results 2^-24."""
import math

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


def inputs(T, S, seed, masked=True, ref=True, per_seq=False, before=0, after=0):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    rnd = lambda n: torch.randn(n, device=DEV, generator=gen)  # noqa: E731
    cut = torch.sort(torch.randint(before, T - after + 1, (S - 1,), device=DEV, generator=gen)).values
    off = torch.cat([torch.tensor([before], device=DEV), cut, torch.tensor([T - after], device=DEV)])
    lp = -torch.exp(rnd(T))
    old = lp - 0.3 * rnd(T)
    r = lp + 0.5 * rnd(T) if ref else None
    tg = torch.where(torch.rand(T, device=DEV, generator=gen) < 0.4, -100, 11) if masked else None
    return dict(lp=lp, old=old, adv=rnd(S if per_seq else T), ref=r, targets=tg, offsets=off)


def check(gs, i, reduction, dual=0.0, kl=0.05, dloss=None, low=0.2, high=0.28, guard=17.0):
    T = i["lp"].numel()
    S = 1 if i["offsets"] is None else i["offsets"].numel() - 1
    kl = 0.0 if i["ref"] is None else kl
    ws = torch.full((gs.gs_policy_loss_ws_bytes(T, S),), 0xEE, dtype=torch.uint8, device=DEV)
    loss, stats = torch.full((1,), guard, device=DEV), torch.full((4,), guard, device=DEV)
    grad = torch.full((T,), guard, device=DEV)
    scale = None if dloss is None else torch.full((1,), dloss, device=DEV)
    run = lambda l, g, s: gs.gs_policy_loss(i["lp"], i["old"], i["adv"], l, ws, g, s, i["ref"], i["targets"],  # noqa: E731
                                            i["offsets"], scale, low, high, dual, kl, reduction)
    run(loss, grad, stats)
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    want, wstats, wgrad, size = mr.policy_loss(i["lp"], i["old"], i["adv"], i["ref"], i["targets"], i["offsets"],
                                               f32(low), f32(high), f32(dual), f32(kl), reduction,
                                               1.0 if dloss is None else dloss)
    g, out = grad.cpu().double(), torch.isnan(wgrad)
    assert bool((g[out] == guard).all())                 # in no sequence: as it was
    tol = size * abs(dloss or 1.0) * 2.0 ** -20 + wgrad.abs() * 2.0 ** -24
    assert bool(((g - wgrad).abs() <= tol)[~out].all())
    total = float(size.sum())
    assert abs(float(loss) - want) <= total * 2.0 ** -20 + abs(want) * 2.0 ** -23
    n = wstats[0]
    assert float(stats[0]) == float(torch.tensor(n).float()) and abs(float(stats[2]) - wstats[2]) <= 2.0 ** -24
    for k in (1, 3):
        assert abs(float(stats[k]) - wstats[k]) <= 2.0 ** -20 * (abs(wstats[k]) + (1.0 if k == 1 else 2.0)) * (3 if n else 0)
    # the same bits again, and the loss alone
    loss2, grad2, loss3 = torch.zeros(1, device=DEV), torch.full((T,), guard, device=DEV), torch.zeros(1, device=DEV)
    run(loss2, grad2, None)
    run(loss3, None, None)
    assert torch.equal(loss, loss2) and torch.equal(grad, grad2) and torch.equal(loss, loss3)


@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
@pytest.mark.parametrize("T,S,masked,ref,per_seq", [
    (1, 1, False, True, True), (5, 9, True, True, True), (255, 3, True, False, False), (1024, 16, True, True, True),
    (1025, 40, False, True, False), (4608, 2048, True, True, True), (4608, 7, True, True, False),
    (4609, 7, True, True, True), (3000, 2049, False, True, True), (20000, 3, False, False, True), (70001, 300, True, True, True),
    (300000, 20000, True, True, True), (262144, 5, True, True, False), (500001, 1, True, False, True)])
def test_loss_and_gradient(gs, reduction, T, S, masked, ref, per_seq):
    i = inputs(T, S, T + S, masked, ref, per_seq)
    check(gs, i, reduction, dual=3.0 if T % 2 else 0.0, dloss=0.25 if S % 2 else None)


@pytest.mark.parametrize("T", [300, 6000, 50000])
@pytest.mark.parametrize("reduction", ["token", "sequence"])
def test_tokens_outside_every_sequence(gs, T, reduction):
    """A buffer longer than its sequences: what lies outside neither counts nor
    is written, NaN or not."""
    i = inputs(T, 5, 3, before=37, after=101, per_seq=True)
    for k in ("lp", "old", "ref"):
        i[k][:37] = math.nan
        i[k][T - 101:] = math.inf
    check(gs, i, reduction)


@pytest.mark.parametrize("T", [500, 9000])
def test_masked_tokens_hold_anything(gs, T):
    i = inputs(T, 4, 5)
    dead = i["targets"] < 0
    for k, v in (("lp", math.nan), ("old", math.inf), ("ref", -math.inf), ("adv", math.nan)):
        i[k][dead] = v
    check(gs, i, "token")
    check(gs, i, "sequence")
    i["targets"].fill_(-1)                               # nothing counts
    for reduction in ("token", "sequence", "sum"):
        check(gs, i, reduction)


@pytest.mark.parametrize("T", [1000, 9000])
def test_without_offsets_and_unaligned(gs, T):
    i = inputs(T, 1, 6)
    i["offsets"] = None
    for reduction in ("token", "sequence", "sum"):
        check(gs, i, reduction)
    j = {k: v for k, v in i.items()} | {"targets": None}
    check(gs, j, "sequence")
    for k in ("lp", "old", "ref", "adv", "targets"):     # views one element on
        i[k] = torch.cat([i[k][:1], i[k]])[1:]
    check(gs, i, "token")
    j["adv"] = i["adv"][:1].clone()                      # one for the only sequence
    if T != 1:
        check(gs, j, "token")


def test_borders_lie_where_the_logarithm_puts_them(gs):
    """Ratios next to a border, told apart by less than fp32's step at 1: the
    difference of two fp32 numbers can lie that near to the logarithm."""
    low, high = 0.2, 0.28
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    lp, old, adv = [], [], []
    for a, border in ((1.0, math.log(1 + f32(high))), (-1.0, math.log(1 - f32(low)))):
        for base in (-0.001, -1.7, -9.3, -40.1):
            for step in range(-3, 4):
                x = torch.tensor(base, dtype=torch.float32)
                y = torch.tensor(float(x) - border, dtype=torch.float32)
                for _ in range(abs(step)):
                    y = torch.nextafter(y, torch.tensor(math.copysign(1e9, step)))
                lp.append(float(x)), old.append(float(y)), adv.append(a)
    t = lambda v: torch.tensor(v, dtype=torch.float32, device=DEV)  # noqa: E731
    i = dict(lp=t(lp), old=t(old), adv=t(adv), ref=None, targets=None, offsets=None)
    check(gs, i, "sum", low=low, high=high)


def test_small_divergences_keep_their_digits(gs):
    T = 256
    y = torch.logspace(-18, 1.5, T, base=2.0, device=DEV) * torch.where(torch.arange(T, device=DEV) % 2 == 0, 1, -1)
    z = torch.zeros(T, device=DEV)
    ws = torch.empty(gs.gs_policy_loss_ws_bytes(T, 1), dtype=torch.uint8, device=DEV)
    loss, stats = torch.zeros(1, device=DEV), torch.zeros(4, device=DEV)
    for k in range(0, T, 16):                            # one at a time: the mean is it
        keep = torch.full((T,), -1, dtype=torch.int64, device=DEV)
        keep[k] = 0
        gs.gs_policy_loss(z, z, z, loss, ws, None, stats, y.float(), keep, None, None, kl_coef=1.0, reduction="sum")
        v = y.float()[k].double()
        want = float(torch.expm1(v) - v)
        # series: a few roundings; beyond 1/2: e^y - 1 - y of e^y to 2^-22
        assert abs(float(loss) - want) <= want * 2.0 ** -21 + (math.exp(float(v)) * 2.0 ** -22 if abs(float(v)) > 0.5 else 0)


def test_extreme_settings(gs):
    i = inputs(2000, 3, 8)
    check(gs, i, "token", low=1.0, high=math.inf)
    check(gs, i, "token", low=5.0, high=0.0)
    check(gs, i, "token", low=0.0, high=0.0, dual=1.0)
    i["adv"].zero_()
    check(gs, i, "token", dual=2.0)
