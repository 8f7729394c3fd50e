"""The policy loss at the edges of its numbers, against a float64 restatement:
a divergence that is only watched, ratios and divergences beyond fp32's range, NaN
under an advantage of zero, advantages that cancel, one advantage per sequence in a
batch of as many sequences as tokens.

Tolerances, as in test_gpu_policy_loss.py: 2^-20 of the terms' sizes, and half a step
of the result.  d and y = x'' - x are rounded to fp32, 2^-24 |d| and 2^-24 |y| of which
their exponentials carry on: sizes are (2 + |d|) rho |A| and (2 + |y|) (e^y + 1).  A
result beyond fp32's range is its infinity, one below its subnormals within a step of
them."""
import math

import pytest
import torch

import more_refs as mr
from gpu_helpers import DEV
from test_gpu_policy_loss import inputs

pytestmark = pytest.mark.gpu

REDUCTIONS = ["token", "sequence", "sum"]
LENGTHS = [40, 3000, 9001]                               # one CTA's, by either form; many CTAs'


@pytest.fixture(scope="module")
def gs():
    import mixed_precision_numerics_gradscaler_gb300 as gs
    torch.cuda.set_device(0)
    return gs


def f32(v):
    return float(torch.tensor(v, dtype=torch.float32))


def run(gs, i, reduction, dual=0.0, kl=0.0, ref="ref", **k):
    T = i["lp"].numel()
    S = 1 if i["offsets"] is None else i["offsets"].numel() - 1
    ws = torch.full((gs.gs_policy_loss_ws_bytes(T, S),), 0xEE, dtype=torch.uint8, device=DEV)
    loss, stats, grad = torch.zeros(1, device=DEV), torch.zeros(4, device=DEV), torch.full((T,), 17.0, device=DEV)
    gs.gs_policy_loss(i["lp"], i["old"], i["adv"], loss, ws, grad, stats, i[ref] if ref else None, i["targets"],
                      i["offsets"], None, 0.2, 0.28, dual, kl, reduction, **k)
    return float(loss), stats.cpu().double(), grad.cpu().double()


def near(got, want, tol):
    """got (fp32 values in float64) within tol of want, or the infinity that want
    rounds to."""
    got, want, tol = (torch.as_tensor(v, dtype=torch.float64) for v in (got, want, tol))
    most = torch.finfo(torch.float32).max
    at_edge = (want.abs() / most - 1).abs() < 2.0 ** -16  # either side of the last finite value
    ok = torch.where(torch.isinf(want.float()), got == want.float().double(), (got - want).abs() <= tol + 2.0 ** -148)
    ok |= at_edge & (got.sign() == want.sign()) & (got.abs() >= most * (1 - 2.0 ** -15))
    assert bool(ok.all()), (got[~ok], want[~ok])


def sizes(i, weights, dual, kl):
    """What a token's terms are rounded by: the objective as far as it is not held."""
    T = i["lp"].numel()
    d, a = i["lp"].cpu().double() - i["old"].cpu().double(), i["adv"].cpu().double()
    top = torch.where(a > 0, 1.28, dual if dual else math.inf)
    size = (2 + d.abs()) * torch.minimum(d.exp(), top) * a.abs() + 1.28 * a.abs()
    if i["ref"] is not None:
        y = i["ref"].cpu().double() - i["lp"].cpu().double()
        size = size + abs(kl) * (2 + y.abs()) * (y.exp() + 1)
    return torch.where(weights > 0, weights * size, torch.zeros(T, dtype=torch.float64))


def weights_of(i, reduction):
    T = i["lp"].numel()
    live = torch.ones(T, dtype=torch.float64) if i["targets"] is None else (i["targets"].cpu() >= 0).double()
    if reduction == "sum":
        return live
    if reduction == "token":
        return live / live.sum().clamp(min=1)
    off = i["offsets"].cpu()
    seq = torch.searchsorted(off[1:], torch.arange(T), right=True)
    n = torch.zeros(off.numel() - 1, dtype=torch.float64).index_add_(0, seq, live)
    return live / n.clamp(min=1)[seq] / (n > 0).sum().clamp(min=1)


def check(gs, i, reduction, dual=0.0, kl=0.0, **k):
    loss, stats, grad = run(gs, i, reduction, dual, kl, "ref" if i["ref"] is not None else None, **k)
    want, wstats, wgrad, _ = mr.policy_loss(i["lp"], i["old"], i["adv"], i["ref"], i["targets"], i["offsets"],
                                            f32(0.2), f32(0.28), f32(dual), f32(kl), reduction)
    size = sizes(i, weights_of(i, reduction), dual, kl)
    near(grad, wgrad, size * 2.0 ** -20 + wgrad.abs() * 2.0 ** -24)
    near(loss, want, float(size.sum()) * 2.0 ** -20 + abs(want) * 2.0 ** -23)
    # the mean ratio's error counts d's rounding: (2 + |d|) rho, as size has it
    live = torch.ones(i["lp"].numel(), dtype=torch.bool) if i["targets"] is None else i["targets"].cpu() >= 0
    d = (i["lp"].cpu().double() - i["old"].cpu().double())[live]
    n = max(1, d.numel())
    near(stats[1], wstats[1], float(((2 + d.abs()) * d.exp()).sum()) / n * 2.0 ** -20 + abs(wstats[1]) * 2.0 ** -24)
    near(stats[2], wstats[2], 2.0 ** -24)
    if i["ref"] is not None:
        y = (i["ref"].cpu().double() - i["lp"].cpu().double())[live]
        near(stats[3], wstats[3], float(((2 + y.abs()) * (y.exp() + 1)).sum()) / n * 2.0 ** -20 + abs(wstats[3]) * 2.0 ** -24)


def live_places(i, n):
    return (i["targets"] >= 0).nonzero().flatten()[:n] if i["targets"] is not None else torch.arange(n, device=DEV)


@pytest.mark.parametrize("T", LENGTHS)
@pytest.mark.parametrize("reduction", REDUCTIONS)
def test_a_divergence_that_is_only_watched(gs, T, reduction):
    """kl_coef 0 with a reference: loss and gradient do not depend on it, however
    far it is."""
    i = inputs(T, 3, T + 1)
    at = live_places(i, 6)
    i["ref"][at] = i["lp"][at] + torch.tensor([89.0, 120.0, 3e38, 700.0, -math.inf, -200.0], device=DEV)
    loss, stats, grad = run(gs, i, reduction)
    loss0, stats0, grad0 = run(gs, i, reduction, ref=None)
    assert math.isfinite(loss) and bool(torch.isfinite(grad).all())
    assert loss == loss0 and torch.equal(grad, grad0) and torch.equal(stats[:3], stats0[:3])


@pytest.mark.parametrize("T", LENGTHS)
@pytest.mark.parametrize("reduction", REDUCTIONS)
@pytest.mark.parametrize("far", [80.0, 88.7, 89.0, 100.0, 400.0])
@pytest.mark.parametrize("sign,dual", [(1.0, 0.0), (-1.0, 3.0), (-1.0, 0.0)])
def test_ratios_beyond_the_range(gs, T, reduction, far, sign, dual):
    """Counted tokens whose ratio leaves fp32: held where the objective is held,
    else in the loss and the gradient as far as those reach."""
    i = inputs(T, 3, T + 2)
    at = live_places(i, 9)
    i["old"][at] = i["lp"][at] - far
    i["adv"][at] = sign
    check(gs, i, reduction, dual, 0.05)


@pytest.mark.parametrize("T", LENGTHS)
@pytest.mark.parametrize("reduction", REDUCTIONS)
@pytest.mark.parametrize("far", [87.0, 89.0, 95.0, 300.0, -1000.0])
def test_divergences_beyond_the_range(gs, T, reduction, far):
    i = inputs(T, 3, T + 3)
    at = live_places(i, 5)
    i["ref"][at] = i["lp"][at] + far
    check(gs, i, reduction, kl=0.05)
    check(gs, i, reduction, kl=-2.0)


@pytest.mark.parametrize("T", LENGTHS)
def test_sums_beyond_the_range_whose_mean_is_not(gs, T):
    """Ratios of 1e38 and advantages of 1e30 in every token: their sums leave fp32."""
    i = inputs(T, 3, T + 4)
    i["old"] = i["lp"] - 88.0 - 0.5 * torch.rand(T, device=DEV)
    i["ref"] = i["lp"] + 87.5 + 0.5 * torch.rand(T, device=DEV)
    i["adv"] = -i["adv"].abs()
    for reduction in REDUCTIONS:
        check(gs, i, reduction, kl=0.5)
    i["adv"] = i["adv"].abs() * 1e37
    for reduction in REDUCTIONS:
        check(gs, i, reduction, kl=0.5)


@pytest.mark.parametrize("T", LENGTHS)
@pytest.mark.parametrize("reduction", REDUCTIONS)
def test_infinite_log_probabilities(gs, T, reduction):
    """log probability -Inf: ratio 0.  Old one -Inf: ratio Inf, held or not."""
    i = inputs(T, 3, T + 5, ref=False)
    at = live_places(i, 4)
    i["lp"][at[:2]] = -math.inf
    i["old"][at[2:]] = -math.inf
    i["adv"][at] = torch.tensor([1.0, -1.0, 1.0, 2.0], device=DEV)
    loss, stats, grad = run(gs, i, reduction)
    assert math.isfinite(loss) and bool((grad[at.cpu()] == 0.0).all()) and float(stats[1]) == math.inf
    i["adv"][at[3]] = -2.0                               # l = +Inf, its gradient too
    loss, _, grad = run(gs, i, reduction)
    assert loss == math.inf and float(grad[at[3]]) == math.inf and bool((grad[at[:3].cpu()] == 0.0).all())


@pytest.mark.parametrize("T", LENGTHS)
@pytest.mark.parametrize("reduction", REDUCTIONS)
@pytest.mark.parametrize("name", ["lp", "old"])
def test_nan_shows_under_an_advantage_of_zero(gs, T, reduction, name):
    i = inputs(T, 3, T + 6, ref=False)
    i["adv"].zero_()
    loss, _, grad = run(gs, i, reduction)
    assert loss == 0.0 and bool((grad == 0.0).all())
    at = int(live_places(i, 3)[2])
    i[name][at] = math.nan
    loss, stats, grad = run(gs, i, reduction)
    assert math.isnan(loss) and math.isnan(float(grad[at])) and math.isnan(float(stats[1]))
    assert int(torch.isnan(grad).sum()) == 1
    i[name][at] = i["lp" if name == "old" else "old"][at] + (300.0 if name == "lp" else -300.0)
    loss, _, grad = run(gs, i, reduction)                # a ratio beyond fp32 times 0
    assert loss == 0.0 and bool((grad == 0.0).all())


@pytest.mark.parametrize("reduction", REDUCTIONS)
@pytest.mark.parametrize("T,S", [(5120, 16), (1024, 2048), (5121, 16), (5120, 2049), (40000, 16)])
def test_advantages_that_cancel(gs, reduction, T, S):
    """Advantages less their mean, ratios within 2^-19 of 1: the loss is a small part
    of its terms.  Up to 5120 tokens and 2048 sequences A and A (rho - 1) are summed
    apart, the latter to 2^-20 of itself (its series, a product, the sum's steps),
    the former as pairs of fp32 numbers: 2^-40 of the terms.  Beyond, 2^-20 of the
    terms as everywhere."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(T + S)
    off = torch.linspace(0, T, S + 1, device=DEV).long()
    adv = torch.randn(T, device=DEV, generator=gen)
    adv -= adv.mean()
    lp = -torch.exp(torch.randn(T, device=DEV, generator=gen))
    old = lp + (torch.rand(T, device=DEV, generator=gen) - 0.5) * 2.0 ** -18
    i = dict(lp=lp, old=old, adv=adv, ref=None, targets=None, offsets=off)
    loss, _, _ = run(gs, i, reduction, ref=None)
    want, _, _, size = mr.policy_loss(lp, old, adv, None, None, off, f32(0.2), f32(0.28), 0.0, 0.0, reduction)
    terms = float(size.sum())
    moved = float((size.cpu() * torch.expm1(lp.cpu().double() - old.cpu().double()).abs()).sum())
    tol = moved * 2.0 ** -20 + terms * 2.0 ** -40 if T <= 5120 and S <= 2048 else terms * 2.0 ** -20
    assert abs(loss - want) <= tol + abs(want) * 2.0 ** -24


@pytest.mark.parametrize("reduction", REDUCTIONS)
@pytest.mark.parametrize("T", [1, 7, 300, 6000])
def test_as_many_sequences_as_tokens(gs, reduction, T):
    """Some sequences empty, some longer: the length of the advantages does not tell
    whether they are the tokens' or the sequences'."""
    i = inputs(T, T, T + 7)
    check(gs, i, reduction, kl=0.05)                     # unless said: the tokens'
    check(gs, i, reduction, kl=0.05, per_sequence=False)
    loss, stats, grad = run(gs, i, reduction, kl=0.05, per_sequence=True)
    seq = torch.searchsorted(i["offsets"][1:], torch.arange(T, device=DEV), right=True).clamp(max=T - 1)
    each = i | {"adv": i["adv"][seq].contiguous()}
    loss2, stats2, grad2 = run(gs, each, reduction, kl=0.05, per_sequence=False)
    tol = float(sizes(each, weights_of(each, reduction), 0.0, 0.05).sum()) * 2.0 ** -20
    assert abs(loss - loss2) <= tol and torch.equal(stats, stats2)
    assert bool(((grad - grad2).abs() <= grad2.abs() * 2.0 ** -22).all())
    check(gs, each, reduction, kl=0.05, per_sequence=False)


@pytest.mark.parametrize("seed", range(24))
def test_far_tokens_among_others(gs, seed):
    """Lengths from one token on, a few tokens of any distance either way."""
    gen = torch.Generator()
    gen.manual_seed(seed)
    rnd = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=gen))  # noqa: E731
    T = int(math.exp(torch.rand(1, generator=gen).item() * 9.5))
    i = inputs(T, rnd(1, max(1, min(T, 3000))), seed, masked=seed % 3 > 0, ref=seed % 4 > 0)
    for name, other, sign in (("old", "lp", -1), ("ref", "lp", 1)):
        if i[name] is not None:
            at = torch.randint(0, T, (rnd(0, 6),), generator=gen).to(DEV)
            far = (torch.rand(at.numel(), generator=gen) - 0.5) * 600
            i[name][at] = i[other][at] + sign * far.to(DEV)
    check(gs, i, REDUCTIONS[seed % 3], 3.0 if seed % 2 else 0.0, 0.05 if i["ref"] is not None else 0.0)
