"""The 4-bit products, the policy loss and the orthogonalised momentum together,
as examples/policy_step.py runs them: gradients against autograd, steps captured
into a graph, overflowing steps skipped."""
import importlib.util
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location("policy_step", os.path.join(ROOT, "examples", "policy_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def batch(ex, head, seqs=8, seed=1):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    x = torch.randn(head.tokens, head.w.shape[1], device="cuda", generator=gen).bfloat16()
    offsets = torch.linspace(0, head.tokens, seqs + 1, device="cuda").long()
    targets, old, adv, _ = ex.sample(head, x, offsets)
    old = old + 0.2 * torch.randn(old.shape, device="cuda", generator=gen)
    ref = old + 0.2 * torch.randn(old.shape, device="cuda", generator=gen)
    return x, targets, old, ref, adv, offsets


def test_gradients_against_autograd(ex):
    """The gradient of the logits against autograd in float64 of the usual form
    of the loss, on the logits the step formed (bf16 out: half a step of 2^-8
    and fp32's share); the backward products against products of what the codes
    stand for (bf16 out)."""
    gs = ex.gs
    head = ex.PolicyHead(256, 128, 320, 8, scale=1024.0)
    x, targets, old, ref, adv, off = batch(ex, head)
    head.step(x, targets, old, ref, adv, off)
    z = head.logits.double().requires_grad_()
    lp = torch.log_softmax(z, 1).gather(1, targets.clamp(min=0)[:, None])[:, 0]
    seq = torch.repeat_interleave(torch.arange(8, device="cuda"), off.diff())
    a = adv.double()[seq]
    f32 = lambda v: float(torch.tensor(v, dtype=torch.float32))  # noqa: E731
    rho = torch.exp(lp - old.double())
    obj = torch.minimum(rho * a, rho.clamp(1 - f32(0.2), 1 + f32(0.28)) * a)
    obj = torch.where(a < 0, torch.maximum(obj, 3.0 * a), obj)
    y = ref.double() - lp
    live = targets >= 0
    n = torch.zeros(8, device="cuda", dtype=torch.float64).index_add_(0, seq, live.double())
    w = torch.where(live, 1 / (n[seq] * 8), 0.0)
    loss = (w * (f32(0.02) * (torch.exp(y) - 1 - y) - obj)).sum()
    loss.backward()
    want = z.grad * 1024.0
    assert abs(float(head.loss) - float(loss.detach())) < 1e-5
    got = head.dlogits.double()
    # p and the weights carry errors of about 2^-20, of the row's largest entry where p - 1 cancels
    tol = want.abs() * 2.0 ** -8 + want.abs().amax(1, keepdim=True) * 2.0 ** -16
    assert bool(((got - want).abs() <= tol).all())

    def value(c, t):
        q, s = (c.qt, c.st) if t else (c.q, c.s)
        v = torch.empty(q.shape[0], 2 * q.shape[1], device="cuda")
        gs.fp4_dequant(q, s, "nvfp4", v, c.t)
        return v.double()

    for d, left, right in ((head.dx, value(head.d4, False), value(head.w4, True)),
                           (head.dw, value(head.d4, True), value(head.x4, True))):
        exact, terms = left @ right.t(), left.abs() @ right.abs().t()
        # fp32 values of codes: 2^-24 each side; sums as stated; bf16 out
        tol = terms * (2.0 ** -23 * (left.shape[1] / 16 + 8) + 2.0 ** -22) + exact.abs() * 2.0 ** -8
        assert bool(((d.double() - exact).abs() <= tol).all())


def test_steps_run_and_overflowing_ones_are_skipped(ex):
    rewards, head = ex.train(6, tokens=256, hidden=128, vocab=256, seqs=8)
    assert len(rewards) == 6 and bool(torch.isfinite(head.w).all()) and torch.equal(head.w_bf16, head.w.bfloat16())
    head.scale.fill_(2.0 ** 60)                          # FP16 gradients overflow
    keep = head.w.clone(), head.momentum.clone()
    head.step(*batch(ex, head))
    assert int(head.found_inf) == 1 and torch.equal(head.w, keep[0]) and torch.equal(head.momentum, keep[1])
    assert float(head.scale) == 2.0 ** 59


def test_a_captured_step_replays_as_single_steps_do(ex):
    one, two = (ex.PolicyHead(256, 128, 256, 8, scale=256.0) for _ in range(2))
    b = batch(ex, one)
    start = one.w.clone()
    for _ in range(3):
        one.step(*b)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        two.step(*b)                                     # whatever a first call sets up
    torch.cuda.synchronize()
    two.w.copy_(start), two.w_bf16.copy_(start), two.momentum.zero_()
    two.scale.fill_(256.0), two.tracker.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        two.step(*b)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for name in ("w", "w_bf16", "momentum", "loss", "stats", "dlogprob", "dx", "grad", "scale"):
        assert torch.equal(getattr(one, name), getattr(two, name)), name
