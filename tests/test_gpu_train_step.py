"""The operators of a training step together, as examples/mixed_precision_step.py
runs them: against a torch step of the same layers, and over many steps."""
import importlib.util
import math
import os

import pytest
import torch

from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    torch.cuda.set_device(0)
    spec = importlib.util.spec_from_file_location(
        "mixed_precision_step", os.path.join(ROOT, "examples", "mixed_precision_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_gradients_against_autograd(ex):
    """dx and the unscaled gradients of one step against autograd in float64 on
    the logits the step itself formed (so that FP8 rounding is not compared):
    fp16 gradients and products of them, a relative 2-norm of 2^-8 (eight
    roundings' worth of 2^-11)."""
    head = ex.Head(256, 256, 384, scale=256.0)
    x, target = next(ex.batches(head))
    w0 = head.w_bf16.clone()
    head.step(x, target)
    assert int(head.found_inf) == 0 and int(head.head_step) == 1 and int(head.norm_step) == 1
    xd = x.double().requires_grad_()
    g = torch.ones(256, device="cuda", dtype=torch.float64, requires_grad=True)
    b = torch.zeros(256, device="cuda", dtype=torch.float64, requires_grad=True)
    w = w0.double().requires_grad_()
    y = torch.nn.functional.layer_norm(xd, (256,), g, b, 1e-5)
    z = y @ w.t()
    z = z + (head.logits.double() - z).detach()
    loss = torch.nn.functional.nll_loss(torch.log_softmax(z, 1), target, ignore_index=-100,
                                        reduction="sum") / head.tokens
    loss.backward()
    for got, want in ((head.grads[0], w.grad), (head.grads[1], g.grad), (head.grads[2], b.grad),
                      (head.dx.double() / 256.0, xd.grad)):
        assert float((got.double() - want).norm() / want.norm()) < 2.0 ** -8
    norm = math.sqrt(sum(float(t.double().square().sum()) for t in head.grads))
    assert math.isclose(float(head.grad_norm), norm, rel_tol=1e-5)


def test_loss_falls_and_overflowing_steps_are_skipped(ex):
    losses, head = ex.train(150, tokens=1024, hidden=256, vocab=512)
    skipped = 150 - int(head.head_step)
    assert skipped >= 1 and int(head.norm_step) == int(head.head_step)
    assert float(head.scale) == 2.0 ** (24 - skipped)
    # two equally likely continuations: ln 2 is the best possible
    assert losses[0] > 5.0 and math.log(2) - 0.1 < losses[-1] < 1.5, (losses[0], losses[-1])
