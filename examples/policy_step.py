"""A policy-gradient step of an output head on 4-bit products, every operation
through the package: NVFP4 quantisation of activations and weights (as they lie
and transposed, in one pass each), the head's product, log probabilities of the
sampled tokens, the clipped policy loss with its divergence term and gradient,
the gradient of the logits under the loss scale, both backward products in
4 bits, the unscale / check of the FP16 gradient and the update by orthogonalised
momentum, skipped on the device when a gradient overflowed.

    python examples/policy_step.py [steps]

The data is synthetic: sampled tokens of random activations, rewarded when they
lie in the lower half of the vocabulary.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_numerics_gradscaler_gb300 as gs  # noqa: E402

DEV = "cuda:0"


class Codes:
    """A [rows, cols] tensor's NVFP4 codes and scales, its transpose's, and its
    tensor scale; sizes are multiples of 32."""

    def __init__(self, rows: int, cols: int, ws: torch.Tensor):
        u8 = lambda *s: torch.empty(s, dtype=torch.uint8, device=DEV)  # noqa: E731
        self.q, self.s = u8(rows, cols // 2), u8(gs.fp4_scale_bytes(rows, cols, "nvfp4"))
        self.qt, self.st = u8(cols, rows // 2), u8(gs.fp4_scale_bytes(cols, rows, "nvfp4"))
        self.t, self.ws = torch.empty(1, device=DEV), ws

    def quantise(self, x: torch.Tensor) -> None:
        gs.fp4_quant(x, "nvfp4", self.q, self.s, self.t, self.ws, self.qt, self.st)


def product(a, b, d, a_t=False, b_t=False):
    """d = a b^T of two Codes, either of them transposed."""
    qa, sa = (a.qt, a.st) if a_t else (a.q, a.s)
    qb, sb = (b.qt, b.st) if b_t else (b.q, b.s)
    gs.fp4_gemm_block_scaled(qa, sa, qb, sb, "nvfp4", d, a.t, b.t)


class PolicyHead:
    """An output head over [tokens, hidden] activations of `seqs` sequences and
    the state of its training."""

    def __init__(self, tokens: int, hidden: int, vocab: int, seqs: int, scale: float = 2.0 ** 16, seed: int = 0):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(seed)
        f32 = dict(dtype=torch.float32, device=DEV)
        self.tokens, self.vocab, self.gen = tokens, vocab, gen
        self.w = torch.randn(vocab, hidden, generator=gen, **f32) * 0.02
        self.w_bf16 = self.w.bfloat16()
        self.momentum = torch.zeros_like(self.w)
        # products of gradients are bf16; the gradient list that is checked is FP16
        self.dw, self.dw_f16 = (torch.zeros(vocab, hidden, dtype=t, device=DEV) for t in (torch.bfloat16, torch.float16))
        self.grad = torch.zeros(vocab, hidden, **f32)
        self.tensor_list = gs.gs_tensor_list_create([self.dw_f16], [self.grad])
        self.muon = gs.gs_muon_list_create([self.w], [self.grad], [self.momentum], [self.w_bf16])
        self.scale = torch.full((1,), scale, **f32)
        self.tracker, self.found_inf = (torch.zeros(1, dtype=torch.int32, device=DEV) for _ in range(2))
        self.grad_norm = torch.zeros(1, **f32)
        ws = torch.empty(gs.gs_ws_bytes(), dtype=torch.uint8, device=DEV)
        self.x4, self.w4, self.d4 = Codes(tokens, hidden, ws), Codes(vocab, hidden, ws), Codes(tokens, vocab, ws)
        self.logits = torch.empty(tokens, vocab, dtype=torch.bfloat16, device=DEV)
        self.dlogits = torch.empty(tokens, vocab, dtype=torch.bfloat16, device=DEV)
        self.dx = torch.empty(tokens, hidden, dtype=torch.bfloat16, device=DEV)
        self.logprob, self.lse, self.dlogprob = (torch.zeros(tokens, **f32) for _ in range(3))
        self.loss, self.stats = torch.zeros(1, **f32), torch.zeros(4, **f32)
        self.loss_ws = torch.empty(gs.gs_policy_loss_ws_bytes(tokens, seqs), dtype=torch.uint8, device=DEV)

    def forward(self, x: torch.Tensor, targets: torch.Tensor) -> None:
        """Logits and log probabilities of bf16 activations' sampled tokens."""
        self.x4.quantise(x)
        self.w4.quantise(self.w_bf16)
        product(self.x4, self.w4, self.logits)
        gs.gs_token_logprob(self.logits, targets, self.logprob, self.lse)

    def step(self, x, targets, old, ref, advantages, offsets, lr: float = 0.02, reduction: str = "sequence") -> None:
        """One update; nothing is read on the host."""
        self.forward(x, targets)
        gs.gs_policy_loss(self.logprob, old, advantages, self.loss, self.loss_ws, self.dlogprob, self.stats, ref,
                          targets, offsets, None, 0.2, 0.28, 3.0, 0.02, reduction, per_sequence=True)
        gs.gs_token_logprob_bwd(self.logits, targets, self.lse, self.dlogprob, self.dlogits, loss_scale=self.scale)
        self.d4.quantise(self.dlogits)
        product(self.d4, self.w4, self.dx, b_t=True)                 # dX = dY W
        product(self.d4, self.x4, self.dw, a_t=True, b_t=True)       # dW = dY^T X
        self.dw_f16.copy_(self.dw)
        gs.gs_unscale_check_update_norm(self.tensor_list, self.scale, self.tracker, self.found_inf, self.grad_norm,
                                        None, 2.0, 0.5, 1000)
        gs.gs_master_update_muon(self.muon, self.found_inf, lr, 0.9, 0.0, True, 5, "rms", 1.0, self.grad_norm)


def sample(head: PolicyHead, x: torch.Tensor, offsets: torch.Tensor):
    """Tokens drawn from the head's present distribution over x, their log
    probabilities, and a per-sequence advantage: the share of tokens in the
    lower half of the vocabulary, less the mean over sequences."""
    blank = torch.zeros(head.tokens, dtype=torch.int64, device=DEV)
    head.forward(x, blank)
    noise = torch.rand(head.logits.shape, device=DEV, generator=head.gen).clamp(min=1e-20)
    tokens = (head.logits.float() - torch.log(-torch.log(noise))).argmax(1)
    tokens[offsets[:-1].clamp(max=head.tokens - 1)] = -100           # each answer's prompt
    head.forward(x, tokens)
    n = offsets.diff()
    seq = torch.repeat_interleave(torch.arange(n.numel(), device=DEV), n)
    good = ((tokens >= 0) & (tokens < head.vocab // 2)).float()
    share = torch.zeros(n.numel(), device=DEV).index_add_(0, seq, good) / n.clamp(min=1)
    return tokens, head.logprob.clone(), share - share.mean(), share


def train(steps: int, tokens: int = 1024, hidden: int = 256, vocab: int = 512, seqs: int = 16, report: int = 0):
    """Mean rewards before each step, and the head."""
    head, rewards = PolicyHead(tokens, hidden, vocab, seqs), []
    offsets = torch.linspace(0, tokens, seqs + 1, device=DEV).long()
    for s in range(steps):
        # (a mean that is not zero: what a head without biases can learn from)
        x = (torch.randn(tokens, hidden, device=DEV, generator=head.gen) + 0.5).bfloat16()
        targets, old, advantages, share = sample(head, x, offsets)
        head.step(x, targets, old, old, advantages, offsets)
        rewards.append(float(share.mean()))
        if report and s % report == 0:
            n, ratio, held, kl = head.stats.tolist()
            print(f"step {s:4d}  reward {rewards[-1]:6.3f}  loss {float(head.loss):9.5f}  ratio {ratio:6.4f}  "
                  f"held {held:6.4f}  divergence {kl:8.2e}  tokens {n:.0f}  loss scale {float(head.scale):.0f}")
    assert gs.gs_device_status() == gs.GS_OK
    return rewards, head


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 60, report=5)
