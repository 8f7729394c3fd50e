"""A mixed-precision training step of a language model's last layers, every
operation through the package: layer norm, 1x128 and 128x128 FP8 quantisation,
the block-scaled GEMM of the output head, log probabilities of the next
tokens, their gradient under the loss scale, layer norm's backward pass, the
unscale/check of the FP16 gradients and AdamW on FP32 masters (8-bit moments
for the head, 32-bit ones without decay for the norm).

    python examples/mixed_precision_step.py [steps]

The data is synthetic: token t is followed by one of two fixed tokens.  The
loss scale starts too high on purpose: the first steps overflow, are skipped
on the device and halve the scale until the gradients fit.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mixed_precision_numerics_gradscaler_gb300 as gs  # noqa: E402

DEV = "cuda:0"


class Head:
    """Norm and output head over [tokens, hidden] activations, and the state
    of their training."""

    def __init__(self, tokens: int, hidden: int, vocab: int, scale: float = 2.0 ** 24, seed: int = 0):
        gen = torch.Generator(device=DEV)
        gen.manual_seed(seed)
        self.tokens, self.hidden, self.vocab, self.gen = tokens, hidden, vocab, gen
        f32 = dict(dtype=torch.float32, device=DEV)
        f16 = dict(dtype=torch.float16, device=DEV)
        # masters, their bf16 copy (the head's) and FP16 scaled gradients
        self.w = torch.randn(vocab, hidden, generator=gen, **f32) * 0.02
        self.w_bf16 = self.w.bfloat16()
        self.gamma, self.beta = torch.ones(hidden, **f32), torch.zeros(hidden, **f32)
        self.dw = torch.zeros(vocab, hidden, **f16)
        self.dgamma, self.dbeta = torch.zeros(hidden, **f16), torch.zeros(hidden, **f16)
        grads = [self.dw, self.dgamma, self.dbeta]
        self.grads = [torch.zeros(g.shape, **f32) for g in grads]
        self.tensor_list = gs.gs_tensor_list_create(grads, self.grads)
        # loss scale and what a step reports
        self.scale = torch.full((1,), scale, **f32)
        self.tracker = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.found_inf = torch.zeros(1, dtype=torch.int32, device=DEV)
        self.grad_norm = torch.zeros(1, **f32)
        # AdamW: E4M3 moments for the head, fp32 ones without decay for the norm
        blocks = -(-self.w.numel() // 128)
        codes = lambda: torch.zeros(vocab, hidden, dtype=torch.uint8, device=DEV)  # noqa: E731
        self.head_list = gs.gs_adamw_list_create(
            [self.w], [self.grads[0]], [codes()], [codes()], [torch.zeros(blocks, **f32)],
            [torch.zeros(blocks, **f32)], [self.w_bf16])
        zeros = lambda: [torch.zeros(hidden, **f32) for _ in range(2)]  # noqa: E731
        self.norm_list = gs.gs_adamw_list_create([self.gamma, self.beta], self.grads[1:], zeros(), zeros(),
                                                 decay=[0.0, 0.0])
        self.head_step, self.norm_step = (torch.zeros(1, dtype=torch.int64, device=DEV) for _ in range(2))
        # activations and workspaces, allocated once
        self.y = torch.empty(tokens, hidden, **f16)
        self.mean, self.rstd = torch.empty(tokens, **f32), torch.empty(tokens, **f32)
        self.qy = torch.empty(tokens, hidden, dtype=torch.uint8, device=DEV)
        self.sy = torch.empty(tokens, hidden // 128, **f32)
        self.qw = torch.empty(vocab, hidden, dtype=torch.uint8, device=DEV)
        self.sw = torch.empty(vocab // 128, hidden // 128, **f32)
        self.logits = torch.empty(tokens, vocab, dtype=torch.bfloat16, device=DEV)
        self.logprob, self.lse, self.entropy = (torch.empty(tokens, **f32) for _ in range(3))
        self.top_ids = torch.empty(tokens, 2, dtype=torch.int32, device=DEV)
        self.top_logprob = torch.empty(tokens, 2, **f32)
        self.dlogprob = torch.empty(tokens, **f32)
        self.dlogits = torch.empty(tokens, vocab, **f16)
        self.dx = torch.empty(tokens, hidden, **f16)
        self.ws = torch.empty(gs.gs_layernorm_ws_bytes(tokens, hidden), dtype=torch.uint8, device=DEV)

    def step(self, x: torch.Tensor, targets: torch.Tensor, lr: float = 2e-3) -> None:
        """One training step on fp16 activations x [tokens, hidden]; a negative
        target has no loss.  Nothing is read on the host."""
        # forward: norm, FP8 head, loss
        gs.gs_layernorm_fwd(x, self.gamma, self.beta, self.y, self.mean, self.rstd)
        gs.fp8_quant_block(self.y, 1, 128, "e4m3", self.qy, self.sy)
        gs.fp8_quant_block(self.w_bf16, 128, 128, "e4m3", self.qw, self.sw)
        gs.fp8_gemm_block_scaled(self.qy, self.sy, self.qw, self.sw, "e4m3", self.logits)
        gs.gs_token_logprob(self.logits, targets, self.logprob, self.lse, self.entropy, self.top_ids,
                            self.top_logprob)
        # backward: the mean negative log probability, times the loss scale
        self.dlogprob.fill_(-1.0 / max(1, self.tokens))
        gs.gs_token_logprob_bwd(self.logits, targets, self.lse, self.dlogprob, self.dlogits,
                                loss_scale=self.scale)
        torch.matmul(self.dlogits.t(), self.y, out=self.dw)
        dy = self.dlogits @ self.w_bf16.half()
        gs.gs_layernorm_bwd(dy, x, self.gamma, self.mean, self.rstd, self.dx, self.dgamma, self.dbeta,
                            self.ws)
        # update, skipped on the device if any gradient overflowed
        gs.gs_unscale_check_update_norm(self.tensor_list, self.scale, self.tracker, self.found_inf,
                                        self.grad_norm, None, 2.0, 0.5, 1000)
        clip = dict(max_norm=1.0, grad_norm=self.grad_norm)
        gs.gs_master_update_adamw(self.head_list, self.head_step, self.found_inf, lr, 0.9, 0.99, 1e-8, 0.01,
                                  seed=1, **clip)
        gs.gs_master_update_adamw(self.norm_list, self.norm_step, self.found_inf, lr, 0.9, 0.99, 1e-8, 0.01,
                                  **clip)


def batches(head: Head, seed: int = 1):
    """Endless (activations, next tokens): each token's activation is its fixed
    embedding plus noise, and it is followed by one of two fixed tokens."""
    gen = torch.Generator(device=DEV)
    gen.manual_seed(seed)
    embed = torch.randn(head.vocab, head.hidden, device=DEV, generator=gen)
    follow = torch.randint(0, head.vocab, (head.vocab, 2), device=DEV, generator=gen)
    while True:
        t = torch.randint(0, head.vocab, (head.tokens,), device=DEV, generator=gen)
        pick = torch.randint(0, 2, (head.tokens,), device=DEV, generator=gen)
        noise = 0.1 * torch.randn(head.tokens, head.hidden, device=DEV, generator=gen)
        target = follow[t, pick]
        target[:4] = -100                                    # as for prompt tokens
        yield (embed[t] + noise).half(), target


def train(steps: int, tokens: int = 2048, hidden: int = 512, vocab: int = 1024, report: int = 0):
    """Losses (mean negative log probability) after each step, and the head."""
    head, losses = Head(tokens, hidden, vocab), []
    data = batches(head)
    for s in range(steps):
        x, target = next(data)
        head.step(x, target)
        losses.append(float(-head.logprob[target >= 0].mean()))
        if report and s % report == 0:
            hit = (head.top_ids == target[:, None]).any(1)[target >= 0].float().mean()
            print(f"step {s:4d}  loss {losses[-1]:7.4f}  entropy {float(head.entropy.mean()):6.3f}  "
                  f"target among the first two {float(hit):5.3f}  loss scale {float(head.scale):9.0f}  "
                  f"updates {int(head.head_step)}")
    assert gs.gs_device_status() == gs.GS_OK
    return losses, head


if __name__ == "__main__":
    train(int(sys.argv[1]) if len(sys.argv) > 1 else 200, report=10)
