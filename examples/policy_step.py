"""A policy-gradient step around a weight transfer: scores, their gradient, a bounded gradient norm, the FP8 wire.

The trainer scores the sampled tokens (``score``, differentiable), weighs them with their advantages and an entropy
bonus, averages and clips the gradients that the ranks have summed and quantizes them for the wire.  The inference
engine, on the weights that it was sent, decodes a few tokens through its experts (examples/moe_block.py) and reports
the log probabilities of what it sampled with the alternatives; the two sides' scores of the same tokens are what a
transfer is checked by.

    python examples/policy_step.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_transfer_gb300 as fp8q  # noqa: E402


class _Score(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, targets, temperature):
        logprobs, entropy, _, _, stats = fp8q.fp8q_token_logprobs(logits, targets, temperature, want_entropy=True, want_stats=True)
        ctx.save_for_backward(logits, targets, stats, entropy)
        ctx.temperature = temperature
        return logprobs, entropy

    @staticmethod
    def backward(ctx, dlogprobs, dentropy):
        logits, targets, stats, entropy = ctx.saved_tensors
        return fp8q.fp8q_token_logprobs_backward(logits, targets, stats, dlogprobs.contiguous(), entropy, dentropy.contiguous(),
                                                 ctx.temperature), None, None


def score(logits, targets, temperature=1.0):
    """-> (log probability of each target, entropy of each row), float32; differentiable in the logits."""
    return _Score.apply(logits, targets, temperature)


def policy_loss(logits, targets, advantages, temperature=1.0, bonus=0.01):
    logprobs, entropy = score(logits, targets, temperature)
    return -(advantages * logprobs).mean() - bonus * entropy.mean()


class Trainer:
    """Parameters of one rank, with lasting gradient buffers and what is sent of them."""

    def __init__(self, parameters, ranks: int, max_norm: float, fmt: str = "e4m3"):
        self.parameters, self.ranks, self.max_norm, self.fmt = list(parameters), ranks, max_norm, fmt
        for p in self.parameters:
            p.grad = torch.zeros_like(p)
        self.clipped = [torch.empty(p.numel(), dtype=torch.bfloat16, device=p.device) for p in self.parameters]
        self.grads = fp8q.fp8q_grad_list([p.grad for p in self.parameters], self.clipped)

    def zero_grad(self):
        for p in self.parameters:
            p.grad.zero_()

    def send(self):
        """The gradients (sums over the ranks) averaged, clipped and quantized -> (norm and coefficient, codes, scales)."""
        if not self.grads.holds(p.grad for p in self.parameters):
            raise RuntimeError("a gradient was replaced: use zero_grad(), which keeps the buffers")
        norm, _ = fp8q.fp8q_grad_clip(self.grads, self.max_norm, scale=1.0 / self.ranks)
        codes, scales = fp8q.fp8q_quantize_blockwise_group(self.clipped, self.fmt)
        return norm, codes, scales


def report(logits, sampled, top=5, temperature=1.0):
    """What an engine returns with its tokens -> (their log probabilities, the best alternatives' and their ids)."""
    logprobs, _, top_logprobs, top_ids, _ = fp8q.fp8q_token_logprobs(logits, sampled, temperature, top)
    return logprobs, top_logprobs, top_ids


def main():
    torch.manual_seed(0)
    rows, hidden, vocab, ranks = 512, 1024, 50257, 8
    x = torch.randn(rows, hidden, device="cuda").bfloat16()
    head = torch.nn.Parameter((torch.randn(vocab, hidden, device="cuda") * hidden ** -0.5).bfloat16())
    gain = torch.nn.Parameter(torch.ones(hidden, device="cuda"))
    trainer = Trainer([head, gain], ranks, max_norm=1e-3)
    targets = torch.randint(0, vocab, (rows,), device="cuda")
    advantages = torch.randn(rows, device="cuda")
    logits = (x * gain.bfloat16()) @ head.T
    loss = policy_loss(logits, targets, advantages)
    loss.backward()
    norm, codes, scales = trainer.send()
    logprobs, top_logprobs, top_ids = report(logits.detach(), targets)
    sent = sum(c.numel() + 4 * s.numel() for c, s in zip(codes, scales))
    print(f"loss {loss.item():.4f}, gradient norm {norm[0].item():.3e}, clipped by {norm[1].item():.3f}, {sent / 1e6:.1f} MB sent")
    print(f"mean log probability {logprobs.mean().item():.3f}, best alternative {top_logprobs[:, 0].mean().item():.3f}")


if __name__ == "__main__":
    main()
