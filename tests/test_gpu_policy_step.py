"""Scores, their gradient, the gradient norm, clipping, the FP8 wire and the
expert layer for a few tokens in a run, as the examples use them, each stage
against 64 bits on what it was given; and the examples themselves."""
import math
import os
import subprocess
import sys

import pytest
import torch

import weight_transfer_gb300 as w
from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
import moe_block  # noqa: E402
import policy_step  # noqa: E402

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.mark.parametrize("example", ["policy_step.py", "moe_block.py"])
def test_examples_run(example):
    r = subprocess.run([sys.executable, os.path.join(ROOT, "examples", example)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stdout + r.stderr


def gradients_by_hand(x, head, targets, advantages, temperature, bonus):
    """The loss's gradients in 64 bits, from the bf16 logits as the model made them."""
    logits = (x @ head.T).double() / temperature
    logp = torch.log_softmax(logits, 1)
    p = logp.exp()
    rows = x.shape[0]
    H = -(p * logp).sum(1, keepdim=True)
    d = -p * (-advantages.double() / rows)[:, None]
    d[torch.arange(rows, device=x.device), targets] += -advantages.double() / rows
    d -= p * (logp + H) * (-bonus / rows)
    return d / temperature


def test_gradients_through_the_loss():
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, hidden, vocab = 96, 256, 5003
    x = torch.randn(rows, hidden, generator=g, device="cuda").bfloat16()
    head = (torch.randn(vocab, hidden, generator=g, device="cuda") * 0.1).bfloat16().requires_grad_()
    targets = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    advantages = torch.randn(rows, generator=g, device="cuda")
    logits = x @ head.T
    logits.retain_grad()
    policy_step.policy_loss(logits, targets, advantages, 0.8, 0.02).backward()
    want = gradients_by_hand(x, head.detach(), targets, advantages, float(torch.tensor(0.8)), 0.02)
    # entries of bf16 (half a step 2^-8), 32-bit scores of size up to 20 and their upstream gradients below
    assert ((logits.grad.double() - want).abs() <= want.abs() * (2.0 ** -8 + 200 * U) + 2.0 ** -20 * want.abs().amax(1, keepdim=True)).all()
    assert torch.equal(head.grad, (logits.grad.T @ x))


def test_a_step_of_two_ranks_and_the_wire():
    """Two ranks' gradients summed, averaged, clipped, sent: every stage on the outputs of the one before it."""
    g = torch.Generator(device="cuda").manual_seed(2)
    shapes = [(300, 77), (5003,), (64, 128), (3,)]
    params = [torch.zeros(s, device="cuda", dtype=torch.bfloat16 if i % 2 == 0 else torch.float32) for i, s in enumerate(shapes)]
    trainer = policy_step.Trainer(params, ranks=2, max_norm=0.5)
    for p in params:
        p.grad.copy_(torch.randn(p.shape, generator=g, device="cuda") * 0.01)
    total = math.sqrt(sum(float(p.grad.double().square().sum()) for p in params)) / 2
    norm, codes, scales = trainer.send()
    assert abs(norm[0].item() - total) <= 10 * U * total
    factor = min(1.0, 0.5 / (total + 1e-6)) / 2
    for p, c, q, s in zip(params, trainer.clipped, codes, scales):
        want = p.grad.double().flatten() * factor
        assert ((c.double() - want).abs() <= want.abs() * (2.0 ** -8 + 14 * U)).all()
        n = c.numel()
        back = q.view(torch.float8_e4m3fn).double() * s.double().repeat_interleave(128)[:n]
        top = torch.nn.functional.pad(c.double().abs(), (0, -n % 128)).view(-1, 128).amax(1).repeat_interleave(128)[:n]
        # half a step of e4m3, or of its smallest values, and the scale's rounding
        assert ((back - c.double()).abs() <= c.double().abs() * (2.0 ** -4 + 4 * U) + top / 448 * 2.0 ** -10 * 1.01).all()
    kept = [c.clone() for c in trainer.clipped]
    norm2, codes2, _ = trainer.send()                      # the list serves again, on new gradients too
    assert torch.equal(norm, norm2) and all(torch.equal(a, b) for a, b in zip(codes, codes2))
    for p in params:
        p.grad.mul_(0.25)
    trainer.send()
    small = 0.25 * total
    f = min(1.0, 0.5 / (small + 1e-6)) / 2
    assert all(((c.double() - p.grad.double().flatten() * f).abs() <= p.grad.double().flatten().abs() * f * (2.0 ** -8 + 14 * U)).all()
               for p, c in zip(params, trainer.clipped)) and len(kept) == 4


def test_a_decode_step_with_scores():
    """Norm, routing and experts for a few tokens, logits, the sampled tokens' scores with alternatives."""
    norm_w, router, gate, up, down = moe_block.random_block(16, 256, 128, seed=3)
    block = moe_block.MoeBlock(norm_w, router, gate, up, down, 4)
    g = torch.Generator(device="cuda").manual_seed(4)
    x, residual = (torch.randn(5, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
    out, stream = block.decode(x, residual)
    many, many_stream = block.forward(x, residual)
    assert torch.equal(stream, many_stream)
    # the sorted path rounds h to 8 bits (half a step is 2^-4) and each expert's row to bf16; the layer's output is a sum
    # of 128 * 4 terms of either sign, far below their absolute sum: an eighth of its norm bounds the difference amply
    assert (out.float() - many.float()).norm() <= 0.125 * many.float().norm()
    head = (torch.randn(30011, 256, generator=g, device="cuda") * 0.06).bfloat16()
    logits = (stream + out) @ head.T
    sampled = torch.randint(0, 30011, (5,), generator=g, device="cuda")
    logprobs, top_logprobs, top_ids = policy_step.report(logits, sampled, 5)
    want = torch.log_softmax(logits.double(), 1)
    assert ((logprobs.double() - want.gather(1, sampled[:, None])[:, 0]).abs() <= 1e-4).all()
    assert torch.equal(top_ids, torch.sort(logits.double(), dim=1, descending=True, stable=True).indices[:, :5].int())
    assert ((top_logprobs.double() - want.gather(1, top_ids.long())).abs() <= 1e-4).all()


def test_a_captured_decode_step():
    """The whole step captured into a graph and replayed on new tokens."""
    block = moe_block.MoeBlock(*moe_block.random_block(16, 256, 128, seed=5), 4)
    g = torch.Generator(device="cuda").manual_seed(6)
    head = (torch.randn(5003, 256, generator=g, device="cuda") * 0.06).bfloat16()
    x, residual = (torch.randn(3, 256, generator=g, device="cuda").bfloat16() for _ in range(2))
    sampled = torch.tensor([1, 5002, 77], device="cuda")

    def step():
        out, stream = block.decode(x, residual)
        return policy_step.report((stream + out) @ head.T, sampled, 3)
    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(3):
        x.copy_(torch.randn(3, 256, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, step()))
