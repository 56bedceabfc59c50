"""The expert-block operators together, through examples/moe_block.py.

Serving: against the same block in 64 bits on the dequantized weights, where the only other errors are the roundings of
activations to MXFP8 (e4m3, 3 mantissa bits: a uniform relative error of at most 2^-4, rms 2^-4 / sqrt(3) = 0.036 per
rounding for values spread over a binade) at two places and bf16 at three: each output is a sum of many independent
terms, so the relative error of the whole (2-norms) stays near sqrt(0.036^2 + 0.036^2) = 0.05, and 0.06 is asked.
Training: the gradients against torch's own in 32 bits; bf16 roundings (2^-9) at about ten places in a row:
10 * 2^-9 = 0.02."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    import moe_block
    return moe_block


def rel(a, b):
    return float((a.detach().double() - b.detach().double()).norm() / b.detach().double().norm())


@pytest.mark.parametrize("tokens,experts,k,f,topk", [(1, 16, 512, 256, 4), (64, 16, 512, 256, 4), (300, 8, 1024, 384, 2)])
def test_serving(ex, tokens, experts, k, f, topk):
    import weight_transfer_gb300 as w
    norm_w, router, gate, up, down = ex.random_block(experts, k, f, seed=tokens)
    block = ex.MoeBlock(norm_w, router, gate, up, down, topk)
    x, res = (torch.randn(tokens, k, device="cuda").bfloat16() for _ in range(2))
    out, stream = block.forward(x, res)
    assert torch.equal(stream, (x.float() + res.float()).bfloat16())
    h = x.double() + res.double()
    y = h / torch.sqrt((h * h).mean(1, keepdim=True) + 1e-6) * norm_w.double()
    _, _, _, y16, _ = w.mxfp8_rmsnorm_quantize(x, norm_w, residual=res, want_bf16=True)
    score, ids = torch.topk((y16 @ router.T).float(), topk, dim=1)       # the router's own choice
    p = torch.softmax(score.double(), 1)
    deq = [w.mxfp8_dequantize_swizzled(c, s).double() for c, s in (block.gate, block.up, block.down)]
    want = torch.zeros(tokens, k, dtype=torch.float64, device="cuda")
    for t in range(tokens):
        for j in range(topk):
            e = int(ids[t, j])
            g, u = deq[0][e] @ y[t], deq[1][e] @ y[t]
            want[t] += p[t, j] * (deq[2][e] @ (g * torch.sigmoid(g) * u))
    assert rel(out, want) < 0.06


def test_training(ex):
    tokens, experts, k, f, topk = 96, 6, 256, 128, 2
    norm_w, router, gate, up, down = ex.random_block(experts, k, f, seed=5)
    x, res = (torch.randn(tokens, k, device="cuda").bfloat16() for _ in range(2))
    leaves = [t.clone().requires_grad_() for t in (x, res, norm_w, router)]
    out, stream = ex.train_block(*leaves[:3], leaves[3], gate, up, down, topk)
    dout, ds = torch.randn_like(out), torch.randn_like(out)
    torch.autograd.backward([out, stream], [dout, ds])

    plain = [t.float().requires_grad_() for t in (x, res, norm_w, router)]
    h = plain[0] + plain[1]
    y = h * torch.rsqrt(h.square().mean(1, keepdim=True) + 1e-6) * plain[2]
    with torch.no_grad():                       # the choice is the block's own, so that both differentiate the same thing
        y16 = ex.norm(x, res, norm_w)[0]
        ids = torch.topk((y16 @ router.T).float(), topk, dim=1).indices
    p = torch.softmax(torch.gather(y @ plain[3].T, 1, ids), 1)
    want = 0
    for j in range(topk):
        g = torch.einsum("tk,tfk->tf", y, gate.float()[ids[:, j]])
        u = torch.einsum("tk,tfk->tf", y, up.float()[ids[:, j]])
        want = want + p[:, j, None] * torch.einsum("tf,tkf->tk", torch.nn.functional.silu(g) * u, down.float()[ids[:, j]])
    torch.autograd.backward([want, h], [dout.float(), ds.float()])
    assert rel(out, want.detach()) < 0.02
    for a, b in zip(leaves, plain):
        assert rel(a.grad, b.grad) < 0.02


def test_example_runs(ex):
    ex.main()
