"""The expert-block operators together, through examples/moe_block.py.

Serving: the block is the composition of its calls, bit for bit, and each stage is checked in 64 bits against the codes
that the stage before it left, so that no bound has to allow for a rounding to 8 bits: gate/up codes are roundings of
h64 within the products' accumulation error (k/32 + 1 steps of 2^-22 of the sum of magnitudes, on g and on u, carried
through silu(g) * u with |silu'| <= 1.1) plus 2^-19 relative; the output is within half a bf16 step (2^-8) of each
expert row and of itself.
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
    codes, scales, stream2, y16, _ = w.mxfp8_rmsnorm_quantize(x, norm_w, residual=res, want_bf16=True)
    score, ids = torch.topk((y16 @ router.T).float(), topk, dim=1)       # the router's own choice
    p = torch.softmax(score, 1)
    off, order, slots = w.fp8q_moe_sort(ids, experts)
    rows, row_scales = w.mxfp8_moe_gather(codes, scales, slots, off)
    h, hs = w.mxfp8_moe_swiglu(rows, row_scales, *block.gate, *block.up, off)
    y = w.mxfp8_moe_matmul(h, hs, *block.down, off)
    assert torch.equal(stream, stream2) and torch.equal(out, w.fp8q_moe_combine(y, slots, off, p))

    value = lambda c, e: c.view(torch.float8_e4m3fn).double() * (2.0 ** (e.double() - 127)).repeat_interleave(32, 1)  # noqa: E731
    src = order.long() // topk
    assert torch.equal(rows, codes[src]) and torch.equal(row_scales, scales[src])
    e_of = ids.reshape(-1)[order.long()]
    gate64, up64, down64 = (w.mxfp8_dequantize_swizzled(c, s).double() for c, s in (block.gate, block.up, block.down))
    a, hv = value(rows, row_scales), value(h, hs)
    h64, slack, y64, y_slack = (torch.zeros(len(src), n, dtype=torch.float64, device="cuda") for n in (f, f, k, k))
    for e in range(experts):
        m = e_of == e
        g, u = a[m] @ gate64[e].T, a[m] @ up64[e].T
        eps = (k / 32 + 1) * 2.0 ** -22
        dg, du = eps * (a[m].abs() @ gate64[e].abs().T), eps * (a[m].abs() @ up64[e].abs().T)
        h64[m] = g * torch.sigmoid(g) * u
        slack[m] = 1.1 * dg * (u.abs() + du) + (g.abs() + dg) * du + 2.0 ** -19 * h64[m].abs()
        y64[m] = hv[m] @ down64[e].T
        y_slack[m] = (f / 32 + 1) * 2.0 ** -22 * (hv[m].abs() @ down64[e].abs().T)
    step = 2.0 ** (hs.double() - 127).repeat_interleave(32, 1)           # value of code 1: codes are steps of 2^-3 of their
    half = torch.maximum(hv.abs() * 2.0 ** -3, step * 2.0 ** -8) / 2      # power of two, at least 2^-9; half of one either way
    assert ((hv - h64).abs() <= half + slack + (h64.abs() - 448 * step).clamp(min=0)).all()
    assert ((y.double() - y64).abs() <= 2.0 ** -8 * y64.abs() + 2 * y_slack).all()
    terms = y.double()[slots.long()] * p.double()[..., None]
    assert ((out.double() - terms.sum(1)).abs() <= 2.0 ** -8 * terms.sum(1).abs() + topk * 2.0 ** -24 * terms.abs().sum(1)).all()


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
