"""A mixture-of-experts block on MXFP8 expert weights, as it serves and as it trains.

Serving (``MoeBlock.forward``): the residual stream is normalized and quantized in one pass, the router picks experts
from the bf16 rows, the MXFP8 rows travel to their experts, the gate/up and down products read the weights exactly as
mxfp8_quantize_swizzled wrote them (what a refit ships), and the experts' rows are summed back with the router's weights.
A few tokens (``MoeBlock.decode``) go through their experts in one call, without sorting or carrying rows.

Training (``norm``, ``gather`` and ``combine`` below): the same norm and routing with gradients, around whatever the
experts compute in bf16.

    python examples/moe_block.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import weight_transfer_gb300 as fp8q  # noqa: E402


class MoeBlock:
    """Weights of one block: norm [k], router [experts, k], gate and up [experts, f, k], down [experts, k, f], all bf16."""

    def __init__(self, norm, router, gate, up, down, topk: int, eps: float = 1e-6):
        self.norm, self.router, self.topk, self.eps = norm, router, topk, eps
        self.experts = router.shape[0]
        self.gate, self.up, self.down = (fp8q.mxfp8_quantize_swizzled(w) for w in (gate, up, down))

    def forward(self, x: torch.Tensor, residual: torch.Tensor):
        """x, residual bf16 [tokens, k] -> (the block's output, the new residual stream), both bf16."""
        codes, scales, stream, y, _ = fp8q.mxfp8_rmsnorm_quantize(x, self.norm, self.eps, residual=residual, want_bf16=True)
        score, ids = torch.topk((y @ self.router.T).float(), self.topk, dim=1)
        weights = torch.softmax(score, 1)
        offsets, _, slots = fp8q.fp8q_moe_sort(ids, self.experts)
        rows, row_scales = fp8q.mxfp8_moe_gather(codes, scales, slots, offsets)
        h, h_scales = fp8q.mxfp8_moe_swiglu(rows, row_scales, *self.gate, *self.up, offsets)
        out = fp8q.mxfp8_moe_matmul(h, h_scales, *self.down, offsets)
        return fp8q.fp8q_moe_combine(out, slots, offsets, weights), stream


    def decode(self, x: torch.Tensor, residual: torch.Tensor):
        """forward() for a few tokens (at most FP8Q_MOE_DECODE_MAX_TOKENS): the experts in one call."""
        codes, scales, stream, y, _ = fp8q.mxfp8_rmsnorm_quantize(x, self.norm, self.eps, residual=residual, want_bf16=True)
        score, ids = torch.topk((y @ self.router.T).float(), self.topk, dim=1)
        return fp8q.mxfp8_moe_decode(codes, scales, ids, torch.softmax(score, 1), *self.gate, *self.up, *self.down), stream


class _Norm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, eps):
        codes, scales, stream, y, rstd = fp8q.fp8q_rmsnorm_quantize(x, weight, eps, residual=residual, want_bf16=True,
                                                                    want_rstd=True)
        ctx.save_for_backward(stream, weight, rstd)
        ctx.mark_non_differentiable(codes, scales)
        return y, stream, codes, scales

    @staticmethod
    def backward(ctx, dy, dstream, _codes, _scales):
        stream, weight, rstd = ctx.saved_tensors
        dx, dw = fp8q.fp8q_rmsnorm_backward(dy.contiguous(), stream, weight, rstd,
                                            dsum=None if dstream is None else dstream.contiguous())
        return dx, dx, dw.to(weight.dtype), None


class _Gather(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, slots, offsets):
        ctx.save_for_backward(slots, offsets)
        return fp8q.fp8q_moe_gather(x, slots, offsets)

    @staticmethod
    def backward(ctx, drows):
        slots, offsets = ctx.saved_tensors
        return fp8q.fp8q_moe_combine(drows.contiguous(), slots, offsets), None, None


class _Combine(torch.autograd.Function):
    @staticmethod
    def forward(ctx, y, weights, slots, offsets):
        ctx.save_for_backward(y, weights, slots, offsets)
        return fp8q.fp8q_moe_combine(y, slots, offsets, weights)

    @staticmethod
    def backward(ctx, dout):
        y, weights, slots, offsets = ctx.saved_tensors
        dy, dw = fp8q.fp8q_moe_combine_backward(dout.contiguous(), y, slots, offsets, weights)
        return dy, dw, None, None


def norm(x, residual, weight, eps=1e-6):
    """-> (y bf16, residual stream bf16, y's e4m3 codes, their scales); differentiable in x, residual and weight."""
    return _Norm.apply(x, residual, weight, eps)


def gather(x, slots, offsets):
    """Rows of x by expert; differentiable in x."""
    return _Gather.apply(x, slots, offsets)


def combine(y, weights, slots, offsets):
    """The experts' rows summed back; differentiable in y and weights."""
    return _Combine.apply(y, weights, slots, offsets)


def train_block(x, residual, norm_weight, router, gate, up, down, topk):
    """The block in bf16 with gradients; the experts' products are torch's, one expert after the other."""
    y, stream, _, _ = norm(x, residual, norm_weight)
    score, ids = torch.topk((y @ router.T).float(), topk, dim=1)
    weights = torch.softmax(score, 1)
    offsets, _, slots = fp8q.fp8q_moe_sort(ids, router.shape[0])
    rows = gather(y, slots, offsets)
    outs, cuts = [], offsets.tolist()
    for e in range(router.shape[0]):
        r = rows[cuts[e]:cuts[e + 1]]
        outs.append((torch.nn.functional.silu(r @ gate[e].T) * (r @ up[e].T)) @ down[e].T)
    return combine(torch.cat(outs), weights, slots, offsets), stream


def random_block(experts, k, f, seed=0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    r = lambda *s, scale: (torch.randn(*s, generator=g, device=device) * scale).bfloat16()  # noqa: E731
    return ((1 + r(k, scale=0.1)), r(experts, k, scale=k ** -0.5), r(experts, f, k, scale=k ** -0.5),
            r(experts, f, k, scale=k ** -0.5), r(experts, k, f, scale=f ** -0.5))


def main():
    experts, k, f, topk, tokens = 128, 2048, 768, 8, 512
    norm_w, router, gate, up, down = random_block(experts, k, f)
    block = MoeBlock(norm_w, router, gate, up, down, topk)
    x, residual = (torch.randn(tokens, k, device="cuda").bfloat16() for _ in range(2))
    out, stream = block.forward(x, residual)
    with torch.no_grad():
        ref, ref_stream = train_block(x, residual, norm_w, router, gate, up, down, topk)
    err = (out.float() - ref.float()).norm() / ref.float().norm()
    print(f"{tokens} tokens, {experts} experts, top {topk}: MXFP8 block against bf16 experts: relative difference {err:.4f}")
    assert torch.equal(stream, ref_stream) and err < 0.1
    few, few_stream = block.decode(x[:8], residual[:8])
    err = (few.float() - out[:8].float()).norm() / out[:8].float().norm()
    print(f"8 tokens in one call against the same through the sorted path: relative difference {err:.4f}")
    assert torch.equal(few_stream, stream[:8]) and err < 0.05
    leaves = [t.clone().requires_grad_() for t in (x, residual, norm_w)]
    y, _ = train_block(*leaves, router, gate, up, down, topk)
    y.float().square().mean().backward()
    print("gradient norms:", ", ".join(f"{t.grad.float().norm():.3e}" for t in leaves))


if __name__ == "__main__":
    main()
