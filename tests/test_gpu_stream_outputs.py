"""Outputs and workspaces that the calls make when a stream is passed, against
work that is still queued on the current stream.

The current stream sleeps, then writes over a tensor that has been dropped by
then: its block goes back to the allocator at once and may be handed to the next
tensor of its size, which a call on another stream would write too early.  In
the other direction, an output that is dropped while a copy of it waits on the
current stream must keep its memory until that copy has run."""
import pytest
import torch

pytestmark = pytest.mark.gpu

SLEEP = 40_000_000          # cycles: about 20 ms


@pytest.fixture(scope="module")
def w():
    import weight_transfer_gb300 as m
    return m


def expert_calls(w):
    """name -> call with a stream, over inputs that are ready"""
    g = torch.Generator().manual_seed(4)
    rows, k, tokens, topk, experts = 4096, 1024, 4096, 4, 16
    x = torch.randn(rows, k, generator=g).bfloat16().cuda()
    wt = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    rstd = torch.rsqrt(x.float().square().mean(1))
    ids = torch.randint(0, experts, (tokens, topk), generator=g).cuda()
    off, _, slots = w.fp8q_moe_sort(ids, experts)
    codes, scales, *_ = w.mxfp8_rmsnorm_quantize(x, wt)
    y = torch.randn(tokens * topk, k, generator=g).bfloat16().cuda()
    p = torch.rand(tokens, topk, generator=g).cuda()
    wc, ws = w.mxfp8_quantize_swizzled(torch.randn(experts, 256, k, generator=g).bfloat16().cuda())
    rc, rs = w.mxfp8_moe_gather(codes, scales, slots, off)
    return {
        "norm": lambda **s: w.mxfp8_rmsnorm_quantize(x, wt, residual=x, want_bf16=True, want_rstd=True, **s),
        "norm_blockwise": lambda **s: w.fp8q_rmsnorm_quantize(x, wt, **s)[:2],
        "norm_gradient": lambda **s: w.fp8q_rmsnorm_backward(x, x, wt, rstd, **s),
        "sort": lambda **s: w.fp8q_moe_sort(ids, experts, **s),
        "gather": lambda **s: (w.fp8q_moe_gather(x, slots, off, **s),),
        "gather_mxfp8": lambda **s: w.mxfp8_moe_gather(codes, scales, slots, off, **s),
        "combine": lambda **s: (w.fp8q_moe_combine(y, slots, off, p, **s),),
        "combine_gradient": lambda **s: w.fp8q_moe_combine_backward(x, y, slots, off, p, **s),
        "matmul": lambda **s: (w.mxfp8_moe_matmul(rc, rs, wc, ws, off, **s),),
        "swiglu": lambda **s: w.mxfp8_moe_swiglu(rc, rs, wc, ws, wc, ws, off, **s),
    }


EXPERT = ["norm", "norm_blockwise", "norm_gradient", "sort", "gather", "gather_mxfp8", "combine", "combine_gradient",
          "matmul", "swiglu"]


def check(call):
    want = [t.clone() for t in call()]
    sizes = [t.numel() * t.element_size() for t in want] + [1 << 16, 1 << 20, 1 << 22]
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        # nothing that the current stream still writes is handed out
        torch.cuda.synchronize()
        torch.cuda._sleep(SLEEP)
        for n in sizes:
            torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xA5)
        got = call(stream=handle)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        # nothing that the current stream still reads is taken back
        del got
        got = call(stream=handle)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(SLEEP)
        kept = [t.clone() for t in got]
        del got
        with torch.cuda.stream(s):
            spoil = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes]
        torch.cuda.synchronize()
        for a, b in zip(kept, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        del spoil


@pytest.mark.parametrize("name", EXPERT)
def test_expert_block(w, name):
    check(expert_calls(w)[name])


def codec_calls(w):
    g = torch.Generator().manual_seed(6)
    n = 1 << 21
    xs = [torch.randn(n, generator=g).bfloat16().cuda() for _ in range(2)]
    q = [w.fp8q_quantize_blockwise(x) for x in xs]
    codes, scales = [c for c, _ in q], [s for _, s in q]
    hop = lambda: {"in_codes": codes[0], "in_scales": scales[0], "local": xs[1], "want_bf16": True}  # noqa: E731
    wt = xs[0].view(4, 512, 1024)
    wc, ws = w.mxfp8_quantize_swizzled(wt)
    f32 = xs[0].float()
    return {
        "quantize": lambda **s: w.fp8q_quantize_blockwise(xs[0], **s),
        "quantize_group": lambda **s: sum(w.fp8q_quantize_blockwise_group(xs, **s), []),
        "quantize_tensorwise": lambda **s: w.fp8q_quantize_tensorwise(xs[0], **s),
        "encode": lambda **s: (w.fp8q_encode_f32(f32, **s),),
        "dequantize": lambda **s: w.fp8q_dequantize(codes[0], scales[0], want_bf16=True, **s),
        "dequant_reduce": lambda **s: w.fp8q_dequant_reduce(codes, scales, **s),
        "dequant_reduce_unfused": lambda **s: w.fp8q_dequant_reduce_unfused(codes, scales, **s),
        "dequant_reduce_unfused_static": lambda **s: w.fp8q_dequant_reduce_unfused_static(
            [c[:1 << 20] for c in codes], [t[:1 << 13] for t in scales], **s),
        "ring_hop": lambda **s: w.fp8q_ring_hop(codes[0], scales[0], xs[1], want_bf16=True, **s),
        "ring_hop_group": lambda **s: w.fp8q_ring_hop_group([hop()], **s)[0],
        "ring_hop_bf16_requant": lambda **s: w.fp8q_ring_hop_bf16_requant(codes[0], scales[0], xs[1], want_bf16=True, **s),
        "gather_decode": lambda **s: w.fp8q_gather_decode(codes[0], scales[0], 2, **s),
        "ring_allreduce": lambda **s: w.fp8q_ring_allreduce_sim(xs, **s)[0],
        "mx_quantize": lambda **s: w.mxfp8_quantize_swizzled(wt, **s),
        "mx_quantize_group": lambda **s: sum(w.mxfp8_quantize_swizzled_group([wt, wt], **s), []),
        "mx_dequantize": lambda **s: (w.mxfp8_dequantize_swizzled(wc, ws, **s),),
        "mx_unswizzle": lambda **s: (w.mxfp8_unswizzle_scales(ws, 4, 512, 1024, **s),),
        "mismatches": lambda **s: (w.fp8q_count_mismatches(xs[0], xs[1], **s),),
    }


CODEC = ["quantize", "quantize_group", "quantize_tensorwise", "encode", "dequantize", "dequant_reduce", "dequant_reduce_unfused",
         "dequant_reduce_unfused_static", "ring_hop", "ring_hop_group", "ring_hop_bf16_requant", "gather_decode",
         "ring_allreduce", "mx_quantize", "mx_quantize_group", "mx_dequantize", "mx_unswizzle", "mismatches"]


@pytest.mark.parametrize("name", CODEC)
def test_codec(w, name):
    check(codec_calls(w)[name])
