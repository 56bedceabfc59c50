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
