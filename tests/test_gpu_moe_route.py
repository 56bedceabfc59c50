"""Sort by expert, gather, combine and their gradients against plain 64-bit
implementations.  Sorts and copies are exact.  A combined value is a sum of
topk products, each fused into a binary32 accumulator: at most topk roundings
of partial sums no larger than sum |w y|, so topk * 2^-24 of that sum before
the bf16 rounding.  A dot product over k columns runs in 32 lanes of k/32
additions and 5 joins: (k/32 + 5) * 2^-24 of sum |d y|, one more for slack."""
import numpy as np
import pytest
import torch

from expert_block_ref import check_bf16, sort_ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    import weight_transfer_gb300 as m
    return m


def ids_of(tokens, topk, experts, seed, how):
    rng = np.random.default_rng(seed)
    if how == "one":                                    # every choice names the same expert
        ids = np.full((tokens, topk), experts - 1)
    elif how == "none":                                 # no choice names an expert
        ids = rng.choice([-1, -7, experts, experts + 5], (tokens, topk))
    else:
        ids = (rng.random((tokens, topk)) ** 2 * experts).astype(np.int64)
        if how == "drop":
            ids[rng.random(ids.shape) < 0.3] = -1
            ids[tokens // 2] = experts                  # a token that no expert takes
    return torch.from_numpy(ids.astype(np.int64))


SORTS = [(1, 1, 1), (1, 8, 128), (3, 2, 5), (31, 1, 4), (33, 3, 7), (257, 8, 60), (300, 7, 1024), (1024, 8, 128),
         (2049, 1, 384), (5000, 6, 129), (20011, 8, 256)]


@pytest.mark.parametrize("tokens,topk,experts", SORTS)
@pytest.mark.parametrize("how", ["any", "drop", "one", "none"])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_sort(w, tokens, topk, experts, how, dtype):
    ids = ids_of(tokens, topk, experts, tokens + experts, how)
    got = w.fp8q_moe_sort(ids.to(dtype).cuda(), experts)
    for g, e in zip(got, sort_ref(ids, experts)):
        assert np.array_equal(g.cpu().numpy(), e)


def test_sort_wide_ids(w):
    """64-bit ids whose low 32 bits name an expert are out of range all the same."""
    ids = torch.tensor([[3, (1 << 32) + 3], [-(1 << 40) + 1, 1]])
    got = w.fp8q_moe_sort(ids.cuda(), 4)
    for g, e in zip(got, sort_ref(ids, 4)):
        assert np.array_equal(g.cpu().numpy(), e)


def test_sort_of_nothing(w):
    off, order, slots = w.fp8q_moe_sort(torch.empty(0, 4, dtype=torch.int32, device="cuda"), 9,
                                        offsets=torch.full((10,), 5, dtype=torch.int32, device="cuda"))
    assert not off.any() and order.numel() == 0 and slots.shape == (0, 4)


CASES = [(1, 1, 1, 8, "any"), (1, 8, 128, 2048, "any"), (13, 3, 5, 264, "drop"), (5, 32, 40, 1032, "drop"),
         (64, 2, 9, 4096, "none"), (211, 6, 60, 1408, "drop"), (7, 5, 3, 8200, "any"), (1000, 8, 128, 512, "drop")]


def routed(w, tokens, topk, experts, how):
    ids = ids_of(tokens, topk, experts, tokens, how)
    off, order, slots = w.fp8q_moe_sort(ids.cuda(), experts)
    return ids, off, order, slots, int(off[-1])


# short rows, few choices: a warp has several tokens, the last one fewer
SHORT = [(5, 1, 3, 256, "any"), (203, 1, 7, 64, "drop"), (77, 2, 9, 128, "drop"), (131, 2, 5, 480, "any"), (33, 2, 6, 512, "drop"),
         (67, 1, 4, 672, "drop"), (45, 4, 8, 96, "drop")]


@pytest.mark.parametrize("tokens,topk,experts,k,how", CASES + SHORT)
def test_gather(w, tokens, topk, experts, k, how):
    ids, off, order, slots, n = routed(w, tokens, topk, experts, how)
    x = torch.randn(tokens, k, device="cuda").bfloat16()
    src = order.long() // topk
    want = x[src].clone()
    want[n:] = 0
    got = w.fp8q_moe_gather(x, slots, off, rows=torch.full((tokens * topk, k), float("nan"), dtype=torch.bfloat16, device="cuda"))
    assert torch.equal(got, want)


@pytest.mark.parametrize("tokens,topk,experts,k,how", [(c[0], c[1], c[2], -(-c[3] // 32) * 32, c[4]) for c in CASES + SHORT])
def test_gather_mxfp8(w, tokens, topk, experts, k, how):
    ids, off, order, slots, n = routed(w, tokens, topk, experts, how)
    codes = torch.randint(0, 256, (tokens, k), dtype=torch.uint8, device="cuda")
    scales = torch.randint(0, 256, (tokens, k // 32), dtype=torch.uint8, device="cuda")
    src = order.long() // topk
    fill = lambda c: torch.full((tokens * topk, c), 0xA5, dtype=torch.uint8, device="cuda")  # noqa: E731
    gc, gs = w.mxfp8_moe_gather(codes, scales, slots, off, fill(k), fill(k // 32))
    for g, s in ((gc, codes), (gs, scales)):
        want = s[src].clone()
        want[n:] = 0
        assert torch.equal(g, want)


# few choices: a warp sums several 256-column pieces of a row, the last of them partly or wholly outside
FEW = [(37, 1, 9, 4104, "drop"), (3, 1, 2, 1800, "any"), (50, 1, 4, 256, "drop"), (41, 2, 7, 2056, "drop"),
       (19, 2, 3, 768, "any"), (29, 4, 11, 1032, "drop"), (23, 3, 5, 264, "any")]


@pytest.mark.parametrize("tokens,topk,experts,k,how", CASES + FEW + SHORT)
@pytest.mark.parametrize("weighted", [False, True])
def test_combine(w, tokens, topk, experts, k, how, weighted):
    ids, off, order, slots, n = routed(w, tokens, topk, experts, how)
    y = torch.randn(tokens * topk, k, device="cuda").bfloat16()
    y[n:] = float("nan")                                # rows of dropped choices are never looked at
    wt = torch.randn(tokens, topk, device="cuda") if weighted else None
    got = w.fp8q_moe_combine(y, slots, off, wt)
    sl = slots.cpu().long()
    live = (sl < n)[..., None]
    w64 = torch.ones(tokens, topk, dtype=torch.float64) if wt is None else wt.double().cpu()
    terms = torch.where(live, y.double().cpu()[sl] * w64[..., None], 0.0)
    check_bf16(got, terms.sum(1), topk * 2.0 ** -24, terms.abs().sum(1))


@pytest.mark.parametrize("tokens,topk,experts,k,how", CASES)
def test_combine_gradient(w, tokens, topk, experts, k, how):
    ids, off, order, slots, n = routed(w, tokens, topk, experts, how)
    y = torch.randn(tokens * topk, k, device="cuda").bfloat16()
    y[n:] = float("nan")
    dout = torch.randn(tokens, k, device="cuda").bfloat16()
    wt = torch.randn(tokens, topk, device="cuda")
    dy, dw = w.fp8q_moe_combine_backward(dout, y, slots, off, wt,
                                         dy=torch.full((tokens * topk, k), float("nan"), dtype=torch.bfloat16, device="cuda"))
    sl = slots.cpu().long()
    live = sl < n
    d64 = dout.double().cpu()
    want = torch.zeros(tokens * topk, k, dtype=torch.float64)
    want[sl.reshape(-1)] = torch.where(live[..., None], d64[:, None] * wt.double().cpu()[..., None], 0.0).reshape(-1, k)
    check_bf16(dy, want, 2.0 ** -24)
    terms = torch.where(live[..., None], d64[:, None] * y.double().cpu()[sl], 0.0)
    err = (dw.double().cpu() - terms.sum(-1)).abs()
    assert (err <= (k / 32 + 6) * 2.0 ** -24 * terms.abs().sum(-1)).all()


def test_gradients_are_the_derivatives(w):
    """<dout, combine(y)> moves by dy and dweights, <drows, gather(x)> by the combine of drows: the operators are
    linear, so the differences are exact up to the outputs' rounding."""
    tokens, topk, experts, k = 9, 3, 4, 64
    ids, off, order, slots, n = routed(w, tokens, topk, experts, "drop")
    y = torch.randn(tokens * topk, k, device="cuda").bfloat16()
    wt, dout = torch.rand(tokens, topk, device="cuda"), torch.randn(tokens, k, device="cuda").bfloat16()
    dy, dw = w.fp8q_moe_combine_backward(dout, y, slots, off, wt)
    for _ in range(3):
        vy, vw = torch.randn_like(y), torch.randn_like(wt)
        sl, live = slots.long(), (slots < n)[..., None]
        out = lambda yy, ww: (torch.where(live, yy.double()[sl], 0.0) * ww.double()[..., None]).sum(1)  # noqa: E731
        lhs = float((dout.double() * (out(vy, wt) + out(y, vw))).sum())
        rhs = float((dy.double() * vy.double()).sum() + (dw.double() * vw.double()).sum())
        # dy is rounded to bf16 (2^-9 of each term); terms of size ~1, tokens * topk * k of them with random signs
        bound = 2.0 ** -9 * float((dy.double() * vy.double()).abs().sum()) + 1e-4
        assert abs(lhs - rhs) <= bound
    x, drows = torch.randn(tokens, k, device="cuda").bfloat16(), torch.randn(tokens * topk, k, device="cuda").bfloat16()
    dx = w.fp8q_moe_combine(drows, slots, off)
    lhs = float((drows.double() * w.fp8q_moe_gather(x, slots, off).double()).sum())
    bound = 2.0 ** -8 * float((dx.double() * x.double()).abs().sum()) + 1e-4
    assert abs(lhs - float((dx.double() * x.double()).sum())) <= bound


def test_slots_out_of_range_are_skipped(w):
    """Slots that no sort wrote are neither read nor written through."""
    slots = torch.tensor([[0, 4], [-1, 2]], dtype=torch.int32, device="cuda")       # 4 rows: 4 and -1 are outside
    off = torch.tensor([0, 2, 4], dtype=torch.int32, device="cuda")
    x = torch.randn(2, 64, device="cuda").bfloat16()
    buf = torch.full((8, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    rows = w.fp8q_moe_gather(x, slots, off, rows=buf[2:6])
    assert torch.equal(rows[0], x[0]) and torch.equal(rows[2], x[1])
    assert (buf[[0, 1, 3, 5, 6, 7]] == 5).all()
    y = torch.randn(4, 64, device="cuda").bfloat16()
    assert torch.equal(w.fp8q_moe_combine(y, slots, off), y[[0, 2]])


def test_long_rows_pass_32_bits(w):
    """tokens * topk * k beyond 2^31 elements: the last rows land in place."""
    tokens, topk, k = 66000, 8, 4096
    if torch.cuda.mem_get_info()[0] < 16 << 30:
        pytest.skip("needs 16 GB of free device memory")
    ids = torch.arange(topk, device="cuda", dtype=torch.int32).repeat(tokens, 1)
    off, order, slots = w.fp8q_moe_sort(ids, topk)
    x = (torch.arange(tokens, device="cuda")[:, None] % 251 + torch.arange(k, device="cuda")[None] % 3).bfloat16()
    rows = w.fp8q_moe_gather(x, slots, off)
    assert torch.equal(rows[-tokens:], x) and torch.equal(rows[:tokens], x)
    out = w.fp8q_moe_combine(rows, slots, off, torch.full((tokens, topk), 1 / topk, device="cuda"))
    assert torch.equal(out, x)                # eighths of the same row add up exactly


def test_other_stream(w):
    ids, off, order, slots, n = routed(w, 211, 6, 60, "drop")
    y = torch.randn(211 * 6, 512, device="cuda").bfloat16()
    want = w.fp8q_moe_combine(y, slots, off)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        off2, _, slots2 = w.fp8q_moe_sort(ids.cuda(), 60)
        got = w.fp8q_moe_combine(y, slots2, off2)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(slots, slots2)


def test_stream_argument(w):
    """A stream passed to the calls, with outputs and workspaces made by them: nothing is reused while in use there."""
    tokens, topk, experts = 20011, 8, 256
    ids = ids_of(tokens, topk, experts, 1, "drop").cuda()
    want = sort_ref(ids, experts)
    x = torch.randn(1500, 1408, device="cuda").bfloat16()
    rstd, wt = torch.rsqrt(x.float().square().mean(1)), torch.ones(1408, device="cuda").bfloat16()
    ref = w.fp8q_rmsnorm_backward(x, x, wt, rstd)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for handle in (s, s.cuda_stream):
        got, grads = [], []
        for _ in range(4):
            with torch.cuda.stream(s):
                torch.cuda._sleep(1_000_000)
            got.append(w.fp8q_moe_sort(ids, experts, stream=handle))
            grads.append(w.fp8q_rmsnorm_backward(x, x, wt, rstd, stream=handle))
            for _ in range(8):                          # would take a workspace that is free too early
                torch.full((tokens * 32,), -1, dtype=torch.int32, device="cuda")
        s.synchronize()
        for g in got:
            for a, b in zip(g, want):
                assert np.array_equal(a.cpu().numpy(), b)
        for g in grads:
            assert torch.equal(g[0], ref[0]) and torch.equal(g[1], ref[1])
