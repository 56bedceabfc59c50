"""The expert layer for a few tokens against the formula in 64 bits.

Tolerances.  A product's sum over K runs in blocks of 32 products, each summed
exactly or with a rounding of 2^-23 per product, and the K / 32 blocks one after
the other or in any tree: (K / 32 + 72) * 2^-24 of the sum of absolute values.
The activation carries 2^-20 relative and the derivative's share of g's error;
h is held as two f16 terms, each of which leaves 2^-11 of what it rounds: 2^-22
of a value, and of the largest in its block of 32 half of 2^-24 / 2^14 = 2^-39,
where a value is small enough to be subnormal.  The outer sums add
(topk + N / 32 + 72) * 2^-24, the output its rounding."""
import pytest
import torch

import weight_transfer_gb300 as w
from gpu_util import Guarded

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


def values(codes, scales):
    return codes.view(torch.float8_e4m3fn).double() * torch.pow(2.0, scales.double() - 127).repeat_interleave(32, -1)


def weights(g, experts, n, k, size, far=False):
    m = torch.randn(experts, n, k, generator=g, device="cuda") * size
    if far:                                   # blocks of very different magnitude, and some of zeros
        m *= torch.exp2(torch.randint(-30, 30, (experts, n, k // 32, 1), generator=g, device="cuda").float()).expand(
            -1, -1, -1, 32).reshape(experts, n, k)
        m[:, ::5, :32] = 0
    codes, scales = w.mxfp8_quantize_swizzled(m.bfloat16())
    flat = w.mxfp8_unswizzle_scales(scales, experts, n, k)
    return codes, scales, values(codes, flat.view(experts, n, k // 32))


def layer(tokens, topk, experts, n, k, seed, far=False, id_dtype=torch.int64):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, k, generator=g, device="cuda")
    if far:
        x *= torch.exp2(torch.randint(-20, 20, (tokens, k // 32, 1), generator=g, device="cuda").float()).expand(
            -1, -1, 32).reshape(tokens, k)
    xc, xs = w.mxfp8_quantize_swizzled(x.bfloat16())
    xs = w.mxfp8_unswizzle_scales(xs, 1, tokens, k).view(tokens, k // 32)
    ids = torch.randint(0, experts, (tokens, topk), generator=g, device="cuda").to(id_dtype)
    p = torch.softmax(torch.randn(tokens, topk, generator=g, device="cuda"), 1)
    gate, up = weights(g, experts, n, k, k ** -0.5, far), weights(g, experts, n, k, k ** -0.5, far)
    return dict(xc=xc, xs=xs, ids=ids, p=p, gate=gate, up=up, down=weights(g, experts, k, n, n ** -0.5))


def formula(s):
    """-> (out, tolerance) in 64 bits."""
    x = values(s["xc"], s["xs"])
    tokens, k = x.shape
    experts, n = s["gate"][2].shape[:2]
    out, tol = torch.zeros_like(x), torch.zeros_like(x)
    c1, c2 = (k / 32 + 72) * U, (s["ids"].shape[1] + n / 32 + 72) * U
    for t in range(tokens):
        for j in range(s["ids"].shape[1]):
            e = int(s["ids"][t, j])
            if not 0 <= e < experts:
                continue
            G, V, D = s["gate"][2][e], s["up"][2][e], s["down"][2][e]
            g, u = G @ x[t], V @ x[t]
            eg, eu = c1 * (G.abs() @ x[t].abs()), c1 * (V.abs() @ x[t].abs())
            sig = torch.sigmoid(g)
            h = g * sig * u
            # |silu'| <= 1.1 everywhere; g enters exp(-g) with |g| 2^-24
            eh = 1.1 * eg * (u.abs() + eu) + (g * sig).abs() * eu + h.abs() * (2.0 ** -20 + 4 * U * g.abs().clamp(max=100))
            eh = eh + h.abs() * 2.0 ** -22 + h.abs().view(-1, 32).amax(1).repeat_interleave(32) * 2.0 ** -39
            p = float(s["p"][t, j])
            out[t] += p * (D @ h)
            tol[t] += abs(p) * (D.abs() @ (eh + c2 * h.abs()))
    return out, tol + out.abs() * 2.0 ** -8 + 2.0 ** -134


def call(s, **kw):
    return w.mxfp8_moe_decode(s["xc"], s["xs"], s["ids"], s["p"], *s["gate"][:2], *s["up"][:2], *s["down"][:2], **kw)


def check(s):
    tokens, k = s["xc"].shape
    buf = Guarded(tokens * k, torch.bfloat16)
    got = call(s, out=buf.t).view(tokens, k)
    torch.cuda.synchronize()
    assert buf.intact()
    want, tol = formula(s)
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), got[bad][:4], want[bad][:4], tol[bad][:4])
    return got


@pytest.mark.parametrize("n,k", [(32, 32), (32, 64), (64, 32), (96, 160), (160, 96), (128, 128), (256, 512), (224, 1056), (1056, 224),
                                 (768, 2048), (1760, 736)])
def test_shapes(n, k):
    for tokens, topk, experts in ((1, 1, 1), (1, 2, 3), (3, 2, 5)):
        check(layer(tokens, topk, experts, n, k, seed=n + k + tokens))


@pytest.mark.parametrize("n,k", [(32, 16384), (16384, 32), (2560, 8192)])
def test_long_rows(n, k):
    for tokens in (1, 32):
        check(layer(tokens, 2, 3, n, k, seed=n))


@pytest.mark.parametrize("tokens", [1, 2, 3, 4, 5, 7, 8, 9, 15, 16, 17, 31, 32])
@pytest.mark.parametrize("topk,experts", [(1, 1), (2, 4), (6, 60)])
def test_tokens(tokens, topk, experts):
    """Experts with up to 64 rows (all tokens' choices on one expert), and with one or none."""
    check(layer(tokens, topk, experts, 96, 256, seed=tokens))


@pytest.mark.parametrize("topk,experts", [(8, 128), (32, 40), (32, 1), (1, 1024), (8, 1024), (32, 1024)])
def test_choices(topk, experts):
    for tokens in (1, 3, 32):
        check(layer(tokens, topk, experts, 32, 64, seed=topk + experts))


def test_the_same_expert_twice():
    s = layer(4, 4, 6, 64, 128, seed=1)
    s["ids"][0] = 2
    s["ids"][1, 1:3] = 5
    check(s)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_dropped_choices(dtype):
    s = layer(6, 3, 4, 96, 160, seed=2, id_dtype=dtype)
    s["ids"][0] = -1
    s["ids"][1, 0] = 4
    s["ids"][2, 2] = -100
    s["ids"][3, 1] = 2 ** 31 - 1 if dtype == torch.int32 else 2 ** 40
    s["p"][0] = float("nan")                        # weights of dropped choices are not looked at
    got = check_dropped(s)
    assert not got[0].any()
    s["ids"].fill_(-1)
    assert not call(s).any()


def check_dropped(s):
    live = (s["ids"] >= 0) & (s["ids"] < s["gate"][0].shape[0])
    clean = dict(s, p=torch.where(live, s["p"], 0.0))
    want, tol = formula(clean)
    got = call(s)
    assert ((got.double() - want).abs() <= tol).all()
    return got


def test_blocks_of_very_different_magnitude():
    check(layer(5, 2, 4, 96, 320, seed=3, far=True))


def test_weights_of_any_sign_and_size():
    s = layer(5, 3, 4, 64, 96, seed=4)
    s["p"] = torch.tensor([0.0, -1.0, 1e3, 1e-6, 2.0], device="cuda")[:, None] * torch.ones(1, 3, device="cuda")
    check(s)


def test_large_gates():
    """exp(-g) overflows on one side and vanishes on the other."""
    s = layer(3, 2, 3, 64, 96, seed=5)
    s["xs"] += 7
    check(s)


def test_no_tokens():
    s = layer(2, 2, 3, 64, 96, seed=6)
    for name in ("xc", "xs", "ids", "p"):
        s[name] = s[name][:0]
    assert call(s).shape == (0, 96)


def test_nan_stays_with_its_token():
    s = layer(4, 2, 5, 64, 96, seed=7)
    clean = call(s)
    s["xc"][2, 40] = 0x7F
    got = call(s)
    assert got[2].isnan().all() and torch.equal(got[[0, 1, 3]], clean[[0, 1, 3]])


def test_the_same_bits_every_time():
    s = layer(9, 4, 16, 256, 512, seed=8)
    a = call(s)
    for _ in range(5):
        assert torch.equal(a, call(s))


def test_next_to_the_sorted_path():
    """The same layer through sort, gather, swiglu, matmul and combine, whose h is rounded to 8 bits: half a step is
    2^-4 of each h, so 2^-4 of the absolute sum at most."""
    s = layer(8, 4, 12, 256, 512, seed=9)
    offsets, _, slots = w.fp8q_moe_sort(s["ids"], 12)
    rows, scales = w.mxfp8_moe_gather(s["xc"], s["xs"], slots, offsets)
    h, hs = w.mxfp8_moe_swiglu(rows, scales, *s["gate"][:2], *s["up"][:2], offsets)
    y = w.fp8q_moe_combine(w.mxfp8_moe_matmul(h, hs, *s["down"][:2], offsets), slots, offsets, s["p"])
    hv = values(h, hs)
    size = torch.zeros(8, 512, dtype=torch.float64, device="cuda")
    for t in range(8):
        for j in range(4):
            size[t] += float(s["p"][t, j]) * (s["down"][2][int(s["ids"][t, j])].abs() @ hv[int(slots[t, j])].abs())
    assert ((call(s).double() - y.double()).abs() <= size * (2.0 ** -4 * 1.07 + 2.0 ** -7)).all()


def test_captured_on_another_stream_and_two_at_once():
    s, r = layer(5, 3, 8, 128, 256, seed=10), layer(2, 2, 4, 96, 160, seed=11)
    want, want_r = call(s), call(r)
    torch.cuda.synchronize()
    side = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        a, b = call(s, stream=side[0]), call(r, stream=side[1])
        torch.cuda.synchronize()
        assert torch.equal(a, want) and torch.equal(b, want_r)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = call(s), call(r)
    for _ in range(3):
        a.zero_(), b.zero_()
        graph.replay()
        assert torch.equal(a, want) and torch.equal(b, want_r)
    s["ids"].copy_(s["ids"].flip(0))
    graph.replay()
    assert torch.equal(a, call(s))


def test_ids_and_weights_made_just_before():
    """Inputs written by the launch right before the call, and outputs read by the one right behind it."""
    s = layer(8, 4, 16, 256, 512, seed=12)
    want = call(s)
    ids, p = s["ids"].clone(), s["p"].clone()
    for _ in range(20):
        s["ids"].fill_(-1)
        s["p"].zero_()
        s["p"].copy_(p)
        s["ids"].copy_(ids)
        assert torch.equal(call(s).clone(), want)


def test_weights_made_just_before():
    """Weights that the launch right before the call writes over those of the call before it."""
    s, r = layer(3, 2, 4, 256, 512, seed=14), layer(3, 2, 4, 256, 512, seed=15)
    for name in ("xc", "xs", "ids", "p"):
        r[name] = s[name]
    g = torch.Generator(device="cuda").manual_seed(16)
    raw = [torch.randn(4, 512, 256, generator=g, device="cuda").bfloat16() * 0.06 for _ in range(2)]
    live = w.mxfp8_quantize_swizzled(raw[0])
    want = []
    for v in raw:
        s["down"] = w.mxfp8_quantize_swizzled(v)
        want.append(call(s).clone())
    s["down"] = live
    torch.cuda.synchronize()
    got = []
    for i in range(30):
        w.mxfp8_quantize_swizzled(raw[i % 2], codes=live[0], scales_swizzled=live[1])
        got.append(call(s))
    assert all(torch.equal(v, want[i % 2]) for i, v in enumerate(got))


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 6, 8, 9, 11, 20])
def test_rows_of_one_expert(rows):
    """Every number of rows that a tile's columns hold, with lengths that end inside a group of four blocks."""
    for n, k in ((160, 736), (224, 96)):
        check(layer(rows, 1, 1, n, k, seed=rows + n))


@pytest.mark.parametrize("rows", [2, 3, 4, 7, 12])
def test_nan_stays_with_its_row_of_an_expert(rows):
    """A row without numbers beside others of the same expert, in the products' columns as in their sums."""
    s = layer(rows, 1, 1, 96, 224, seed=rows)
    clean = call(s)
    for bad in (0, rows - 1):
        r = dict(s, xc=s["xc"].clone())
        r["xc"][bad] = 0x7F
        got = call(r)
        others = [i for i in range(rows) if i != bad]
        assert got[bad].isnan().all() and torch.equal(got[others], clean[others])


@pytest.mark.parametrize("tokens,topk,n", [(2, 8, 768), (3, 6, 640), (1, 13, 1120)])
def test_items_between_two_and_three_per_multiprocessor(tokens, topk, n):
    """Which on 152 of them run with three blocks on each."""
    s = layer(tokens, topk, 40, n, 256, seed=n)
    s["ids"] = torch.randperm(40, device="cuda")[:tokens * topk].view(tokens, topk)
    check(s)


def test_refusals_of_the_binding():
    s = layer(4, 2, 3, 64, 96, seed=13)
    with pytest.raises(ValueError, match="ids"):
        call(dict(s, ids=s["ids"].float()))
    with pytest.raises(ValueError, match="weights"):
        call(dict(s, p=s["p"][:, :1].contiguous()))
    with pytest.raises(ValueError, match="down_codes"):
        call(dict(s, down=s["gate"]))
    with pytest.raises(w.Fp8qError, match="SIZE"):
        call(dict(s, **{k: s[k].repeat(9, 1) for k in ("xc", "xs", "ids", "p")}))
