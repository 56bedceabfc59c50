"""The experts' MXFP8 products.

Layout tests use small whole numbers as codes and scales of 1, 2 and 4: every
partial sum is then a whole number below 2^24, exact in binary32 whatever the
order, so the bf16 result is the rounding of the exact one, bit for bit.  The
random tests allow each accumulation step of 32 products 2^-22 of the sum of
magnitudes (the tensor core aligns a step's products and the accumulator to the
largest of them and may cut bits off below its last place): (k/32 + 1) * 2^-22."""
import pytest
import torch

from expert_block_ref import check_bf16, check_mx, decode, unswizzle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    import weight_transfer_gb300 as m
    return m


def whole_mx(shape, seed):
    """MXFP8 of whole numbers of magnitude <= 4 under scales 1, 2, 4: codes, exponent bytes, values."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(-4, 5, shape, generator=g).float()
    e = torch.randint(0, 3, (*shape[:-1], shape[-1] // 32), generator=g)
    codes = v.to(torch.float8_e4m3fn).view(torch.uint8)
    return codes, (e + 127).to(torch.uint8), v.double() * (2.0 ** e.double()).repeat_interleave(32, -1)


def swizzle(e):
    """[..., m, kb] bytes -> flat tiled bytes, padding 0."""
    lead, (m, kb) = e.shape[:-2], e.shape[-2:]
    r, c = -(-m // 128), -(-kb // 4)
    full = torch.zeros(*lead, r * 128, c * 4, dtype=torch.uint8)
    full[..., :m, :kb] = e
    n = len(lead)
    return full.reshape(*lead, r, 4, 32, c, 4).permute(*range(n), n, n + 3, n + 2, n + 1, n + 4).reshape(-1)


def groups(counts, rows):
    off = torch.tensor([0] + list(counts)).cumsum(0).to(torch.int32)
    assert int(off[-1]) <= rows
    e_of = torch.full((rows,), -1)
    for e in range(len(counts)):
        e_of[off[e]:off[e + 1]] = e
    return off.cuda(), e_of


def product(a, wv, e_of):
    out = torch.zeros(a.shape[0], wv.shape[1], dtype=torch.float64)
    for e in range(wv.shape[0]):
        out[e_of == e] = a[e_of == e] @ wv[e].T
    return out


COUNTS = [
    ([1], 1), ([16], 16), ([17], 17), ([224], 224), ([225], 230), ([112, 113], 225), ([1000], 1000),
    ([0, 3, 0, 1, 129, 0], 140), ([0, 0, 0], 5), ([5] * 40, 200), ([0, 500, 1, 30], 531), ([33, 0, 255, 47], 400),
]
NK = [(128, 128), (256, 2048), (96, 32), (160, 96), (768, 512), (131, 160), (32, 1056)]


@pytest.mark.parametrize("counts,rows", COUNTS)
@pytest.mark.parametrize("n,k", NK)
def test_matmul_exact(w, counts, rows, n, k):
    E = len(counts)
    off, e_of = groups(counts, rows)
    ac, ae, av = whole_mx((rows, k), 1)
    wc, we, wv = whole_mx((E, n, k), 2)
    out = torch.full((rows + 2, n + 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    buf = out.view(-1)[: rows * n].view(rows, n)
    got = w.mxfp8_moe_matmul(ac.cuda(), ae.cuda(), wc.cuda(), swizzle(we).cuda(), off, out=buf)
    want = product(av, wv, e_of)
    assert want.abs().max() < 2 ** 24
    assert torch.equal(got.cpu(), want.float().bfloat16())
    assert out.view(-1)[rows * n:].isnan().all()


@pytest.mark.parametrize("counts,rows", COUNTS)
@pytest.mark.parametrize("n,k", [(32, 32), (128, 128), (768, 2048), (160, 96), (96, 1056)])
def test_swiglu(w, counts, rows, n, k):
    """Whole-number products are exact, so only the activation's own error is left: expf (2 ulp), one addition, one
    division and one product, under 2^-20 relative; a small output scale keeps g in the range where silu bends."""
    E = len(counts)
    off, e_of = groups(counts, rows)
    ac, ae, av = whole_mx((rows, k), 3)
    gc, ge, gv = whole_mx((E, n, k), 4)
    uc, ue, uv = whole_mx((E, n, k), 5)
    ge, gv = ge - 10, gv * 2.0 ** -10
    buf = torch.full((rows * n + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    sbuf = torch.full((rows * n // 32 + 64,), 0xA5, dtype=torch.uint8, device="cuda")
    codes, scales = w.mxfp8_moe_swiglu(ac.cuda(), ae.cuda(), gc.cuda(), swizzle(ge).cuda(), uc.cuda(), swizzle(ue).cuda(), off,
                                       out_codes=buf[: rows * n].view(rows, n), out_scales=sbuf[: rows * n // 32].view(rows, n // 32))
    g, u = product(av, gv, e_of), product(av, uv, e_of)
    h = g / (1 + torch.exp(-g)) * u
    check_mx(h, codes, scales.cpu().long(), 2.0 ** -20)
    assert (buf[rows * n:] == 0xA5).all() and (sbuf[rows * n // 32:] == 0xA5).all()


@pytest.mark.parametrize("rows,E,n,k", [(8, 128, 256, 768), (513, 6, 384, 2048), (97, 2, 200, 4128)])
def test_matmul_random(w, rows, E, n, k):
    g = torch.Generator().manual_seed(rows)
    wt = (torch.randn(E, n, k, generator=g) * 0.02).bfloat16().cuda()
    wc, ws = w.mxfp8_quantize_swizzled(wt)
    x = torch.randn(rows, k, generator=g).bfloat16().cuda()
    ac, ae, *_ = w.mxfp8_rmsnorm_quantize(x, torch.ones(k, dtype=torch.bfloat16, device="cuda"))
    cuts = torch.sort(torch.randint(0, rows + 1, (E - 1,), generator=g)).values.tolist()
    counts = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
    off, e_of = groups(counts, rows)
    got = w.mxfp8_moe_matmul(ac, ae, wc, ws, off)
    av = decode(ac) * (2.0 ** (ae.cpu().double() - 127)).repeat_interleave(32, 1)
    per = ws.numel() // E
    exps = torch.stack([unswizzle(ws[e * per:(e + 1) * per].cpu(), n, k // 32)[0] for e in range(E)])
    wv = decode(wc) * (2.0 ** (exps.double() - 127)).repeat_interleave(32, 2)
    check_bf16(got, product(av, wv, e_of), (k / 32 + 1) * 2.0 ** -22, product(av.abs(), wv.abs(), e_of))


def test_extreme_scales_and_codes(w):
    """The largest codes under scales whose product is in range; zero codes under the smallest scale; and a NaN scale in
    a row that belongs to another expert's tile stays there."""
    rows, n, k = 3, 128, 128
    ac = torch.full((rows, k), 0x7E, dtype=torch.uint8)              # 448
    ac[1] = 0
    ae = torch.full((rows, k // 32), 127, dtype=torch.uint8)
    ae[1] = 0
    ae[2] = 255                                                       # NaN scale
    wc = torch.full((2, n, k), 0xFE, dtype=torch.uint8)               # -448
    we = torch.full((2, n, k // 32), 100, dtype=torch.uint8)
    off = torch.tensor([0, 2, 3], dtype=torch.int32)
    got = w.mxfp8_moe_matmul(ac.cuda(), ae.cuda(), wc.cuda(), swizzle(we).cuda(), off.cuda()).cpu()
    assert (got[0] == torch.tensor(-448.0 * 448 * 128 * 2.0 ** -27).bfloat16()).all()
    assert (got[1] == 0).all() and got[2].isnan().all()


def test_offsets_outside_the_rows_are_clamped(w):
    rows, n, k = 20, 64, 64
    ac, ae, av = whole_mx((rows, k), 1)
    wc, we, wv = whole_mx((3, n, k), 2)
    off = torch.tensor([-5, 7, 7, 90], dtype=torch.int32).cuda()
    got = w.mxfp8_moe_matmul(ac.cuda(), ae.cuda(), wc.cuda(), swizzle(we).cuda(), off)
    e_of = torch.tensor([0] * 7 + [2] * 13)
    assert torch.equal(got.cpu(), product(av, wv, e_of).float().bfloat16())


def test_other_stream_and_graph(w):
    rows, n, k = 140, 256, 512
    off, e_of = groups([0, 3, 0, 1, 129, 0], rows)
    ac, ae, av = whole_mx((rows, k), 1)
    wc, we, wv = whole_mx((6, n, k), 2)
    a = [t.cuda() for t in (ac, ae, wc, swizzle(we))]
    want = product(av, wv, e_of).float().bfloat16()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = w.mxfp8_moe_matmul(*a, off)
    s.synchronize()
    assert torch.equal(got.cpu(), want)
    out = torch.zeros(rows, n, dtype=torch.bfloat16, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        w.mxfp8_moe_matmul(*a, off, out=out)
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out.cpu(), want)


def test_empty(w):
    e = lambda *s: torch.empty(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    off = torch.zeros(3, dtype=torch.int32, device="cuda")
    out = w.mxfp8_moe_matmul(e(0, 64), e(0, 2), e(2, 96, 64), e(2 * 512), off)
    assert out.shape == (0, 96)


@pytest.mark.parametrize("counts,rows", [([60, 300, 0, 209, 70], 640), ([49], 49), ([417, 415], 840), ([1, 1, 700, 2, 0], 704),
                                         ([64] * 12, 768), ([49, 51], 100)])
@pytest.mark.parametrize("n,k", [(256, 160), (384, 128), (1100, 96), (130, 288), (512, 1024)])
def test_matmul_many_rows_per_expert(w, counts, rows, n, k):
    """Pairs of blocks (an even number of feature tiles, or at least 8), an odd tile out, and single blocks."""
    off, e_of = groups(counts, rows)
    ac, ae, av = whole_mx((rows, k), 6)
    wc, we, wv = whole_mx((len(counts), n, k), 7)
    got = w.mxfp8_moe_matmul(ac.cuda(), ae.cuda(), wc.cuda(), swizzle(we).cuda(), off)
    assert torch.equal(got.cpu(), product(av, wv, e_of).float().bfloat16())


@pytest.mark.parametrize("counts,rows", [([60, 300, 0, 209, 70], 640), ([113, 225], 350), ([1, 1, 700, 2, 0], 704)])
@pytest.mark.parametrize("n,k", [(256, 160), (1120, 96), (384, 1024), (288, 64)])
def test_swiglu_many_rows_per_expert(w, counts, rows, n, k):
    off, e_of = groups(counts, rows)
    ac, ae, av = whole_mx((rows, k), 8)
    gc, ge, gv = whole_mx((len(counts), n, k), 9)
    uc, ue, uv = whole_mx((len(counts), n, k), 10)
    ge, gv = ge - 10, gv * 2.0 ** -10
    codes, scales = w.mxfp8_moe_swiglu(ac.cuda(), ae.cuda(), gc.cuda(), swizzle(ge).cuda(), uc.cuda(), swizzle(ue).cuda(), off)
    g, u = product(av, gv, e_of), product(av, uv, e_of)
    check_mx(g / (1 + torch.exp(-g)) * u, codes, scales.cpu().long(), 2.0 ** -20)


@pytest.mark.parametrize("counts,rows", [([60, 300, 0, 209, 70], 640), ([49], 49), ([1, 1, 700, 2, 0], 704)])
@pytest.mark.parametrize("n,k", [(256, 1056), (384, 1248), (1120, 1056), (96, 1952)])
def test_long_odd_scale_rows(w, counts, rows, n, k):
    """Scale rows of 33, 39 and 61 bytes, shared by two warps: pairs and single blocks, up to the arrays' last byte."""
    test_matmul_many_rows_per_expert(w, counts, rows, n, k)
    test_swiglu_many_rows_per_expert(w, counts, rows, n, k)


@pytest.mark.parametrize("experts,rows,n", [(1024, 1300, 4096), (1, 150_000, 4096)])
def test_more_tiles_than_are_listed_ahead(w, experts, rows, n):
    """Over 128 tiles per block: those behind are found one by one."""
    k = 32
    g = torch.Generator().manual_seed(1)
    cuts = torch.sort(torch.randint(0, rows + 1, (experts - 1,), generator=g)).values.tolist()
    counts = [b - a for a, b in zip([0] + cuts, cuts + [rows])]
    off, e_of = groups(counts, rows)
    ac, ae, av = whole_mx((rows, k), 3)
    v = torch.randint(-4, 5, (experts, n, k), generator=g, dtype=torch.int8).cuda()
    wc = v.float().to(torch.float8_e4m3fn).view(torch.uint8)
    ws = torch.zeros(experts, n // 128, 512, dtype=torch.uint8, device="cuda")
    ws.view(experts, n // 128, 32, 4, 4)[..., 0] = 127               # one scale column of 1
    got = w.mxfp8_moe_matmul(ac.cuda(), ae.cuda(), wc, ws.reshape(-1), off)
    av, e_of = av.float().cuda(), e_of.cuda()
    for r0 in range(0, rows, 10_000):
        r = slice(r0, min(rows, r0 + 10_000))
        if experts == 1:
            want = av[r] @ v[0].float().T
        else:
            want = torch.einsum("rk,rnk->rn", av[r], v[e_of[r]].float())
        assert torch.equal(got[r], want.bfloat16())


def test_repeatable(w):
    rows, n, k = 3000, 768, 1056
    off, _ = groups([1000, 0, 1500, 100], rows)
    g = torch.Generator().manual_seed(2)
    wt = (torch.randn(4, n, k, generator=g) * 0.02).bfloat16().cuda()
    wc, ws = w.mxfp8_quantize_swizzled(wt)
    ac, ae, *_ = w.mxfp8_rmsnorm_quantize(torch.randn(rows, k, generator=g).bfloat16().cuda(),
                                          torch.ones(k, dtype=torch.bfloat16, device="cuda"))
    first = w.mxfp8_moe_matmul(ac, ae, wc, ws, off), *w.mxfp8_moe_swiglu(ac, ae, wc, ws, wc, ws, off)
    for _ in range(5):
        again = w.mxfp8_moe_matmul(ac, ae, wc, ws, off), *w.mxfp8_moe_swiglu(ac, ae, wc, ws, wc, ws, off)
        assert all(torch.equal(a, b) for a, b in zip(first, again))
