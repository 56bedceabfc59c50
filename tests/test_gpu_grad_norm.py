"""The global gradient norm and clipping against the formulas in 64 bits.

Tolerances.  A thread sums 64 squares in binary32, in eight chains of 8 and three
joins, and a warp its 32 sums in five more: 16 roundings of 2^-24, which the
square root halves; then one of the result.  So 9 (taken as 10) * 2^-24 for a
norm, one more for the coefficient; a clipped
gradient carries the coefficient's, the factor's and the product's roundings and
that of its type."""
import math

import pytest
import torch

import weight_transfer_gb300 as w

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
KINDS = [torch.bfloat16, torch.float32]


def views(sizes, kinds, seed, gap=0, size=1e-3):
    """Tensors one after the other in a flat buffer per type, `gap` elements apart; -> (tensors, flat buffers)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    flat = {k: (torch.randn(sum(n + gap for n, t in zip(sizes, kinds) if t is k) + 1, generator=g, device="cuda") * size).to(k)
            for k in KINDS}
    at = dict.fromkeys(KINDS, 0)
    out = []
    for n, k in zip(sizes, kinds):
        out.append(flat[k][at[k]:at[k] + n])
        at[k] += n + gap
    return out, flat


def squares(tensors):
    return torch.stack([t.double().square().sum() for t in tensors]) if tensors else torch.zeros(0, dtype=torch.float64, device="cuda")


def check_norm(norm, each, tensors, max_norm, scale):
    sq = squares(tensors)
    want = math.sqrt(float(sq.sum())) * scale
    coefficient = min(1.0, max_norm / (want + 1e-6))
    near(norm[:1].double(), torch.tensor([want], device="cuda", dtype=torch.float64), 10)
    near(norm[1:].double(), torch.tensor([coefficient], device="cuda", dtype=torch.float64), 11)
    if each is not None:
        near(each.double(), sq.sqrt() * scale, 10)
    return coefficient


def near(got, want, roundings):
    """Within so many roundings; half a step of 2^-149 among the smallest, and infinite past binary32's range."""
    over = want.float().isinf()
    ok = torch.where(over, got == want.float().double(), (got - want).abs() <= roundings * U * want + 2.0 ** -149)
    assert ok.all(), (got[~ok][:3], want[~ok][:3])


def check_clip(sizes, kinds, out_kinds, max_norm, scale, seed=0, gap=3, size=1e-3):
    grads, flat = views(sizes, kinds, seed, gap, size)
    before = {k: v.clone() for k, v in flat.items()}
    outs, oflat = views(sizes, out_kinds, seed + 1, gap)
    for f in oflat.values():
        f.fill_(9.0)
    norm, each = w.fp8q_grad_clip(grads, max_norm, scale, outs=outs, want_each=True)
    coefficient = check_norm(norm, each, grads, max_norm, scale)
    for g, o in zip(grads, outs):
        want = g.double() * (coefficient * scale)
        tol = want.abs() * (14 * U + HALF[o.dtype]) + 2.0 ** -134
        assert ((o.double() - want).abs() <= tol).all()
        o.fill_(9.0)
    for k in KINDS:
        assert torch.equal(flat[k], before[k]), "a gradient changed"
        assert (oflat[k] == 9.0).all(), "something was written between the outputs"


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 255, 4095, 16383, 16384, 16385, 16399, 100003, 1 << 20])
def test_one_tensor(n, kind):
    g, _ = views([n], [kind], seed=n)
    norm, each = w.fp8q_grad_norm(g, 0.5, 0.25, want_each=True)
    check_norm(norm, each, g, 0.5, 0.25)
    for out in KINDS:
        check_clip([n], [kind], [out], 1e-3, 0.25, seed=n)


@pytest.mark.parametrize("offset", range(9))
@pytest.mark.parametrize("kind", KINDS)
def test_unaligned(kind, offset):
    for n in (1, 6, 20, 16384, 33000):
        flat = torch.full((n + 24,), float("nan"), dtype=kind, device="cuda")
        g = flat[offset:offset + n]
        g.normal_()
        norm, _ = w.fp8q_grad_norm([g])
        check_norm(norm, None, [g], math.inf, 1.0)


@pytest.mark.parametrize("count", [1, 2, 31, 32, 33, 300, 1024, 1025, 2500])
def test_many_ragged_tensors(count):
    g = torch.Generator().manual_seed(count)
    sizes = [int(s) for s in torch.randint(1, 3000, (count,), generator=g)]
    sizes[count // 2] = 70001
    if count > 4:
        sizes[3] = 0
    kinds = [KINDS[i % 3 == 1] for i in range(count)]
    for gap in (0, 5):
        check_clip(sizes, kinds, [KINDS[i % 2] for i in range(count)], 0.01, 0.125, seed=count, gap=gap)
        check_clip(sizes, kinds, kinds, 1e9, 1.0, seed=count, gap=gap)


@pytest.mark.parametrize("kind", KINDS)
def test_in_place(kind):
    sizes = [5, 40000, 1, 16384, 777]
    g, flat = views(sizes, [kind] * 5, seed=1, gap=2)
    before = [t.clone() for t in g]
    rest = flat[kind].clone()
    held = w.fp8q_grad_list(g)
    norm, _ = w.fp8q_grad_clip(held, 0.1, 0.5)
    f = torch.tensor(0.5) * norm[1].cpu()
    for t, b in zip(g, before):
        assert torch.equal(t, (b.float() * f.cuda()).to(kind))
        t.zero_()
    at = 0
    for n in sizes:
        rest[at:at + n] = 0
        at += n + 2
    assert torch.equal(flat[kind], rest)
    g2, _ = views(sizes, [kind] * 5, seed=1, gap=2)
    same = [t.clone() for t in g2]
    norm, _ = w.fp8q_grad_clip(g2, 1e6)                       # nothing to clip
    assert norm[1] == 1.0 and all(torch.equal(a, b) for a, b in zip(g2, same))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [1e-44, 1e-38, 1e-30, 1e-20, 1e-13, 1e-11, 1.0, 1e15, 1e19, 1e30, 1e37])
def test_any_magnitude(kind, size):
    """Squares that binary32 cannot hold."""
    n = 30001
    g, _ = views([n, 50], [kind] * 2, seed=2, size=size)
    norm, each = w.fp8q_grad_norm(g, 1.0, 1.0, want_each=True)
    check_norm(norm, each, g, 1.0, 1.0)
    mixed = torch.zeros(n, dtype=kind, device="cuda")
    mixed[::1000] = size
    mixed[5] = size * 1e-6
    norm, _ = w.fp8q_grad_norm([mixed])
    check_norm(norm, None, [mixed], math.inf, 1.0)


@pytest.mark.parametrize("kind", KINDS)
def test_zeros_among_the_gradients(kind):
    """Rows that got no gradient: whole warps of zeros, lanes of zeros beside others, and one value alone."""
    x = torch.zeros(200_000, dtype=kind, device="cuda")
    x[70_000:90_000] = 1e-4
    x[199_999] = -3.0
    x[100_000:120_000:97] = 1e-12
    norm, each = w.fp8q_grad_norm([x, x[:60_000], x[120_000:199_000]], want_each=True)
    check_norm(norm, each, [x, x[:60_000], x[120_000:199_000]], math.inf, 1.0)


def test_zero_and_nothing():
    z = torch.zeros(40000, device="cuda")
    norm, each = w.fp8q_grad_norm([z, z[:0]], 2.0, want_each=True)
    assert norm.tolist() == [0.0, 1.0] and each.tolist() == [0.0, 0.0]
    norm, each = w.fp8q_grad_clip([], 1e-7, want_each=True)
    assert norm[0] == 0.0 and abs(float(norm[1]) - 0.1) < 1e-8 and each.numel() == 0
    norm, _ = w.fp8q_grad_norm([z, z])                          # the same tensor twice
    assert norm[0] == 0.0


@pytest.mark.parametrize("kind", KINDS)
def test_nan_and_infinite_gradients(kind):
    for value in (math.nan, math.inf, -math.inf):
        g = torch.ones(50000, dtype=kind, device="cuda")
        g[40001] = value
        out = torch.empty_like(g)
        norm, each = w.fp8q_grad_clip([g, torch.ones(5, dtype=kind, device="cuda")], 1.0, want_each=True,
                                      outs=[out, torch.empty(5, dtype=kind, device="cuda")])
        if math.isnan(value):
            assert norm.isnan().all() and out.isnan().all() and each[0].isnan()
        else:
            assert norm.tolist() == [math.inf, 0.0] and each[0] == math.inf
            assert out[40001].isnan() and not out[:40000].any()
        assert abs(float(each[1]) - math.sqrt(5)) < 1e-6


def test_the_same_bits_every_time_and_in_any_table():
    sizes = [50001] * 40
    g, _ = views(sizes, [torch.bfloat16] * 40, seed=4)
    a, e = w.fp8q_grad_norm(g, want_each=True)
    for _ in range(4):
        b, f = w.fp8q_grad_norm(w.fp8q_grad_list(g), want_each=True)
        assert torch.equal(a, b) and torch.equal(e, f)


def test_more_than_2_to_the_31_elements():
    """Chunks of more than 16,384 elements, and indexes past 32 bits."""
    n = (1 << 31) + 12345
    x = torch.zeros(n + 1, dtype=torch.bfloat16, device="cuda")[1:]
    x[::10007] = 3.0
    x[-1] = 4.0
    want = math.sqrt(9.0 * len(range(0, n, 10007)) + (16.0 if (n - 1) % 10007 else 7.0))
    norm, each = w.fp8q_grad_clip([x, x[:0]], want / 2, want_each=True)
    assert abs(float(norm[0]) - want) <= 10 * U * want and each[0] == norm[0]
    assert float(x[-1]) == 2.0 and float(x[10007 * 200000]) == 1.5 and int((x != 0).sum()) in (len(range(0, n, 10007)) + 1,
                                                                                               len(range(0, n, 10007)))


def test_captured_on_another_stream_and_two_at_once():
    sizes, kinds = [30000, 7, 100001], [torch.bfloat16, torch.float32, torch.float32]
    g, flat = views(sizes, kinds, seed=5)
    outs, oflat = views(sizes, kinds, seed=6)
    held = w.fp8q_grad_list(g, outs)
    want, _ = w.fp8q_grad_clip(held, 0.05)
    want_outs = [o.clone() for o in outs]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, _ = w.fp8q_grad_clip(held, 0.05, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured, _ = w.fp8q_grad_clip(held, 0.05)
    del held
    for o in oflat.values():
        o.zero_()
    captured.zero_()
    graph.replay()
    assert torch.equal(captured, want) and all(torch.equal(a, b) for a, b in zip(outs, want_outs))
    for k in flat:
        flat[k].mul_(2)
    graph.replay()
    assert abs(float(captured[0] / want[0]) - 2) < 1e-6
    a, _ = views([200001], [torch.float32], seed=7)
    b, _ = views([333, 5555], [torch.bfloat16] * 2, seed=8)
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        na, nb = (w.fp8q_grad_norm(v, stream=q)[0] for v, q in ((a, s[0]), (b, s[1])))
        torch.cuda.synchronize()
        check_norm(na, None, a, math.inf, 1.0)
        check_norm(nb, None, b, math.inf, 1.0)


def test_a_long_list_captured():
    """More tensors than the small table holds, and than one table holds: each node of the graph keeps its own."""
    for count in (65, 1500):
        sizes = [100 + i % 7 for i in range(count)]
        g, flat = views(sizes, [torch.float32] * count, seed=count)
        outs, oflat = views(sizes, [torch.bfloat16] * count, seed=1)
        want, want_each = w.fp8q_grad_clip(g, 0.01, 0.5, outs=outs, want_each=True)
        want_flat = oflat[torch.bfloat16].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got, each = w.fp8q_grad_clip(w.fp8q_grad_list(g, outs), 0.01, 0.5, want_each=True)
        w.fp8q_grad_norm(views([50] * 2000, [torch.float32] * 2000, seed=9)[0])      # another list in between
        oflat[torch.bfloat16].zero_(), got.zero_(), each.zero_()
        graph.replay()
        assert torch.equal(got, want) and torch.equal(each, want_each)
        n = sum(sizes)
        assert torch.equal(oflat[torch.bfloat16][:n], want_flat[:n])


def test_refusals_of_the_binding():
    a, b = torch.ones(10, device="cuda"), torch.ones(10, device="cuda", dtype=torch.float16)
    for bad in ([b], [a.view(2, 5).T]):
        with pytest.raises(ValueError):
            w.fp8q_grad_norm(bad)
    with pytest.raises(ValueError, match="elements"):
        w.fp8q_grad_list([a], [a[:5]])
    with pytest.raises(w.Fp8qError, match="ALIAS"):
        w.fp8q_grad_clip([a, a], 1.0)
    with pytest.raises(w.Fp8qError, match="SIZE"):
        w.fp8q_grad_clip([a], 0.0)
    with pytest.raises(ValueError, match="has its outputs"):
        w.fp8q_grad_clip(w.fp8q_grad_list([a]), 1.0, outs=[a])


@pytest.mark.parametrize("scale,factor", [(1e300, 0.0), (1e-300, 0.0), (1.0 / 3.0, None)])
def test_scale_beyond_binary32(scale, factor):
    """The factor is RN(scale * coefficient) of a scale in binary64: the coefficient of 1e300 is 0, and so is the
    factor; with 1e-300 the factor rounds to 0; with 1/3 it is rounded once."""
    g, _ = views([1000], [torch.float32], seed=5)
    before = g[0].clone()
    norm, _ = w.fp8q_grad_clip(g, 1e30, scale)
    want = torch.tensor(scale * float(norm[1]), dtype=torch.float64).float() if factor is None else torch.tensor(factor)
    assert torch.equal(g[0], before * want.cuda())


def test_infinite_norm_and_limit():
    """inf / inf: the coefficient of an infinite norm is 0 for any finite limit and NaN without one."""
    g = [torch.tensor([1.0, math.inf], device="cuda")]
    assert float(w.fp8q_grad_norm(g, 2.0)[0][1]) == 0.0
    assert math.isnan(float(w.fp8q_grad_norm(g)[0][1]))
