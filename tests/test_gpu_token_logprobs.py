"""Scores of given tokens and their gradient against the formulas in 64 bits.

Tolerances.  Every exponential carries the instruction's 2^-22 and the roundings
of its argument z = (x - m) / T, at most 3 |z| 2^-24; a sum of n terms in any
order at most n 2^-24; each of up to 32 joins of partial results another
exponential and three roundings.  Weighted with p that is, for log S,
2^-24 (n + 128 + 3 E|z|), and for the entropy the same times 1 + E|z|, with the
argument's roundings once more times |z|.  A thread adds at most vocab / 128 + 40
terms by itself."""
import math

import pytest
import torch

import weight_transfer_gb300 as w
from gpu_util import Guarded

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
LOWEST = {t: torch.finfo(t).min for t in TYPES.values()}


def formula(x, targets, T):
    """-> dict of 64-bit scores and the sizes that the tolerances need; masked logits add nothing."""
    x = x.double()
    m = x.max(1, keepdim=True).values
    none = torch.isinf(m) & (m < 0)
    z = torch.where(none, torch.full_like(x, -math.inf), (x - torch.where(none, 0.0, m)) / T)
    e = torch.exp(z)
    S = e.sum(1)
    p = e / torch.where(S > 0, S, 1.0)[:, None]
    zz = torch.where(e > 0, z, 0.0)
    log_s = torch.where(S > 0, torch.log(S), 0.0)
    H = torch.where(S > 0, log_s - (p * zz).sum(1), 0.0)
    logp = torch.where(none, torch.full_like(z, -math.inf), z - log_s[:, None])
    out = {"m": m[:, 0], "log_s": log_s, "H": H, "logp": logp, "p": p, "ez": (p * zz.abs()).sum(1), "ez2": (p * zz * zz).sum(1)}
    if targets is not None:
        t = targets.long()
        ok = (t >= 0) & (t < x.shape[1])
        out["at"] = torch.where(ok, logp.gather(1, torch.where(ok, t, 0)[:, None])[:, 0], 0.0)
    return out


def best(x, top):
    return torch.sort(x.double() + 0.0, dim=1, descending=True, stable=True).indices[:, :top].to(torch.int32)


def terms(vocab):
    return vocab / 128 + 40 + 128


def close(got, want, tol, what):
    got = got.double()
    over = want.float().isinf()               # beyond binary32, where the rounded value is infinite
    same = (got == want) | (torch.isnan(got) & torch.isnan(want)) | (over & (got == want.float().double()))
    bad = ~same & ~((got - want).abs() <= tol)
    assert not bad.any(), (what, got[bad][:4], want[bad][:4], tol[bad][:4] if torch.is_tensor(tol) and tol.dim() else tol)


def check(x, targets, T=1.0, top=0, entropy=True, stats=True):
    """One call with every output in guarded memory, against the formulas; returns (stats, entropy)."""
    rows, vocab = x.shape
    bufs = {"logprobs": Guarded(rows, torch.float32), "entropy": Guarded(rows, torch.float32) if entropy else None,
            "top_logprobs": Guarded(rows * top, torch.float32) if top else None,
            "top_ids": Guarded(rows * top, torch.int32) if top else None,
            "stats": Guarded(rows * 2, torch.float32) if stats else None}
    lp, ent, tl, ti, st = w.fp8q_token_logprobs(x, targets, T, top, want_entropy=entropy, want_stats=stats,
                                                **{k: None if b is None else b.t for k, b in bufs.items()})
    torch.cuda.synchronize()
    for k, b in bufs.items():
        assert b is None or b.intact(), k
    T = float(torch.tensor(T, dtype=torch.float32))
    f = formula(x, targets, T)
    tol_s = U * (terms(vocab) + 3 * f["ez"])
    at = f["at"].abs().nan_to_num(posinf=0.0)
    close(lp, f["at"], tol_s + U * (6 * at + 3 * f["log_s"].abs()), "logprobs")
    if entropy:
        close(ent, f["H"], U * (terms(vocab) * (1 + f["ez"]) + 8 * f["ez2"] + 4 * f["log_s"].abs()), "entropy")
    if stats:
        st = st.view(rows, 2)
        close(st[:, 0], f["m"], 0.0, "stats, largest")
        close(st[:, 1], f["log_s"], tol_s + U * 3 * f["log_s"].abs(), "stats, log S")
    if top:
        ti, tl = ti.view(rows, top), tl.view(rows, top)
        assert torch.equal(ti, best(x, top)), "alternatives"
        want = f["logp"].gather(1, ti.long())
        size = want.abs().nan_to_num(posinf=0.0)
        close(tl, want, (tol_s + U * 3 * f["log_s"].abs())[:, None] + U * 6 * size, "their scores")
    return st, ent


def logits(rows, vocab, dtype, seed, stride=None, offset=0, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    stride = stride or vocab
    flat = torch.randn(rows * stride + offset, generator=g, device="cuda") * spread
    flat[::211] += 9.0
    flat = flat.to(dtype)
    x = flat[offset:].as_strided((rows, vocab), (stride, 1))
    targets = torch.randint(0, vocab, (rows,), generator=g, device="cuda")
    return x, targets


VOCABS = [1, 2, 7, 8, 9, 31, 33, 64, 127, 129, 1000, 4095, 4097, 8192, 8193, 16391, 50257, 151936]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_vocabularies(vocab, dtype):
    for rows, top, T in ((3, min(vocab, 20), 1.0), (1, min(vocab, 1), 0.7), (2, 0, 1.3)):
        x, t = logits(rows, vocab, TYPES[dtype], seed=vocab + rows)
        check(x, t, T, top)
        check(x, t.int(), T, top, entropy=False, stats=False)


@pytest.mark.parametrize("rows", [1, 2, 5, 17, 38, 39, 75, 76, 77, 151, 152, 153, 305, 1000])
@pytest.mark.parametrize("top", [0, 32])
def test_rows(rows, top):
    """Row counts on both sides of each number of blocks per row."""
    x, t = logits(rows, 20011, torch.bfloat16, seed=rows)
    check(x, t, 1.0, top)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offset", [0, 1, 3, 4, 7])
@pytest.mark.parametrize("vocab,stride", [(5, 5), (5, 12), (1001, 1001), (1000, 1003), (40001, 40008)])
def test_rows_apart_and_unaligned(vocab, stride, offset, dtype):
    x, t = logits(9, vocab, TYPES[dtype], seed=offset, stride=stride, offset=offset)
    check(x, t, 1.0, min(5, vocab))


def test_targets_outside_the_vocabulary_score_zero():
    x, _ = logits(6, 500, torch.bfloat16, seed=1)
    t = torch.tensor([-100, -1, 0, 499, 500, 2 ** 40], device="cuda")
    lp = w.fp8q_token_logprobs(x, t)[0]
    assert lp[[0, 1, 4, 5]].tolist() == [0.0] * 4 and (lp[[2, 3]] < 0).all()
    check(x, t)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab", [40, 3000, 70001])
def test_masks(vocab, dtype):
    """Masked with -inf or with the type's lowest value: part of a row, all of it, all but one or a few logits."""
    dt = TYPES[dtype]
    x, t = logits(12, vocab, dt, seed=vocab)
    low = LOWEST[dt]
    x[0] = -math.inf
    x[1] = low
    x[2, vocab // 3:] = -math.inf
    x[3, : vocab // 3] = low
    x[4] = -math.inf; x[4, vocab - 1] = 2.0                 # noqa: E702
    x[5] = low; x[5, 0] = -5.0                              # noqa: E702
    x[6] = -math.inf; x[6, 1::vocab // 7] = 1.0             # noqa: E702
    x[7, ::2] = -math.inf; x[7, 1::2] = low                 # noqa: E702
    x[8] = -math.inf; x[8, vocab // 2] = low                # noqa: E702
    t[4], t[5], t[8] = vocab - 1, 0, vocab // 2
    for T in (1.0, 0.6, 2.0):
        check(x, t, T, 20)
        check(x, t, T, 0, entropy=False)
    lp, ent, tl, ti, st = w.fp8q_token_logprobs(x[:1], t[:1], top=20, want_entropy=True, want_stats=True)
    assert lp.item() == -math.inf and ent.item() == 0.0 and (tl == -math.inf).all() and st.tolist() == [[-math.inf, 0.0]]
    assert ti.tolist() == [list(range(20))]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_large_values(dtype):
    dt = TYPES[dtype]
    x, t = logits(5, 9000, dt, seed=3)
    big = torch.finfo(dt).max
    x[0] *= 1e30
    x[1, 17] = big
    x[2] = big
    x[3, ::2] = big; x[3, 1::2] = -big                      # noqa: E702
    x[4] *= 1e-30
    t[1], t[3] = 17, 4
    check(x, t, 1.0, 8)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [2.0 ** -20, 1e-3, 0.01, 0.1, 30.0, 2.0 ** 20])
def test_temperatures(T, dtype):
    """From one at which only the largest logit counts to one at which all are alike."""
    x, t = logits(6, 9001, TYPES[dtype], seed=12)
    x[1] *= 100
    x[2] *= 1e5
    x[3] *= 1e-3
    x[4, 4000:] = -math.inf
    t[0] = x[0].argmax()
    check(x, t, T, 6)
    check_gradient(x, t, T)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("size", [30.0, 300.0, 3e3, 1e5, 2e5, 1e6])
def test_logits_far_from_zero(size, dtype):
    """Rows whose logits lie around +size and -size, close to one another in the type's own steps."""
    g = torch.Generator(device="cuda").manual_seed(13)
    step = size * (2.0 ** -7 if dtype == "bf16" else 2.0 ** -20)
    x = (size + step * torch.randint(-20, 20, (4, 7003), generator=g, device="cuda")).to(TYPES[dtype])
    x[2:] = -x[2:]
    t = torch.randint(0, 7003, (4,), generator=g, device="cuda")
    check(x, t, 1.0, 5)
    check(x, t, 0.3, 0, entropy=False)
    check_gradient(x, t)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("order", ["equal", "rising", "falling", "steps", "zeros", "late"])
def test_alternatives_in_orders_that_overflow_the_candidates(order, dtype):
    """Equal, rising and stepped logits bring more candidates than there is room for."""
    vocab = 60000
    i = torch.arange(vocab, device="cuda", dtype=torch.float32)
    row = {"equal": torch.full_like(i, 1.5), "rising": i / 5000, "falling": -i / 5000, "steps": (i / 7000).floor(),
           "zeros": torch.where(i.long() % 3 == 0, -0.0, 0.0), "late": torch.where(i > 50000, 3.0, -i / 60000)}[order]
    x = row.to(TYPES[dtype]).expand(3, vocab).contiguous()
    x[1, 5] = 4.0
    x[2, 59990] = 5.0
    t = torch.tensor([0, 5, 59990], device="cuda")
    for top in (1, 20, 32):
        check(x, t, 1.0, top)
    many = x[:1].expand(700, vocab).contiguous()
    check(many, torch.zeros(700, dtype=torch.int64, device="cuda"), 1.0, 32)


@pytest.mark.parametrize("vocab", [151936, 1_000_003, 6_000_001])
def test_long_rows(vocab):
    """Rows whose steps share places of the stored maxima."""
    x, t = logits(2, vocab, torch.bfloat16, seed=14)
    check(x, t, 1.0, 32)
    x[0] = 2.0
    x[1, 7:] = x[1, :-7].sort().values
    check(x, t, 1.0, 32)


@pytest.mark.parametrize("rows", [70, 71, 72, 141, 142, 143, 304])
@pytest.mark.parametrize("top", [0, 5])
def test_rows_around_the_clusters_limits(rows, top):
    x, t = logits(rows, 40009, torch.float32, seed=rows)
    check(x, t, 0.8, top)


def test_many_long_rows():
    """So many rows that each is a block's own, with steps that share places: plain, equal, falling and masked ones."""
    x, t = logits(310, 131075, torch.float32, seed=17)
    x[1] = 3.0
    x[2] = x[2].sort(descending=True).values
    x[3, 5:] = -math.inf
    x[4, ::2] = x[4].max()
    x[5] = torch.arange(131075, device="cuda") // 1000
    check(x, t, 1.0, 8)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab,stride,offset", [(1, 1, 0), (5, 7, 1), (257, 257, 0), (1000, 1003, 3), (4001, 4001, 1), (12000, 12000, 0),
                                                 (12289, 12296, 5)])
def test_many_short_rows(vocab, stride, offset, dtype):
    """More rows than blocks at once, on both sides of the length from which a row has a block: random, masked, equal and
    infinite ones, padding's targets among them."""
    rows = 1217 if vocab > 5000 else 5003
    x, t = logits(rows, vocab, TYPES[dtype], seed=vocab, stride=stride, offset=offset)
    x[1] = -math.inf
    x[2] = torch.finfo(x.dtype).min
    x[3, 1:] = -math.inf
    x[4] = 7.0
    t[5::7] = -1
    t[6] = vocab
    check(x, t, 1.0, 0)
    y = x.clone()
    y[9, vocab // 2] = math.nan
    y[10, 0] = math.inf
    got, want = [w.fp8q_token_logprobs(v, t, want_entropy=True, want_stats=True) for v in (y, x.clone())]
    assert got[0][10].isnan() or t[10] < 0 or t[10] >= vocab
    others = torch.ones(rows, dtype=torch.bool, device="cuda")
    others[9:11] = False
    for a, b in zip(got, want):
        assert a is None or torch.equal(a[others].nan_to_num(2.0), b[others].nan_to_num(2.0))


def test_few_allowed_tokens():
    """Rows of which a grammar leaves a handful of tokens, in any places."""
    x = torch.full((40, 151669), -math.inf, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(15)
    for r in range(40):
        at = torch.randint(0, 151669, (r,), generator=g, device="cuda")
        x[r, at] = torch.randn(r, generator=g, device="cuda").bfloat16()
    check(x, torch.randint(0, 151669, (40,), generator=g, device="cuda"), 1.0, 20)


def test_infinite_and_nan_rows_leave_the_others_alone():
    x, t = logits(6, 5000, torch.float32, seed=8)
    clean = [o.clone() for o in w.fp8q_token_logprobs(x, t, top=5, want_entropy=True, want_stats=True)]
    x[1, 77] = math.nan
    x[4, 4321] = math.inf
    lp, ent, tl, ti, st = w.fp8q_token_logprobs(x, t, top=5, want_entropy=True, want_stats=True)
    keep = [0, 2, 3, 5]
    for a, b in zip((lp, ent, tl, ti, st), clean):
        assert torch.equal(a[keep], b[keep])
    assert lp[[1, 4]].isnan().all() and ent[[1, 4]].isnan().all() and tl[[1, 4]].isnan().all()
    assert ti[4, 0] == 4321
    y = x.clone()
    y[1, 77] = -math.inf                                     # among the alternatives a NaN counts as -inf
    assert torch.equal(ti[1:2], best(y[1:2], 5))
    nothing = torch.full((1, 50), math.nan, device="cuda")
    assert w.fp8q_token_logprobs(nothing, top=4)[3].tolist() == [[0, 1, 2, 3]]


def test_alternatives_without_targets_and_no_rows():
    x, _ = logits(4, 300, torch.bfloat16, seed=2)
    lp, ent, tl, ti, st = w.fp8q_token_logprobs(x, top=3)
    assert lp is None and ent is None and st is None and torch.equal(ti, best(x, 3))
    out = w.fp8q_token_logprobs(x[:0], torch.zeros(0, dtype=torch.int64, device="cuda"), top=3, want_entropy=True)
    assert [tuple(o.shape) for o in out[:4]] == [(0,), (0,), (0, 3), (0, 3)]


def test_the_same_bits_every_time():
    x, t = logits(30, 151936, torch.bfloat16, seed=4)
    a = w.fp8q_token_logprobs(x, t, top=32, want_entropy=True, want_stats=True)
    for _ in range(5):
        assert all(torch.equal(p, q) for p, q in zip(a, w.fp8q_token_logprobs(x, t, top=32, want_entropy=True, want_stats=True)))


# ---- gradient ----

def gradient(x, targets, stats, g, H, dh, T):
    """The formula in 64 bits on the statistics given, and what its tolerance needs."""
    x, st = x.double(), stats.double()
    none = torch.isinf(st[:, :1]) & (st[:, :1] < 0)
    z = torch.where(none, torch.full_like(x, -math.inf), (x - torch.where(none, 0.0, st[:, :1])) / T)
    logp = z - st[:, 1:]
    p = torch.exp(logp)
    lp = torch.where(p > 0, logp, 0.0)
    rows = torch.arange(x.shape[0], device=x.device)
    up = torch.zeros(x.shape[0], dtype=torch.float64, device=x.device)
    d = torch.zeros_like(x)
    size = torch.zeros_like(x)
    if g is not None:
        ok = (targets >= 0) & (targets < x.shape[1])
        up = torch.where(ok, g.double(), 0.0)
        d -= p * up[:, None]
        d[rows[ok], targets.long()[ok]] += up[ok]
        size[rows[ok], targets.long()[ok]] += up[ok].abs()
    inner = up.abs()[:, None]
    if dh is not None:
        d -= dh.double()[:, None] * p * (lp + H.double()[:, None])
        inner = inner + dh.double().abs()[:, None] * (lp.abs() + H.double().abs()[:, None])
    d = torch.where(none, 0.0, d)
    # p: the exponential's 2^-22 and the roundings of an argument of size |z| + |log S|; its factor: four roundings; a p
    # below 2^-126 is 0
    tol = p * inner * U * (16 + 6 * (z.clamp(min=-200).abs() + st[:, 1:].abs())) + 4 * U * size
    tol = tol + torch.where(p < 2.0 ** -125, p * inner, 0.0)
    return d / T, tol / T


def check_gradient(x, targets, T=1.0, policy=True, bonus=True, seed=0, dlogits=None, in_place=False):
    rows = x.shape[0]
    r = torch.Generator(device="cuda").manual_seed(seed)
    g = torch.randn(rows, generator=r, device="cuda") if policy else None
    dh = torch.randn(rows, generator=r, device="cuda") * 0.1 if bonus else None
    _, H, _, _, st = w.fp8q_token_logprobs(x, temperature=T, want_entropy=True, want_stats=True)
    T32 = float(torch.tensor(T, dtype=torch.float32))
    want, tol = gradient(x, targets, st, g, H, dh, T32)
    out = x if in_place else dlogits
    got = w.fp8q_token_logprobs_backward(x, targets if policy else None, st, g, H if bonus else None, dh, T, dlogits=out)
    assert got.shape == x.shape and got.dtype == x.dtype
    if out is not None:
        assert got.data_ptr() == out.data_ptr()
    close(got, want, tol + want.abs() * HALF[x.dtype] + 2.0 ** -133, "gradient")
    return got


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab", VOCABS)
def test_gradient_vocabularies(vocab, dtype):
    x, t = logits(5, vocab, TYPES[dtype], seed=vocab)
    t[1] = -100
    t[3] = vocab
    check_gradient(x, t)
    check_gradient(x, t.int(), 0.7, bonus=False)
    check_gradient(x, t, 1.4, policy=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offset", [0, 1, 5])
@pytest.mark.parametrize("vocab,stride", [(5, 5), (1001, 1001), (1000, 1003), (40001, 40008)])
def test_gradient_rows_apart_and_unaligned(vocab, stride, offset, dtype):
    x, t = logits(9, vocab, TYPES[dtype], seed=offset, stride=stride, offset=offset)
    check_gradient(x, t)
    for dstride, doffset in ((vocab, 0), (stride + 3, 2), (stride, offset)):      # rows that lie otherwise than the logits'
        flat = torch.full((9 * dstride + doffset + 8,), 7.0, dtype=x.dtype, device="cuda")
        d = flat[doffset:].as_strided((9, vocab), (dstride, 1))
        got = check_gradient(x, t, dlogits=d).clone()
        d.fill_(7.0)
        assert (flat == 7.0).all()                                                # nothing between the rows was written
        assert got.isfinite().all()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient_in_place(dtype):
    for vocab, stride in ((50257, 50257), (1000, 1008)):
        x, t = logits(7, vocab, TYPES[dtype], seed=vocab, stride=stride)
        apart = check_gradient(x, t, seed=3).clone()
        assert torch.equal(check_gradient(x, t, seed=3, in_place=True), apart)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradient_masks(dtype):
    dt = TYPES[dtype]
    x, t = logits(6, 3000, dt, seed=9)
    x[0] = -math.inf
    x[1] = LOWEST[dt]
    x[2, 100:] = -math.inf
    x[3, :2000] = LOWEST[dt]
    x[4] = -math.inf; x[4, 7] = 1.0                          # noqa: E702
    t[2], t[4] = 50, 7
    got = check_gradient(x, t)
    assert not got[0].any() and not got[2, 100:].any() and not got[4].any()


def test_rows_that_nothing_reaches_get_zeros():
    x, t = logits(4, 2000, torch.bfloat16, seed=5)
    st = w.fp8q_token_logprobs(x, t, want_stats=True)[4]
    x[1] = math.nan                                          # padding may hold anything
    t[1] = -100
    g = torch.ones(4, device="cuda")
    d = w.fp8q_token_logprobs_backward(x, t, st, g)
    assert not d[1].any() and d[[0, 2, 3]].isfinite().all() and d[0].any()


def test_gradient_against_differences():
    """Central differences of the 64-bit scores along random directions."""
    x, t = logits(3, 400, torch.float32, seed=6, spread=1.0)
    T = 0.8
    _, H, _, _, st = w.fp8q_token_logprobs(x, t, T, want_entropy=True, want_stats=True)
    g, dh = torch.tensor([1.0, -0.5, 2.0], device="cuda"), torch.tensor([0.3, 0.0, -1.0], device="cuda")
    d = w.fp8q_token_logprobs_backward(x, t, st, g, H, dh, T).double()
    T = float(torch.tensor(T, dtype=torch.float32))

    def score(v):
        f = formula(v, t, T)
        return (f["at"] * g + f["H"] * dh).sum()
    for seed in range(4):
        v = torch.randn(x.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").double()
        h = 1e-5
        slope = (score(x.double() + h * v) - score(x.double() - h * v)) / (2 * h)
        # 32-bit gradients of size 1 along a direction of norm 35, third derivatives of size 10 times h^2
        assert abs((d * v).sum() - slope) < 1e-4


def test_captured_and_on_another_stream():
    x, t = logits(20, 30011, torch.bfloat16, seed=7)
    g = torch.randn(20, device="cuda")
    want = w.fp8q_token_logprobs(x, t, top=4, want_entropy=True, want_stats=True)
    want_d = w.fp8q_token_logprobs_backward(x, t, want[4], g)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = w.fp8q_token_logprobs(x, t, top=4, want_entropy=True, want_stats=True, stream=side)
    got_d = w.fp8q_token_logprobs_backward(x, t, got[4], g, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(got_d, want_d)
    graph = torch.cuda.CUDAGraph()
    live = x.clone()
    with torch.cuda.graph(graph):
        out = w.fp8q_token_logprobs(live, t, top=4, want_entropy=True, want_stats=True)
        d = w.fp8q_token_logprobs_backward(live, t, out[4], g)
    for _ in range(2):
        for o in (*out, d):
            o.fill_(3)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(d, want_d)
    live.copy_(x.flip(0))
    graph.replay()
    again = w.fp8q_token_logprobs(live, t, top=4, want_entropy=True, want_stats=True)
    assert all(torch.equal(a, b) for a, b in zip(out, again))


def test_two_calls_at_once():
    a, ta = logits(64, 50257, torch.bfloat16, seed=1)
    b, tb = logits(3, 151936, torch.float32, seed=2)
    want = [w.fp8q_token_logprobs(v, t, top=8, want_entropy=True) for v, t in ((a, ta), (b, tb))]
    torch.cuda.synchronize()
    s = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        got = [w.fp8q_token_logprobs(v, t, top=8, want_entropy=True, stream=q) for (v, t), q in zip(((a, ta), (b, tb)), s)]
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for g_, w_ in zip(got, want) for p, q in zip(g_[:4], w_[:4]))


def test_offsets_past_32_bits():
    """Rows that start beyond 2^32 bytes and 2^31 elements."""
    rows, vocab, stride = 3, 1000, 1 << 30
    flat = torch.zeros(2 * stride + vocab, dtype=torch.bfloat16, device="cuda")
    x = flat.as_strided((rows, vocab), (stride, 1))
    src, t = logits(rows, vocab, torch.bfloat16, seed=11)
    x.copy_(src)
    check(x, t, 1.0, 10)
    _, H, _, _, st = w.fp8q_token_logprobs(src, temperature=1.0, want_entropy=True, want_stats=True)
    g = torch.ones(rows, device="cuda")
    d = w.fp8q_token_logprobs_backward(x, t, st, g, dlogits=x)
    assert torch.equal(d, w.fp8q_token_logprobs_backward(src, t, st, g)) and not flat[vocab:stride].any()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab,stride,offset", [(1, 1, 0), (5, 7, 1), (257, 257, 0), (1000, 1003, 3), (1500, 1500, 0), (1501, 1504, 1),
                                                 (3000, 3000, 0), (3001, 3011, 1)])
def test_gradient_of_many_short_rows(vocab, stride, offset, dtype):
    """On both sides of the length from which a row has a block of its own."""
    x, t = logits(1217, vocab, TYPES[dtype], seed=vocab, stride=stride, offset=offset)
    x[1] = -math.inf
    x[3, 1:] = -math.inf
    t[5::7] = -1
    t[6] = vocab
    check_gradient(x, t)
    check_gradient(x, t, bonus=False)
    check_gradient(x, t, 0.7, policy=False)
