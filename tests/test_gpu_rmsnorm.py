"""Norm with an 8-bit output and its gradient against 64-bit formulas.

Tolerances.  The forward value y carries: one rounding of the sum, at most
(8 * 4 + 5 + 16) roundings in the sum of squares (halved by the square root),
and five more (mean, eps, square root, quotient, two products): under 32
half-steps of 2^-24, so 2^-18 relative; TOL = 2^-17 leaves a factor of two.
Codes may differ from the 64-bit ones only where a rounding boundary lies
within TOL of the value.  Gradient: the same count for xhat and the mean;
errors are relative to |g| + |xhat * mean|, the terms of the difference."""
import pytest
import torch

from expert_block_ref import check_bf16, check_codes, check_mx, decode, unswizzle

pytestmark = pytest.mark.gpu

TOL = 2.0 ** -17
EPS = 1e-6
SHAPES = [(1, 32), (1, 2048), (3, 96), (7, 128), (5, 2080), (129, 256), (2, 4096), (33, 4128), (4, 8192), (3, 8224),
          (2, 16384), (300, 1408)]


@pytest.fixture(scope="module")
def w():
    import weight_transfer_gb300 as m
    return m


def make(rows, k, seed, residual=True):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, k, generator=g) * torch.exp(2 * torch.randn(rows, 1, generator=g))
    x[:, ::17] *= 30
    r = torch.randn(rows, k, generator=g) * 3
    if rows > 2:
        x[1] = 0                      # a row of zeros in x; and with the residual's row zero too, an all-zero row
        r[1] = 0
        x[2, : k // 2] = 0            # whole blocks that hold nothing
        r[2, : k // 2] = 0
    wt = 1 + 0.3 * torch.randn(k, generator=g)
    x, r, wt = x.bfloat16().cuda(), r.bfloat16().cuda(), wt.bfloat16().cuda()
    return x, (r if residual else None), wt


def exact(x, r, wt, eps=EPS):
    h = x.double().cpu() + (0 if r is None else r.double().cpu())
    rstd = 1 / torch.sqrt((h * h).mean(1) + eps)
    return h, rstd, h * rstd[:, None] * wt.double().cpu()


def check_extras(total, y16, rstd, x, r, y, rs):
    assert torch.allclose(rstd.double().cpu(), rs, rtol=TOL, atol=0)
    check_bf16(y16, y, TOL)
    if r is None:
        assert total is None
    else:
        assert torch.equal(total, (x.float() + r.float()).bfloat16())


@pytest.mark.parametrize("rows,k", SHAPES)
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("swizzled", [False, True])
def test_mxfp8(w, rows, k, residual, swizzled):
    x, r, wt = make(rows, k, rows * k, residual)
    _, rs, y = exact(x, r, wt)
    sb = w.mxfp8_swizzled_scale_bytes(1, rows, k) if swizzled else rows * k // 32
    scales = torch.full((sb,), 0xA5, dtype=torch.uint8, device="cuda")
    codes, scales, total, y16, rstd = w.mxfp8_rmsnorm_quantize(x, wt, EPS, residual=r, swizzled=swizzled, want_bf16=True,
                                                               want_rstd=True, scales=scales)
    check_extras(total, y16, rstd, x, r, y, rs)
    if swizzled:
        e, full = unswizzle(scales.cpu().long(), rows, k // 32)
        assert int(full.sum()) == int(e.sum())              # padding is zero
    else:
        e = scales.cpu().long().reshape(rows, k // 32)
    check_mx(y, codes, e, TOL)


@pytest.mark.parametrize("rows,k", [s for s in SHAPES if s[1] % 128 == 0])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_blockwise(w, rows, k, fmt):
    x, r, wt = make(rows, k, rows + k)
    _, rs, y = exact(x, r, wt)
    codes, s, total, y16, rstd = w.fp8q_rmsnorm_quantize(x, wt, EPS, fmt, residual=r, want_bf16=True, want_rstd=True)
    check_extras(total, y16, rstd, x, r, y, rs)
    b = y.reshape(rows, -1, 128)
    fmax = 448.0 if fmt == "e4m3" else 57344.0
    s = s.double().cpu()
    assert torch.allclose(s, b.abs().amax(2) / fmax, rtol=TOL, atol=0)
    q = torch.where(s[..., None] > 0, b / s.clamp(min=1e-300)[..., None], b * 0)
    check_codes(q, decode(codes, fmt).reshape(b.shape), TOL, fmt)


def test_in_place_sum_and_optional_outputs(w):
    x, r, wt = make(65, 2048, 5)
    want = w.mxfp8_rmsnorm_quantize(x, wt, EPS, residual=r)
    assert want[3] is None and want[4] is None
    for over in ("x", "residual"):
        x2, r2 = x.clone(), r.clone()
        got = w.mxfp8_rmsnorm_quantize(x2, wt, EPS, residual=r2, out_sum=x2 if over == "x" else r2)
        for a, b in zip(want[:3], got[:3]):
            assert torch.equal(a, b)


def test_empty(w):
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    wt = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    codes, scales, *_ = w.mxfp8_rmsnorm_quantize(x, wt)
    assert codes.shape == (0, 256) and scales.shape == (0, 8)
    dx, dw = w.fp8q_rmsnorm_backward(x, x, wt, torch.empty(0, device="cuda"), dweight=torch.full((256,), 7.0, device="cuda"))
    assert not dw.any()


def test_quantizes_as_the_weight_quantizer_does(w):
    """With weight 1 and rows scaled so that rstd is exactly 1, the codes and scales are mxfp8_quantize_swizzled's."""
    rows, k = 130, 512
    g = torch.Generator().manual_seed(3)
    x = torch.where(torch.rand(rows, k, generator=g) < 0.5, -1.0, 1.0)      # mean of squares 1, eps 0
    x = x.bfloat16().cuda()
    wt = torch.ones(k, dtype=torch.bfloat16, device="cuda")
    codes, scales, *_ = w.mxfp8_rmsnorm_quantize(x, wt, 0.0, swizzled=True)
    ec, es = w.mxfp8_quantize_swizzled(x)
    assert torch.equal(codes, ec) and torch.equal(scales, es)


@pytest.mark.parametrize("rows,k", SHAPES + [(2000, 512), (1300, 96)])
@pytest.mark.parametrize("residual", [False, True])
def test_gradient(w, rows, k, residual):
    x, r, wt = make(rows, k, 7 * rows + k, True)
    h = (x.float() + r.float()).bfloat16()
    g = torch.Generator().manual_seed(k)
    dy = torch.randn(rows, k, generator=g).bfloat16().cuda()
    dsum = torch.randn(rows, k, generator=g).bfloat16().cuda() if residual else None
    h64, dy64, w64 = h.double().cpu(), dy.double().cpu(), wt.double().cpu()
    rstd = (1 / torch.sqrt((h64 * h64).mean(1) + EPS)).float().cuda()
    dx, dw = w.fp8q_rmsnorm_backward(dy, h, wt, rstd, dsum=dsum)
    rs = rstd.double().cpu()[:, None]
    xh, gg = h64 * rs, dy64 * w64
    mean, size = (gg * xh).mean(1, keepdim=True), (gg * xh).abs().mean(1, keepdim=True)
    want = rs * (gg - xh * mean) + (0 if dsum is None else dsum.double().cpu())
    scale = rs * (gg.abs() + xh.abs() * size) + (0 if dsum is None else dsum.double().cpu().abs())
    check_bf16(dx, want, TOL, scale)
    # dw: per column at most (rows/blocks + blocks/8 + 8) additions of terms with two roundings each
    t = (dy64 * xh).abs().sum(0) * (rows / 152 + 100) * 2.0 ** -24
    assert ((dw.double().cpu() - (dy64 * xh).sum(0)).abs() <= t + 1e-30).all()


def test_gradient_is_the_derivative(w):
    """Central differences of the 64-bit formula, and the chain through both of its inputs."""
    rows, k = 3, 64
    g = torch.Generator().manual_seed(11)
    h = torch.randn(rows, k, generator=g).bfloat16()
    wt = (1 + 0.2 * torch.randn(k, generator=g)).bfloat16()
    dy = torch.randn(rows, k, generator=g).bfloat16()
    f = lambda hh, ww: float((dy.double() * hh / torch.sqrt((hh * hh).mean(1, keepdim=True) + EPS) * ww).sum())  # noqa: E731
    rstd = 1 / torch.sqrt((h.double() ** 2).mean(1) + EPS)
    dx, dw = w.fp8q_rmsnorm_backward(dy.cuda(), h.cuda(), wt.cuda(), rstd.float().cuda())
    step = 1e-5
    for i, j in [(0, 0), (1, 17), (2, 63), (0, 33)]:
        d = torch.zeros(rows, k, dtype=torch.float64)
        d[i, j] = step
        num = (f(h.double() + d, wt.double()) - f(h.double() - d, wt.double())) / (2 * step)
        # bf16 output: half a step of the value; the difference quotient is good to ~1e-8
        assert abs(float(dx[i, j]) - num) <= abs(num) * 2.0 ** -8 + 1e-6
        e = torch.zeros(k, dtype=torch.float64)
        e[j] = step
        num = (f(h.double(), wt.double() + e) - f(h.double(), wt.double() - e)) / (2 * step)
        assert abs(float(dw[j]) - num) <= 1e-5 * max(1.0, abs(num))


def test_gradient_in_place_and_repeatable(w):
    x, r, wt = make(700, 1408, 21)
    rstd = torch.rsqrt(x.float().square().mean(1) + EPS)
    dy, ds = torch.randn_like(x), torch.randn_like(x)
    want = w.fp8q_rmsnorm_backward(dy, x, wt, rstd, dsum=ds)
    a, b = dy.clone(), ds.clone()
    got = w.fp8q_rmsnorm_backward(a, x, wt, rstd, dsum=ds, dx=a)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    got = w.fp8q_rmsnorm_backward(dy, x, wt, rstd, dsum=b, dx=b)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_other_stream(w):
    x, r, wt = make(40, 2048, 9)
    want = w.mxfp8_rmsnorm_quantize(x, wt, EPS, residual=r)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = w.mxfp8_rmsnorm_quantize(x, wt, EPS, residual=r)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want[:3], got[:3]))


# rows of up to 128 elements share a warp, two to eight of them; here the last warp has some without a row
SHORT = [(37, 32), (1001, 64), (515, 128), (9, 96), (5000, 32)]


@pytest.mark.parametrize("rows,k", SHORT)
@pytest.mark.parametrize("residual", [False, True])
def test_short_rows(w, rows, k, residual):
    test_mxfp8(w, rows, k, residual, False)
    test_mxfp8(w, rows, k, residual, True)
    test_gradient(w, rows, k, residual)
    if k % 128 == 0:
        test_blockwise(w, rows, k, "e4m3")


@pytest.mark.parametrize("rows,k", [(37, 32), (51, 128), (9, 384), (5, 2048)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_rows_do_not_meet(w, rows, k, bad):
    """A row that holds NaN or an infinity leaves the others as they are, in both directions."""
    x, r, wt = make(rows, k, rows + 5 * k)
    dy = torch.randn_like(x)
    x2 = x.clone()
    x2[rows // 2, k // 3] = bad
    keep = torch.arange(rows, device="cuda") != rows // 2
    calls = [lambda t: w.mxfp8_rmsnorm_quantize(t, wt, EPS, residual=r, want_bf16=True, want_rstd=True)]
    if k % 128 == 0:
        calls.append(lambda t: w.fp8q_rmsnorm_quantize(t, wt, EPS, residual=r, want_bf16=True, want_rstd=True))
    for call in calls:
        for a, b in zip(call(x), call(x2)):
            a, b = (t.view(torch.uint8).reshape(rows, -1) for t in (a, b))
            assert torch.equal(a[keep], b[keep])
    rstd = torch.rsqrt(x.float().square().mean(1) + EPS)
    a, b = w.fp8q_rmsnorm_backward(dy, x, wt, rstd)[0], w.fp8q_rmsnorm_backward(dy, x2, wt, rstd)[0]
    assert torch.equal(a[keep], b[keep])
