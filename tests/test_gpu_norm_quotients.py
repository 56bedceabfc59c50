"""The blockwise norm's codes are correctly rounded quotients, those of fp8q_quantize_blockwise.

Rows whose elements are all +-2 have a mean of squares of exactly 4; without eps the norm is then +-1 and y is +-weight
exactly, a bf16 value that the quantizer of plain arrays can be given.  The weights hold what shows a quotient that is
off by its last place: multiples m * b of the scale b, m between two codes (a tie that goes to the even one), beside
random values, signed zeros in whole blocks, blocks whose scale is below 2^-58 and 2^-100, subnormals and values near
the top of the range."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    import weight_transfer_gb300 as m
    return m


def weights(k, seed):
    g = torch.Generator().manual_seed(seed)
    wt = torch.randn(k // 128, 128, generator=g) * torch.exp2(torch.randint(-20, 20, (k // 128, 1), generator=g).float())
    for i in range(k // 128):
        kind = (i + seed) % 8
        if kind < 4:                            # the block's largest is 7 * 64 * b up to a power of two: the scale is b
            b = (7, 13, 15, 15)[kind]
            m = torch.randint(8, 16, (128,), generator=g) * 2 + 1
            e = -torch.randint(3, 8, (128,), generator=g).float()
            wt[i] = m * b * torch.exp2(e)
            wt[i, 1 + int(torch.randint(0, 8, (1,), generator=g))] = 7 * b
        elif kind == 4:
            wt[i] = 0
        elif kind == 5:
            wt[i] *= 2.0 ** -60
        elif kind == 6:
            wt[i] = torch.randn(128, generator=g) * (2.0 ** -95 if i % 2 else 2.0 ** -128)
        else:
            wt[i] = torch.randn(128, generator=g).clamp(-3, 3) * 2.0 ** 125
        wt[i, ::9] *= 0
    return (wt.reshape(-1) * torch.where(torch.rand(k, generator=g) < 0.5, -1.0, 1.0)).bfloat16()


@pytest.mark.parametrize("rows,k", [(1, 128), (5, 128), (333, 128), (3, 256), (41, 512), (600, 1024), (3, 2048), (400, 2048),
                                    (7, 8192), (2, 16384), (320, 16384)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("residual", [False, True])
def test_codes_are_the_quantizers(w, rows, k, fmt, residual):
    for seed in range(8 if k < 1024 else 1):
        sign = torch.where(torch.rand(rows, k, generator=torch.Generator().manual_seed(seed)) < 0.5, -1.0, 1.0)
        wt = weights(k, seed).cuda()
        x = (sign if residual else 2 * sign).bfloat16().cuda()
        codes, scales, _, y, rstd = w.fp8q_rmsnorm_quantize(x, wt, 0.0, fmt, residual=x if residual else None,
                                                            want_bf16=True, want_rstd=True)
        want = sign.cuda() * wt.float()
        assert torch.equal(rstd, torch.full_like(rstd, 0.5))
        assert torch.equal(y.view(torch.int16), want.bfloat16().view(torch.int16))
        ec, es = w.fp8q_quantize_blockwise(want.bfloat16(), fmt)
        assert torch.equal(scales.reshape(-1).view(torch.int32), es.view(torch.int32))
        assert torch.equal(codes.reshape(-1), ec)


@pytest.mark.parametrize("rows,k", [(1, 128), (333, 128), (3, 256), (41, 512), (600, 1024), (3, 2048), (400, 2048), (2, 16384)])
@pytest.mark.parametrize("residual", [False, True])
def test_mxfp8_codes_are_the_weight_quantizers(w, rows, k, residual):
    """The same rows with an MXFP8 output, against mxfp8_quantize_swizzled of y."""
    for seed in range(8 if k < 1024 else 1):
        sign = torch.where(torch.rand(rows, k, generator=torch.Generator().manual_seed(seed)) < 0.5, -1.0, 1.0)
        wt = weights(k, seed).cuda()
        x = (sign if residual else 2 * sign).bfloat16().cuda()
        ec, es = w.mxfp8_quantize_swizzled((sign.cuda() * wt.float()).bfloat16())
        codes, scales, *_ = w.mxfp8_rmsnorm_quantize(x, wt, 0.0, residual=x if residual else None, swizzled=True)
        assert torch.equal(codes, ec) and torch.equal(scales, es)
        codes, scales, *_ = w.mxfp8_rmsnorm_quantize(x, wt, 0.0, residual=x if residual else None)
        assert torch.equal(codes, ec) and torch.equal(scales, w.mxfp8_unswizzle_scales(es, 1, rows, k)[0])


@pytest.mark.parametrize("rows,k", [(3, 128), (5, 512), (2, 2048), (400, 2048)])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_infinite_weight(w, rows, k, fmt):
    """An infinite y makes its block's scale and codes NaN; the other blocks are as they are without it."""
    sign = torch.where(torch.rand(rows, k, generator=torch.Generator().manual_seed(1)) < 0.5, -2.0, 2.0).bfloat16().cuda()
    wt = torch.randn(k, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    bad = wt.clone()
    bad[k - 5] = float("inf")
    good_c, good_s, *_ = w.fp8q_rmsnorm_quantize(sign, wt, 0.0, fmt)
    codes, scales, *_ = w.fp8q_rmsnorm_quantize(sign, bad, 0.0, fmt)
    assert torch.equal(codes[:, :k - 128], good_c[:, :k - 128]) and torch.equal(scales[:, :-1], good_s[:, :-1])
    assert scales[:, -1].isnan().all()
    dtype = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    assert codes[:, k - 128:].view(dtype).float().isnan().all()


@pytest.mark.parametrize("rows,k", [(3, 128), (5, 512), (2, 2048), (400, 2048)])
def test_infinite_weight_mxfp8(w, rows, k):
    """An infinite y is the largest code under the largest scale; the other blocks are as they are without it."""
    sign = torch.where(torch.rand(rows, k, generator=torch.Generator().manual_seed(1)) < 0.5, -2.0, 2.0).bfloat16().cuda()
    wt = torch.randn(k, generator=torch.Generator().manual_seed(2)).bfloat16().cuda()
    bad = wt.clone()
    bad[k - 5] = float("inf")
    good_c, good_s, *_ = w.mxfp8_rmsnorm_quantize(sign, wt, 0.0)
    codes, scales, *_ = w.mxfp8_rmsnorm_quantize(sign, bad, 0.0)
    assert torch.equal(codes[:, :k - 32], good_c[:, :k - 32]) and torch.equal(scales[:, :-1], good_s[:, :-1])
    assert (scales[:, -1] == 247).all()
    top = codes[:, k - 5].view(torch.float8_e4m3fn).float()
    assert torch.equal(top, 448 * sign[:, k - 5].float().sign())
    rest = torch.cat([codes[:, k - 32:k - 5], codes[:, k - 4:]], 1).view(torch.float8_e4m3fn).float()
    assert (rest == 0).all()
