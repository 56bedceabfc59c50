"""What the products' accumulators keep: 24 significant bits, each step of 32 products cut off towards zero.

The first block of 32 gives 2^m, the second v, the third takes 2^m away again: what is left of v is what the sum held."""
import pytest
import torch

from test_gpu_moe_product import swizzle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    import weight_transfer_gb300 as m
    return m


def left_of(w, m, v, sign, counts):
    rows, n, k = sum(counts), 160, 96
    a, e = torch.zeros(k), torch.full((3,), 127)
    a[0], a[32], a[64] = sign, v, -sign
    e[0] = e[2] = 127 + m
    codes = a.to(torch.float8_e4m3fn).view(torch.uint8).repeat(rows, 1)
    one = torch.ones(len(counts), n, k).to(torch.float8_e4m3fn).view(torch.uint8)
    off = torch.tensor([0] + list(counts)).cumsum(0).to(torch.int32)
    out = w.mxfp8_moe_matmul(codes.cuda(), e.to(torch.uint8).repeat(rows, 1).cuda(), one.cuda(),
                             swizzle(torch.full((len(counts), n, 3), 127, dtype=torch.uint8)).cuda(), off.cuda())
    assert (out == out[0, 0]).all()
    return float(out[0, 0])


@pytest.mark.parametrize("counts", [[1], [40, 3], [100, 80]])       # small tiles, and larger ones
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_accumulators_hold_24_bits(w, counts, sign):
    for m in range(2, 24):
        for v in (1.0, -1.0):                                       # 2^m + v has at most 24 bits
            assert left_of(w, m, v, sign, counts) == v
    for m in range(2, 23):
        assert left_of(w, m, 1.5 * sign, sign, counts) == 1.5 * sign
    assert left_of(w, 23, 1.5 * sign, sign, counts) == sign         # towards zero: 2^23 + 1.5 -> 2^23 + 1
    assert left_of(w, 24, sign, sign, counts) == 0.0
