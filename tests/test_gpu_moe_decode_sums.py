"""What the few-token experts' sums over a block of 32 keep.  An instruction adds 16 products to the sum so far: bits more
than 25 below the largest term are cut off, and the result to 24 bits, towards zero; a block is two of them.

One block of x holds a 2^16, a value v and a -2^16 as products with the up weights: what is left of v is what the sum
held.  The gate is 64, whose activation is 64 in binary32, and the down weights pass that feature on."""
import pytest
import torch

import weight_transfer_gb300 as w

pytestmark = pytest.mark.gpu

FIRST, SECOND = (0, 1, 2, 8, 9, 16), (4, 5, 6, 12, 13, 20)       # of a block, for the instruction that takes them


def left_of(big, small, minus, e):
    """(2^16 at `big`) + (2^e at `small`) - (2^16 at `minus`)."""
    x, up, gate, down = torch.zeros(1, 32), torch.zeros(1, 32, 32), torch.zeros(1, 32, 32), torch.zeros(1, 32, 32)
    x[0, 31], gate[0, 0, 31], down[0, 0, 0] = 8.0, 8.0, 1.0
    a = 2.0 ** max(-9, min(e, 8))
    for at, p, q in ((big, 256.0, 256.0), (small, a, 2.0 ** e / a), (minus, 256.0, -256.0)):
        x[0, at], up[0, 0, at] = p, q

    def codes(t):
        return t.to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    scales = torch.full((512,), 127, dtype=torch.uint8, device="cuda")
    one = torch.ones(1, 1, device="cuda")
    out = w.mxfp8_moe_decode(codes(x), torch.full((1, 1), 127, dtype=torch.uint8, device="cuda"), torch.zeros_like(one, dtype=torch.int32),
                             one, codes(gate), scales, codes(up), scales, codes(down), scales)
    assert not out[0, 1:].any()
    return float(out[0, 0]) / 64


@pytest.mark.parametrize("group", [FIRST, SECOND])
def test_sixteen_products_keep_25_bits_below_the_largest(group):
    for big, small, minus in ((0, 1, 2), (2, 0, 1), (3, 5, 4), (5, 3, 0)):
        for e in range(14, -10, -1):
            assert left_of(group[big], group[small], group[minus], e) == 2.0 ** e
        assert left_of(group[big], group[small], group[minus], 16 - 26) == 0.0


def test_two_steps_keep_24_bits_towards_zero():
    for a, b, c in ((0, 1, 4), (8, 0, 12), (9, 16, 20)):              # the first step leaves 2^16 + 2^e
        for e in range(14, 16 - 24, -1):
            assert left_of(a, b, c, e) == 2.0 ** e
        assert left_of(a, b, c, 16 - 24) == 0.0
    for a, b, c in ((4, 0, 1), (12, 8, 0), (20, 9, 16)):              # the first step leaves -(2^16 - 2^e)
        for e in range(14, 16 - 25, -1):
            assert left_of(a, b, c, e) == 2.0 ** e
        assert left_of(a, b, c, 16 - 25) == 2.0 ** (16 - 24)          # one step of 24 bits nearer to zero
    for a, b, c in ((0, 4, 1), (8, 12, 0), (9, 20, 16)):              # the first step leaves nothing
        for e in (14, 0, -9, -18):
            assert left_of(a, b, c, e) == 2.0 ** e


def test_far_negative_gates_give_zeros():
    """Where exp(-g) passes binary32 the activation is 0, as the header says; just above, it is the formula's."""
    def layer(g):
        x, up, gate, down = torch.zeros(1, 32), torch.zeros(1, 32, 32), torch.zeros(1, 32, 32), torch.zeros(1, 32, 32)
        x[0, 0], x[0, 1], gate[0, 0, 0], gate[0, 0, 1], up[0, 0, 0], down[0, 0, 0] = 1.0, 1.0, -88.0, g, 1.0, 1.0

        def codes(t):
            return t.to(torch.float8_e4m3fn).view(torch.uint8).cuda()
        scales = torch.full((512,), 127, dtype=torch.uint8, device="cuda")
        high = torch.full((512,), 127 + 120, dtype=torch.uint8, device="cuda")
        one = torch.ones(1, 1, device="cuda")
        return float(w.mxfp8_moe_decode(codes(x), torch.full((1, 1), 127, dtype=torch.uint8, device="cuda"),
                                        torch.zeros_like(one, dtype=torch.int64), one, codes(gate), scales, codes(up), high, codes(down),
                                        scales)[0, 0])
    want = -88.5 / (1 + 2.718281828459045 ** 88.5) * 2.0 ** 120
    assert abs(layer(-0.5) - want) <= abs(want) * (2.0 ** -8 + 8 * 2.0 ** -24)        # bf16's; expf's two units, two roundings
    assert layer(-0.75) == 0.0
