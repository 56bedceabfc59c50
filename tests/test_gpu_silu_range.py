"""The gated activation over the range of its gate, on sums that are exact.

A row of codes with a single 1 picks one column of the weights, so that g and u are the weights' own values.  Error of
g / (1 + exp(-g)) * u as the product's epilogue forms it, relative to the value, with s = exp(-g) / (1 + exp(-g)) <= 1:
  * exp(-g) as 2^(g * -log2(e)): the rounding of the product is 2^-24 of the exponent, |g| * 2^-24 of the power; the
    constant is off by 2^-26.1 of itself, |g| * 2^-26.1; the power's own 2 ulp are 2^-22;
  * the sum 2^-24, the reciprocal's ulp 2^-23 (where it is subnormal, below g = -87.3, 2^-149 * (1 + exp(-g)));
  * two products, 2^-23 together.
Below g = -88.72 exp(-g) passes the binary32 range and the result is -0."""
import math

import pytest
import torch

from expert_block_ref import check_mx
from test_gpu_moe_product import swizzle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    import weight_transfer_gb300 as m
    return m


def silu_tolerance(g, subnormal=False):
    tol = g * (2.0 ** -24 + 2.0 ** -26.1) + 2.0 ** -22 + 2.0 ** -24 + 2.0 ** -23 + 2.0 ** -23
    return (tol + (2.0 ** -149 * (1 + math.exp(g)) if subnormal else 0)) * (1 + 2.0 ** -10)


def check(g, u, codes, scales, tol):
    check_mx(g / (1 + torch.exp(-g)) * u, codes, scales.cpu().long(), tol)


# e4m3 values of one power of two, the exponent of u's scale (so that the values stay in the normal range)
RANGES = [("near 0", [s * m / 64 for m in range(8, 16) for s in (1, -1)], 0), ("2", [s * m / 4 for m in range(8, 16) for s in (1, -1)], 0),
          ("20", [20.0, 18.0, 22.0, 24.0], 0), ("-20", [-20.0, -18.0, -22.0, -24.0], 20), ("60", [60.0, 56.0, 48.0], 0),
          ("-60", [-60.0, -56.0, -52.0], 70), ("-88", [-88.0, -80.0, -72.0], 90), ("200", [208.0, 192.0, 224.0], 0)]


@pytest.mark.parametrize("name,values,up", RANGES)
@pytest.mark.parametrize("rows,experts", [(20, 1), (130, 1), (300, 2)])
def test_range(w, name, values, up, rows, experts):
    n, k = 256, 64
    g = torch.Generator().manual_seed(len(values) + rows)
    gate, upw = torch.zeros(experts, n, k), torch.zeros(experts, n, k)
    pick = torch.randint(0, len(values), (experts, n, k), generator=g)
    gate = torch.tensor(values)[pick]
    # blocks of 32 features get one gate value per row, so that no value of a block is far below another
    gate = gate[:, ::32].repeat_interleave(32, 1)
    upw = torch.randint(8, 16, (experts, n, k), generator=g).float() * torch.where(torch.rand(experts, n, k, generator=g) < 0.5, -1.0, 1.0)
    assert torch.equal(gate.to(torch.float8_e4m3fn).float(), gate)
    col = torch.randint(0, k, (rows,), generator=g)
    a = torch.zeros(rows, k)
    a[torch.arange(rows), col] = 1.0
    codes = lambda t: t.to(torch.float8_e4m3fn).view(torch.uint8).cuda()  # noqa: E731
    one = lambda *s: torch.full(s, 127, dtype=torch.uint8)  # noqa: E731
    off = torch.tensor([0, rows] if experts == 1 else [0, rows // 3, rows], dtype=torch.int32)
    e_of = torch.zeros(rows, dtype=torch.long) if experts == 1 else (torch.arange(rows) >= rows // 3).long()
    got, scales = w.mxfp8_moe_swiglu(codes(a), one(rows, k // 32).cuda(), codes(gate), swizzle(one(experts, n, k // 32)).cuda(),
                                     codes(upw), swizzle(one(experts, n, k // 32) + up).cuda(), off.cuda())
    g64, u64 = gate[e_of, :, col].double(), upw[e_of, :, col].double() * 2.0 ** up
    check(g64, u64, got, scales, silu_tolerance(max(abs(v) for v in values), min(values) < -87.3))


@pytest.mark.parametrize("value", [-96.0, -208.0, -448.0])
def test_below_the_range(w, value):
    """exp(-g) infinite: zeros under the smallest scale."""
    rows, n, k = 20, 64, 32
    one = lambda *s: torch.full(s, 0x38, dtype=torch.uint8)  # noqa: E731
    gate = torch.full((1, n, k), value / 32).to(torch.float8_e4m3fn).view(torch.uint8)
    e = lambda *s: torch.full(s, 127, dtype=torch.uint8)  # noqa: E731
    codes, scales = w.mxfp8_moe_swiglu(one(rows, k).cuda(), e(rows, 1).cuda(), gate.cuda(), swizzle(e(1, n, 1)).cuda(), one(1, n, k).cuda(),
                                       swizzle(e(1, n, 1)).cuda(), torch.tensor([0, rows], dtype=torch.int32).cuda())
    assert ((codes & 0x7F) == 0).all() and (scales == 0).all()
