"""Gate/up and down products at every number of 16-row units that a tile can hold, in pairs of blocks, single blocks and
small tiles, and with most rows on one of many experts.  Whole numbers as in the products' other tests: the sums are
exact, so that the down product is compared bit for bit and the gated one within its activation's own error."""
import pytest
import torch

from test_gpu_moe_product import groups, product, swizzle, whole_mx
from test_gpu_silu_range import check, silu_tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def w():
    import weight_transfer_gb300 as m
    return m


def both(w, counts, rows, n, k):
    off, e_of = groups(counts, rows)
    ac, ae, av = whole_mx((rows, k), 21)
    gc, ge, gv = whole_mx((len(counts), n, k), 22)
    uc, ue, uv = whole_mx((len(counts), n, k), 23)
    a, b, up = (ac.cuda(), ae.cuda()), (gc.cuda(), swizzle(ge).cuda()), (uc.cuda(), swizzle(ue).cuda())
    assert torch.equal(w.mxfp8_moe_matmul(*a, *up, off).cpu(), product(av, uv, e_of).float().bfloat16())
    gv = gv * 2.0 ** -10
    gate = (b[0], swizzle(ge - 10).cuda())
    codes, scales = w.mxfp8_moe_swiglu(*a, *gate, *up, off)
    g, u = product(av, gv, e_of), product(av, uv, e_of)
    check(g, u, codes, scales, silu_tolerance(float(g.abs().max())))


@pytest.mark.parametrize("n", [128, 256, 96])
@pytest.mark.parametrize("units", range(1, 15))
def test_units_of_a_tile(w, units, n):
    """Experts of 16 u - 15, 16 u - 1 and 16 u rows beside one that raises the mean above small tiles."""
    counts = [16 * units - 15, 1000, 16 * units - 1, 16 * units]
    both(w, counts, sum(counts) + 3, n, 160)


@pytest.mark.parametrize("rows", [1, 15, 16, 17, 31, 32, 33, 48])
def test_small_tiles(w, rows):
    both(w, [rows, 0, max(rows - 1, 0)], 2 * rows, 160, 96)


@pytest.mark.parametrize("n,k", [(256, 128), (96, 160)])
def test_most_rows_on_one_expert(w, n, k):
    counts = [0] * 20 + [1500] + [3, 0, 1, 17] * 10 + [40]
    both(w, counts, sum(counts) + 5, n, k)
