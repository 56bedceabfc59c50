"""The gradient norm's time does not depend on how large the gradients are, and its sums keep every magnitude: rows that
hardly anything reached (root mean squares of 1e-13 and less) are ordinary in an output head and in the experts."""
import math

import pytest
import torch

import weight_transfer_gb300 as w
from test_gpu_grad_norm import KINDS, U, check_norm, squares

pytestmark = pytest.mark.gpu


def time_of(tensors, calls=20):
    held = w.fp8q_grad_list(tensors)
    graph = torch.cuda.CUDAGraph()
    w.fp8q_grad_norm(held)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        for _ in range(calls):
            w.fp8q_grad_norm(held)
    best = math.inf
    for _ in range(6):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("kind", KINDS)
def test_the_time_does_not_depend_on_the_magnitude(kind):
    """With binary64 squares of what binary32 cannot hold the same tensor took 9 to 15 times as long; two readings of
    the stage in shared memory instead of one take less than twice as long."""
    x = torch.randn(32 << 20, device="cuda")
    ordinary = time_of([(x * 1e-3).to(kind)])
    for size in (0.0, 1e-20, 1e-14, 1e17, 1e25):
        assert time_of([(x * size).to(kind)]) < 2 * ordinary, size


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", [2.0 ** -133, 2.0 ** -127, 2.0 ** -75, 2.0 ** -52, 2.0 ** -47, 2.0 ** -46, 2.0 ** -40, 2.0 ** 44, 2.0 ** 45,
                                  2.0 ** 49, 2.0 ** 50, 2.0 ** 51, 2.0 ** 126])
def test_sums_around_the_limits(size, kind):
    """Equal gradients whose sums of 64, 2048 and all squares lie around 2^-80 and 2^100, alone and beside smaller and
    larger ones in the same lane, in the same warp and elsewhere."""
    n = 70000
    x = torch.full((n,), size, dtype=kind, device="cuda")
    y = x.clone()
    y[::2] = 0
    y[1::16] *= 2.0 ** -3
    z = torch.zeros_like(x)
    z[12345] = size
    r = torch.randn(n, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)) * min(size, 1e37)
    r[:5000] *= 2.0 ** -11
    r[40000:] *= 2.0 ** -30
    for t in (x, y, z, r.to(kind)):
        norm, each = w.fp8q_grad_norm([t, t[:3], t[777:]], want_each=True)
        check_norm(norm, each, [t, t[:3], t[777:]], math.inf, 1.0)


@pytest.mark.parametrize("kind", KINDS)
def test_one_large_or_not_finite_value_among_tiny_ones(kind):
    for at in (0, 1, 8, 16383, 16384, 30000):
        x = torch.full((30001,), 2.0 ** -60, dtype=kind, device="cuda")
        x[at] = 2.0 ** 120
        norm, _ = w.fp8q_grad_norm([x])
        assert abs(float(norm[0]) - 2.0 ** 120) <= 10 * U * 2.0 ** 120
        for value in (math.inf, -math.inf):
            x[at] = value
            assert float(w.fp8q_grad_norm([x])[0][0]) == math.inf
        x[at] = math.nan
        assert math.isnan(float(w.fp8q_grad_norm([x])[0][0]))
    assert float(squares([torch.zeros(4, device="cuda")])[0]) == 0.0
