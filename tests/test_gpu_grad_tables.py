"""A tensor's norm is the same bits in whatever list it stands: short ones and long ones go through other tables and
kernels, and more than 1024 tensors through several of them."""
import pytest
import torch

import weight_transfer_gb300 as w
from test_gpu_grad_norm import KINDS, views

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
def test_the_same_bits_in_any_table(kind):
    sizes = [50001, 1, 16384, 0, 33, 100003, 7, 8192] * 5
    g, _ = views(sizes, [kind] * len(sizes), seed=4, gap=1)
    others, _ = views([11 + i % 5 for i in range(2100)], [KINDS[i % 2] for i in range(2100)], seed=5)
    want = w.fp8q_grad_norm(g, want_each=True)[1]
    for before, after in ((0, 1), (30, 0), (3, 22), (700, 700), (1000, 1), (1020, 300), (2100, 0)):
        each = w.fp8q_grad_norm(others[:before] + g + others[2100 - after:], want_each=True)[1]
        assert torch.equal(each[before:before + len(g)], want), (before, after)


def test_the_clipped_gradients_are_the_same_bits_in_any_table():
    """With a limit that nothing reaches the factor is the scale's, whatever else is in the list."""
    sizes = [50001, 1, 16384, 33, 100003]
    g, _ = views(sizes, KINDS * 2 + KINDS[:1], seed=6, gap=1)
    others, _ = views([9] * 1500, KINDS[:1] * 1500, seed=7)
    want = [torch.empty(n, dtype=torch.bfloat16, device="cuda") for n in sizes]
    w.fp8q_grad_clip(g, 1e30, 1 / 3, outs=want)
    for before in (0, 60, 1022, 1500):
        outs = [torch.empty(n, dtype=torch.bfloat16, device="cuda") for n in sizes]
        rest = [torch.empty(9, dtype=torch.float32, device="cuda") for _ in range(before)]
        w.fp8q_grad_clip(others[:before] + g, 1e30, 1 / 3, outs=rest + outs)
        assert all(torch.equal(a, b) for a, b in zip(outs, want)), before
