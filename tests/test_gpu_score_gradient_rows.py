"""The scores' gradient on both sides of every limit of rows and of their bytes at which a row goes to a warp, to a block
or to several."""
import pytest
import torch

from test_gpu_token_logprobs import TYPES, check_gradient, logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("per_sm,more", [(8, -1), (8, 0), (12, -1), (12, 0)])
@pytest.mark.parametrize("size", [4096, 4104, 6000, 6008])
def test_rows_around_the_limits(size, per_sm, more, dtype):
    rows = per_sm * torch.cuda.get_device_properties(0).multi_processor_count + more
    dt = TYPES[dtype]
    x, t = logits(rows, size // dt.itemsize, dt, seed=size + rows)
    t[3] = -1
    check_gradient(x, t)
    check_gradient(x, t, 0.7, bonus=False, in_place=True)
