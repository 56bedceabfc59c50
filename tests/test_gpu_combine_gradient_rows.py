"""The combine's gradient element by element where a warp takes several short choices, the last of them fewer, with
dropped choices among them, and with guards around both outputs.  Bounds as in the routing's other tests."""
import pytest
import torch

from expert_block_ref import check_bf16
from gpu_util import Guarded
from test_gpu_moe_route import CASES, FEW, SHORT, routed

pytestmark = pytest.mark.gpu

# k <= 256: four choices a warp, k <= 512: two; here with remainders of one to three
MORE = [(9, 1, 2, 8, "drop"), (7, 3, 4, 256, "drop"), (5, 5, 8, 248, "any"), (3, 2, 3, 264, "drop"), (11, 7, 6, 512, "drop"),
        (2, 1, 2, 520, "any")]


@pytest.fixture(scope="module")
def w():
    import weight_transfer_gb300 as m
    return m


@pytest.mark.parametrize("tokens,topk,experts,k,how", CASES + FEW + SHORT + MORE)
def test_combine_gradient(w, tokens, topk, experts, k, how):
    ids, off, order, slots, n = routed(w, tokens, topk, experts, how)
    y = torch.randn(tokens * topk, k, device="cuda").bfloat16()
    y[n:] = float("nan")                                # rows of dropped choices are never looked at
    dout = torch.randn(tokens, k, device="cuda").bfloat16()
    wt = torch.randn(tokens, topk, device="cuda")
    dy, dw = Guarded(tokens * topk * k, torch.bfloat16), Guarded(tokens * topk, torch.float32)
    w.fp8q_moe_combine_backward(dout, y, slots, off, wt, dy=dy.t, dweights=dw.t)
    assert dy.intact() and dw.intact()
    sl = slots.cpu().long()
    live = sl < n
    d64 = dout.double().cpu()
    want = torch.zeros(tokens * topk, k, dtype=torch.float64)
    want[sl.reshape(-1)] = torch.where(live[..., None], d64[:, None] * wt.double().cpu()[..., None], 0.0).reshape(-1, k)
    check_bf16(dy.t.view(-1, k), want, 2.0 ** -24)
    assert (dy.t.view(-1, k)[n:] == 0).all()
    terms = torch.where(live[..., None], d64[:, None] * y.double().cpu()[sl], 0.0)
    err = (dw.t.view(tokens, topk).double().cpu() - terms.sum(-1)).abs()
    assert (err <= (k / 32 + 6) * 2.0 ** -24 * terms.abs().sum(-1)).all()
    assert (dw.t.view(tokens, topk).cpu()[~live] == 0).all()
