"""A list of gradients goes on with the tensors that it was made of: where they have been replaced it can be asked, and
the example's trainer refuses to send the old ones."""
import os
import sys

import pytest
import torch

import weight_transfer_gb300 as w
from conftest import ROOT

sys.path.insert(0, os.path.join(ROOT, "examples"))
import policy_step  # noqa: E402

pytestmark = pytest.mark.gpu


def test_holds():
    a, b, e = (torch.ones(n, device="cuda", dtype=t) for n, t in ((10, torch.float32), (7, torch.bfloat16), (0, torch.float32)))
    held = w.fp8q_grad_list([a, b, e])
    assert held.holds([a, b, e]) and held.holds(iter([a, b, e])) and held.holds([a.view(2, 5), b, e])
    assert not held.holds([a, b]) and not held.holds([a, b, e, e]) and not held.holds([b, a, e])
    assert not held.holds([a.clone(), b, e]) and not held.holds([None, b, e]) and not held.holds([a[:9], b, e])
    assert not held.holds([a, b.view(torch.int16), e])
    assert w.fp8q_grad_list([]).holds([])
    a.data = a.data.clone()                                  # the same tensor, in other memory
    assert not held.holds([a, b, e])


def step(params, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    sum((p * torch.randn(p.shape, generator=g, device="cuda", dtype=p.dtype)).sum() for p in params).backward()


def test_a_trainer_whose_gradients_were_replaced_does_not_send_the_old_ones():
    params = [torch.nn.Parameter(torch.zeros(n, device="cuda")) for n in (300, 7)]
    optimizer = torch.optim.SGD(params, lr=0.1)
    trainer = policy_step.Trainer(params, ranks=1, max_norm=1e9)
    for seed, clear in enumerate((trainer.zero_grad, lambda: optimizer.zero_grad(set_to_none=False))):
        clear()
        step(params, seed)
        trainer.send()
        for p, c in zip(params, trainer.clipped):
            assert torch.equal(c, p.grad.bfloat16()) and p.grad.any()
    optimizer.zero_grad()                                    # to None
    with pytest.raises(RuntimeError, match="replaced"):
        trainer.send()
    step(params, 5)
    with pytest.raises(RuntimeError, match="replaced"):
        trainer.send()
