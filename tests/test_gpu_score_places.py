"""Every logit counts in the scores, wherever it lies: at a row's ends, around its vectors and steps, and at the
boundaries of the blocks that share it.

Tolerances.  With one or two large logits among far smaller ones, or logits of 0 alone, no sum is rounded: what is left
are the joins, up to six factors each of an exponential of 0 (exact), and the logarithm's last place."""
import math

import pytest
import torch

import weight_transfer_gb300 as w
from test_gpu_score_sums import sms
from test_gpu_token_logprobs import TYPES, U, close, logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows", [1, 2, 40, 76, 160, 320, 1300])
@pytest.mark.parametrize("vocab", [257, 4099, 12001, 50257, 151936])
def test_the_number_of_live_logits(vocab, rows, dtype):
    """Logits of 0 and masked ones: S is a whole number, summed without a rounding, so that one lost or counted twice shows."""
    x = torch.zeros(rows, vocab, dtype=TYPES[dtype], device="cuda")
    live = torch.full((rows,), vocab, dtype=torch.float64, device="cuda")
    for r in range(rows):
        if r % 3 == 1:
            x[r, r % vocab] = -math.inf
            live[r] -= 1
        elif r % 3 == 2:
            x[r, vocab // 2:] = -math.inf
            live[r] = vocab // 2
    st = w.fp8q_token_logprobs(x, want_stats=True)[4]
    ent = w.fp8q_token_logprobs(x, want_entropy=True)[1]
    want = torch.log(live)
    # the logarithm's own error is a unit in its last place
    close(st[:, 1], want, 2 * U * want.abs() + U, "log S")
    close(ent, want, 2 * U * want.abs() + U, "entropy")
    assert vocab > 100_000 or math.log(vocab) - math.log(vocab - 1) > 4 * U * math.log(vocab)


def places(vocab, size, offset):
    """Where a logit could get lost: around a row's ends, vectors, steps, and the boundaries of 1, 2, 4 and 8 blocks."""
    per = 16 // size
    head = -offset % per
    vecs = (vocab - head) // per
    at = {0, 1, head, head + per, head + (vecs - 1) * per, head + vecs * per, vocab - 1, vocab - 2}
    for ranks in (1, 2, 4, 8):
        for r in range(ranks + 1):
            v = vecs * r // ranks
            at |= {head + per * (v + d) + e for d in (-1, 0) for e in (0, per - 1)}
            for step in (32 * 4, 128 * 4, 256 * 4):
                at |= {head + per * (v + step + d) for d in (-1, 0)}
    return sorted(p for p in at if 0 <= p < vocab)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab,offset", [(40, 0), (1000, 3), (12001, 1), (40001, 0), (151936, 5), (600_011, 1)])
def test_one_of_two_large_logits_anywhere(vocab, offset, dtype):
    """S = 2 with both and 1 without either; in calls of one row, of one block a row and of one warp a row."""
    dt = TYPES[dtype]
    at = places(vocab, dt.itemsize, offset)

    def check(rows, spots):
        stride = vocab + -vocab % (16 // dt.itemsize)         # every row lies alike
        flat = torch.full((rows * stride + offset,), -40.0, dtype=dt, device="cuda")
        x = flat[offset:].as_strided((rows, vocab), (stride, 1))
        for r, p in enumerate(spots):
            x[r, p] = 1.0
            x[r, vocab // 3 if p != vocab // 3 else vocab // 3 + 1] = 1.0
        for top in (0, 2):
            lp, ent, tl, ti, st = w.fp8q_token_logprobs(x, torch.tensor(spots, device="cuda"), 1.0, top, want_entropy=True,
                                                        want_stats=True)
            for got, want in ((st[:, 0], 1.0), (st[:, 1], math.log(2)), (ent, math.log(2)), (lp, -math.log(2))):
                assert ((got.double() - want).abs() <= 16 * U).all(), (top, [spots[i] for i in ((got.double() - want).abs() > 16 * U).nonzero()[:4, 0].tolist()])
            if top:
                other = torch.tensor([vocab // 3 if p != vocab // 3 else vocab // 3 + 1 for p in spots], device="cuda")
                mine = torch.tensor(spots, device="cuda")
                assert torch.equal(ti.long(), torch.stack([torch.minimum(mine, other), torch.maximum(mine, other)], 1))
                assert ((tl.double() + math.log(2)).abs() <= 16 * U).all()
    for p in at:
        check(1, [p])
    few = (at * 320)[:160]
    check(160, few)
    check(320, (at * 320)[:320])
    if vocab * dt.itemsize <= 49152:
        check(8 * sms() + 1, (at * 2000)[:8 * sms() + 1])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("vocab", [5, 1000, 12001, 151936])
def test_a_nan_or_an_infinity_anywhere_shows(vocab, dtype):
    dt = TYPES[dtype]
    at = places(vocab, dt.itemsize, 0)
    for rows in (len(at), 8 * sms() + 3) if vocab < 13000 else (len(at),):
        for value in (math.nan, math.inf):
            x, t = logits(rows, vocab, dt, seed=vocab)
            t[:] = torch.arange(rows, device="cuda") % vocab
            clean = w.fp8q_token_logprobs(x.clone(), t, want_entropy=True, want_stats=True)
            bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
            for r, p in enumerate(at):
                x[r, p] = value
                bad[r] = True
            lp, ent, _, _, st = w.fp8q_token_logprobs(x, t, want_entropy=True, want_stats=True)
            assert lp[bad].isnan().all() and ent[bad].isnan().all() and st[bad, 1].isnan().all()
            if value == math.inf:
                assert (st[bad, 0] == math.inf).all()
            for a, b in zip((lp, ent, st), (clean[0], clean[1], clean[4])):
                assert torch.equal(a[~bad], b[~bad])
