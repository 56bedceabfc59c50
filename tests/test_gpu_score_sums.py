"""The scores' sums: a row's error does not grow with its length.

Tolerances.  A thread adds its terms in four chains, of which each takes a quarter of its 16-byte vectors' elements and
at most 256 terms before they go to sums that keep what an addition rounds off: n terms are n roundings of 2^-24.  The
chains' joins, the thread's correction of its reference, and the joins of lanes, warps and blocks, and of the reference
with the largest logit, are 16 additions and 6 factors, each an exponential of 2^-22 and two roundings more: 16 + 6 * 6,
taken as 56.  Every term has its own exponential's 2^-22 and the roundings of its argument, at most 3 |z|.  So log S is
within 2^-24 (n + 60 + 3 E|z| + 3 |log S|), and the entropy within 2^-24 ((n + 60) (1 + E|z|) + 8 E z^2 + 4 |log S|)."""
import math

import pytest
import torch

import weight_transfer_gb300 as w
from test_gpu_token_logprobs import TYPES, U, close, formula, logits

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def chain(rows, vocab, size):
    """Terms that a chain of a thread takes one after another, by the least number of threads that may share a row."""
    if rows >= 8 * sms() and vocab * size <= 49152:
        threads = 32
    elif vocab * size <= 16384:
        threads = 128
    else:                                                     # blocks of a cluster share a row of few: doubled while they fit
        ranks = 1
        slots = 4 * sms()
        steps = -(-vocab * size // 16384)
        while ranks < 8 and rows * ranks * 2 <= (slots - slots // 16 if ranks > 1 else slots) and ranks * 2 <= steps:
            ranks *= 2
        threads = 256 * ranks
    vectors = math.ceil(vocab * size / 16 / threads)
    # whole steps of four vectors, as a block's share need not be a multiple of them
    return min(256, 4 * math.ceil(vectors / 4) * (16 // size) // 4)


def tight(x, T=1.0, top=0):
    rows, vocab = x.shape
    t = torch.zeros(rows, dtype=torch.int64, device="cuda")
    lp, H, _, _, st = w.fp8q_token_logprobs(x, t, T, top, want_entropy=True, want_stats=True)
    n = chain(rows, vocab, x.dtype.itemsize) + 60
    for a in range(0, rows, 64):                              # the formula holds several 64-bit copies of its rows
        f = formula(x[a:a + 64], t[a:a + 64], float(torch.tensor(T, dtype=torch.float32)))
        tol = U * (n + 3 * f["ez"] + 3 * f["log_s"].abs())
        b = slice(a, a + 64)
        close(st[b, 0], f["m"], 0.0, "largest")
        close(st[b, 1], f["log_s"], tol, "log S")
        close(lp[b], f["at"], tol + 6 * U * f["at"].abs().nan_to_num(posinf=0.0), "score")
        close(H[b], f["H"], U * (n * (1 + f["ez"]) + 8 * f["ez2"] + 4 * f["log_s"].abs()), "entropy")


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,vocab", [(1, 151936), (700, 151936), (2, 50257), (320, 40001), (1300, 8000), (1, 262144 * 8 + 16), (1, 3_000_001),
                                        (310, 300_007), (1, 16_000_003)])
def test_equal_terms(rows, vocab, dtype):
    """Terms that are rounded the same way every time: every second logit lies a little below the others."""
    x = torch.zeros(rows, vocab, dtype=TYPES[dtype], device="cuda")
    for off in (0.3, 1.1, 2.5):
        x[:, ::2] = off
        tight(x)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_a_row_of_200_million(dtype):
    """Equal terms again, from the closed form: h logits of `off` and as many of 0."""
    h = 100_000_000
    x = torch.zeros(1, 2 * h, dtype=TYPES[dtype], device="cuda")
    for off in (0.3, 1.1):
        x[:, ::2] = off
        z = -float(x[0, 0])
        S = h * (1 + math.exp(z))
        p = math.exp(z) / (1 + math.exp(z))
        _, H, _, _, st = w.fp8q_token_logprobs(x, want_entropy=True, want_stats=True)
        assert abs(st[0, 1].item() - math.log(S)) <= U * (256 + 60 + 3 * -z * p + 3 * math.log(S))
        assert abs(H.item() - (math.log(S) - p * z)) <= U * (316 * (1 - z * p) + 8 * z * z * p + 4 * math.log(S))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,vocab", [(3, 151936), (310, 131075), (1300, 12000), (2, 4_000_037)])
def test_random_rows(rows, vocab, dtype):
    x, _ = logits(rows, vocab, TYPES[dtype], seed=vocab)
    tight(x)
    tight(x, 0.7, top=8)
    x[0] = x[0].sort().values                                 # the reference is raised again and again
    x[1] = x[1].sort(descending=True).values
    x[1, vocab // 2:] = -math.inf
    tight(x)
