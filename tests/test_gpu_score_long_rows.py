"""Rows so long that a thread's sums go on in shared memory: masks, extremes, temperatures and orders on them, in the
forms with and without alternatives and entropy, captured and on another stream."""
import math

import pytest
import torch

import weight_transfer_gb300 as w
from test_gpu_score_sums import tight
from test_gpu_token_logprobs import LOWEST, TYPES, check, logits

pytestmark = pytest.mark.gpu
LONG = 3_000_011                                              # beyond 262,144 logits for each of eight blocks


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_masks(dtype):
    dt = TYPES[dtype]
    x, t = logits(7, LONG, dt, seed=1)
    x[0] = -math.inf
    x[1] = LOWEST[dt]
    x[2, :LONG // 2] = LOWEST[dt]                             # sums of 2^19 terms, then far larger logits
    x[3, LONG // 2:] = -math.inf
    x[4] = -math.inf; x[4, LONG - 1] = 2.0                    # noqa: E702
    x[5, : LONG - 9] = -math.inf
    x[6, ::2] = torch.finfo(dt).max
    t[4] = LONG - 1
    for T in (1.0, 0.6):
        check(x, t, T, 20)
        check(x, t, T, 0, entropy=False)
        check(x, t, T, 3, entropy=False, stats=False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [2.0 ** -20, 0.01, 0.5, 40.0, 2.0 ** 20])
def test_temperatures(T, dtype):
    x, _ = logits(2, LONG, TYPES[dtype], seed=2)
    x[1] *= 1e-3
    tight(x, T)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_rising_and_falling_logits(dtype):
    """The reference is raised over the whole row, or never again after its start."""
    i = torch.arange(LONG, device="cuda", dtype=torch.float32) / LONG
    x = torch.stack([60 * i - 30, 30 - 60 * i, (20 * i).floor(), 10 * torch.sin(300 * i)]).to(TYPES[dtype])
    tight(x)
    tight(x, 0.3, top=5)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_a_nan_or_an_infinity_shows(value, dtype):
    for at in (0, 9, LONG // 8, LONG // 3, LONG - 1):
        x, t = logits(2, LONG, TYPES[dtype], seed=3)
        clean = w.fp8q_token_logprobs(x.clone(), t, top=2, want_entropy=True, want_stats=True)
        x[1, at] = value
        got = w.fp8q_token_logprobs(x, t, top=2, want_entropy=True, want_stats=True)
        assert all(torch.equal(a[0], b[0]) for a, b in zip(got, clean))
        assert got[0][1].isnan() and got[1][1].isnan() and got[2][1].isnan().all() and got[4][1, 1].isnan()
        if value == math.inf:
            assert got[3][1, 0] == at and got[4][1, 0] == math.inf


def test_many_long_rows_captured_and_on_another_stream():
    x, t = logits(310, 530_001, torch.bfloat16, seed=4)
    want = w.fp8q_token_logprobs(x, t, top=6, want_entropy=True, want_stats=True)
    tight(x[:64].clone(), top=6)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = w.fp8q_token_logprobs(x, t, top=6, want_entropy=True, want_stats=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = w.fp8q_token_logprobs(x, t, top=6, want_entropy=True, want_stats=True)
    for _ in range(2):
        for o in out:
            o.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
