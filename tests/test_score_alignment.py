"""The scores' arrays per row as parts of longer ones: what the calls with FP8Q_ELEMENT_ALIGNED take and refuse (without
a GPU), and their results (on one)."""
import pytest
import torch

from conftest import build_lib
from test_abi import A, ERR_ALIAS, ERR_ALIGN, ERR_FLAGS, ERR_NULL, MB, OK

P = [A + i * 64 * MB for i in range(12)]


@pytest.fixture(scope="module")
def L():
    build_lib()
    import weight_transfer_gb300 as w
    return w.lib()


def test_refusals(L):
    def scores(flags=2, rows=4, ids=P[1], ib=8, lp=P[2], ent=P[3], tl=P[4], ti=P[5], st=P[6]):
        return L.fp8q_token_logprobs_ex(P[0], 2, rows, 1000, 1000, ids, ib, 1.0, 5, lp, ent, tl, ti, st, flags, None)

    def gradient(flags=2, rows=4, ids=P[1], ib=8, st=P[2], g=P[3], ent=P[4], dh=P[5]):
        return L.fp8q_token_logprobs_backward_ex(P[0], 2, rows, 1000, 1000, ids, ib, 1.0, st, g, ent, dh, P[6], 1000, flags, None)
    for call, names in ((scores, ("lp", "ent", "tl", "ti", "st")), (gradient, ("st", "g", "ent", "dh"))):
        assert call(rows=0) == OK and call(rows=0, flags=0) == OK
        for flags in (1, 3, 4, 1 << 31):
            assert call(flags=flags) == ERR_FLAGS and call(flags=flags, rows=0) == ERR_FLAGS
        assert call(ids=P[9] + 4) == ERR_ALIGN and call(ids=P[9] + 2, ib=4) == ERR_ALIGN
        assert call(flags=0, ids=P[9] + 8) == ERR_ALIGN
        assert call(ids=None) == ERR_NULL
        for name in names:
            assert call(**{name: P[9] + 2}) == ERR_ALIGN and call(flags=0, **{name: P[9] + 4}) == ERR_ALIGN
    for name in ("lp", "ent", "tl", "ti", "st"):             # 4 bytes do: the next check finds it over the logits' last row
        assert scores(**{name: P[0] + 7996}) == ERR_ALIAS


def part(t, shift):
    """The same values at `shift` elements from the start of a longer array."""
    flat = torch.zeros(t.numel() + shift + 5, dtype=t.dtype, device=t.device)
    flat[shift:shift + t.numel()] = t.flatten()
    return flat[shift:shift + t.numel()].view(t.shape)


@pytest.mark.gpu
@pytest.mark.parametrize("shift", [1, 2, 3])
@pytest.mark.parametrize("ids", [torch.int32, torch.int64])
@pytest.mark.parametrize("rows,vocab", [(5, 3001), (1300, 500), (3, 70001)])
def test_parts_of_longer_arrays(rows, vocab, ids, shift):
    import weight_transfer_gb300 as w
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn(rows, vocab, generator=g, device="cuda")
    t = torch.randint(0, vocab, (rows,), generator=g, device="cuda").to(ids)
    up, dh = torch.randn(rows, generator=g, device="cuda"), torch.randn(rows, generator=g, device="cuda")
    for top in (0, 4):
        want = w.fp8q_token_logprobs(x, t, 0.8, top, want_entropy=True, want_stats=True)
        outs = [None if o is None else part(torch.zeros_like(o), shift) for o in want]
        got = w.fp8q_token_logprobs(x, part(t, shift), 0.8, top, False, False, *outs)
        for a, b, o in zip(got, want, outs):
            assert a is o and (a is None or torch.equal(a, b))
    _, ent, _, _, st = want
    d = w.fp8q_token_logprobs_backward(x, t, st, up, ent, dh, 0.8)
    assert torch.equal(d, w.fp8q_token_logprobs_backward(x, *(part(v, shift) for v in (t, st, up, ent, dh)), 0.8))


@pytest.mark.gpu
def test_labels_shifted_by_one_and_rows_of_the_statistics():
    """A packed sequence scored against its own next tokens, and the gradient of some of its rows."""
    import weight_transfer_gb300 as w
    x = torch.randn(9, 1000, device="cuda")
    tokens = torch.randint(0, 1000, (10,), device="cuda")
    lp, ent, _, _, st = w.fp8q_token_logprobs(x, tokens[1:], want_entropy=True, want_stats=True)
    assert torch.equal(lp, w.fp8q_token_logprobs(x, tokens[1:].clone())[0])
    up = torch.randn(9, device="cuda")
    whole = w.fp8q_token_logprobs_backward(x, tokens[1:], st, up, ent, up)
    some = w.fp8q_token_logprobs_backward(x[3:7], tokens[4:8], st[3:7], up[3:7], ent[3:7], up[3:7])
    assert torch.equal(some, whole[3:7])
