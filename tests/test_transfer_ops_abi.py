"""Refusals of the scores of given tokens, the gradient norm and the expert
layer for a few tokens: every bad argument is answered with its status before
anything is launched (fake addresses are never dereferenced)."""
import ctypes

import pytest
import torch

from conftest import build_lib
from test_abi import A, ERR_ALIAS, ERR_ALIGN, ERR_FORMAT, ERR_K, ERR_NULL, ERR_SIZE, MB, OK

P = [A + i * 64 * MB for i in range(20)]
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    build_lib()
    import weight_transfer_gb300 as w
    return w.lib()


def test_token_logprobs(L):
    def call(x=P[0], b=2, rows=4, vocab=1000, stride=1000, ids=P[1], ib=8, t=1.0, top=5, lp=P[2], ent=P[3], tl=P[4], ti=P[5],
             st=P[6]):
        return L.fp8q_token_logprobs(x, b, rows, vocab, stride, ids, ib, t, top, lp, ent, tl, ti, st, None)
    assert call(rows=0) == OK
    assert call(b=1) == ERR_FORMAT and call(b=8) == ERR_FORMAT and call(ib=2) == ERR_FORMAT
    assert call(vocab=0) == ERR_K and call(vocab=-5) == ERR_K and call(vocab=(1 << 30) + 1, stride=1 << 31) == ERR_K
    assert call(rows=-1) == ERR_SIZE and call(rows=1 << 27) == ERR_SIZE and call(stride=999) == ERR_SIZE
    assert call(rows=1 << 20, stride=1 << 23) == ERR_SIZE                      # 2^43 elements
    for t in (0.0, -1.0, NAN, INF, 1e-9, 1e9):
        assert call(t=t) == ERR_SIZE
    assert call(top=-1) == ERR_K and call(top=33) == ERR_K and call(vocab=4, top=5) == ERR_K
    assert call(x=None) == ERR_NULL and call(ids=None) == ERR_NULL and call(lp=None) == ERR_NULL
    assert call(tl=None) == ERR_NULL and call(ti=None) == ERR_NULL and call(top=0) == ERR_NULL
    assert call(ids=None, lp=None, ent=None, top=0, tl=None, ti=None, st=None) == ERR_NULL     # nothing asked for
    assert call(x=P[0] + 1) == ERR_ALIGN and call(b=4, x=P[0] + 2) == ERR_ALIGN
    for name in ("ids", "lp", "ent", "tl", "ti", "st"):
        assert call(**{name: P[9] + 8}) == ERR_ALIGN
    assert call(lp=P[0] + 16) == ERR_ALIAS and call(ti=P[4]) == ERR_ALIAS and call(st=P[1]) == ERR_ALIAS
    assert call(ent=P[0] + 16 * 400) == ERR_ALIAS                             # inside the last row


def test_token_logprobs_backward(L):
    def call(x=P[0], b=2, rows=4, vocab=1000, stride=1000, ids=P[1], ib=8, t=1.0, st=P[2], g=P[3], ent=P[4], dh=P[5], dx=P[6],
             ds=1000):
        return L.fp8q_token_logprobs_backward(x, b, rows, vocab, stride, ids, ib, t, st, g, ent, dh, dx, ds, None)
    assert call(rows=0) == OK
    assert call(b=3) == ERR_FORMAT and call(ib=1) == ERR_FORMAT and call(vocab=0) == ERR_K
    assert call(rows=-1) == ERR_SIZE and call(stride=999) == ERR_SIZE and call(ds=999) == ERR_SIZE and call(t=0.0) == ERR_SIZE
    for name in ("x", "ids", "st", "g", "ent", "dh", "dx"):
        assert call(**{name: None}) == ERR_NULL
    assert call(ids=None, g=None, ent=None, dh=None) == ERR_NULL
    assert call(x=P[0] + 1) == ERR_ALIGN and call(dx=P[6] + 1) == ERR_ALIGN
    for name in ("ids", "st", "g", "ent", "dh"):
        assert call(**{name: P[9] + 8}) == ERR_ALIGN
    assert call(dx=P[0], ds=1008) == ERR_ALIAS and call(dx=P[0] + 16) == ERR_ALIAS and call(dx=P[2]) == ERR_ALIAS
    assert call(dx=P[3] - 16) == ERR_ALIAS


def plan_of(L, *tensors, count=None):
    """tensors: (grad, out, n, grad type, out type) -> (status, plan address, workspace bytes, keepalive)."""
    import weight_transfer_gb300 as w
    n = len(tensors) if count is None else count
    arr = (w.fp8q_grad_t * max(len(tensors), 1))(*tensors)
    need = max(L.fp8q_grad_plan_bytes(n), 64)
    mem = ctypes.create_string_buffer(need + 16)
    at = (ctypes.addressof(mem) + 15) & ~15
    ws = ctypes.c_size_t(0)
    return L.fp8q_grad_plan(arr, n, at, need, ctypes.byref(ws)), at, ws.value, mem


def test_grad_plan(L):
    assert L.fp8q_grad_plan_bytes(-1) == 0 and L.fp8q_grad_plan_bytes(16385) == 0
    assert plan_of(L, (P[0], None, 100, 0, 0))[0] == OK
    assert plan_of(L, count=0)[0::2][0] == OK
    assert plan_of(L, (P[0], None, 100, 2, 0))[0] == ERR_FORMAT and plan_of(L, (P[0], P[1], 100, 0, -1))[0] == ERR_FORMAT
    assert plan_of(L, (P[0], None, (1 << 42) + 1, 0, 0))[0] == ERR_SIZE
    assert plan_of(L, (None, None, 100, 0, 0))[0] == ERR_NULL and plan_of(L, (None, None, 0, 0, 0))[0] == OK
    assert plan_of(L, (P[0] + 1, None, 9, 0, 0))[0] == ERR_ALIGN and plan_of(L, (P[0] + 2, None, 9, 1, 0))[0] == ERR_ALIGN
    assert plan_of(L, (P[0] + 2, P[1] + 2, 9, 0, 1))[0] == ERR_ALIGN and plan_of(L, (P[0] + 2, P[1] + 4, 9, 0, 1))[0] == OK
    st, at, ws, mem = plan_of(L, (P[0], None, 100, 0, 0))
    ws2 = ctypes.c_size_t(0)
    import weight_transfer_gb300 as w
    arr = (w.fp8q_grad_t * 1)((P[0], None, 100, 0, 0))
    need = L.fp8q_grad_plan_bytes(1)
    assert L.fp8q_grad_plan(arr, 1, at, need - 1, ctypes.byref(ws2)) == ERR_SIZE
    assert L.fp8q_grad_plan(arr, 1, at + 8, need, ctypes.byref(ws2)) == ERR_ALIGN
    assert L.fp8q_grad_plan(arr, 1, None, need, ctypes.byref(ws2)) == ERR_NULL
    assert L.fp8q_grad_plan(arr, 1, at, need, None) == ERR_NULL and L.fp8q_grad_plan(None, 1, at, need, ctypes.byref(ws2)) == ERR_NULL
    assert L.fp8q_grad_plan(arr, 16385, at, need, ctypes.byref(ws2)) == ERR_SIZE


def test_grad_workspace_grows_with_the_chunks(L):
    """8 bytes for each chunk of 32 KB, of larger ones past 4096 of them."""
    sizes = [1, 16384, 16385, 0, 40000]
    assert plan_of(L, *[(P[i], None, n, 0, 0) for i, n in enumerate(sizes)])[2] == 8 * (1 + 1 + 2 + 0 + 3)
    assert plan_of(L, *[(P[i], None, n, 1, 0) for i, n in enumerate([1, 8192, 8193])])[2] == 8 * (1 + 1 + 2)
    assert plan_of(L, (P[0], None, 3_500_000_000, 0, 0))[2] == 8 * -(-7_000_000_000 // (1 << 21))
    assert plan_of(L, (P[0], None, 1 << 42, 0, 0))[2] == 8 * 4096


@pytest.mark.parametrize("name", ["fp8q_grad_norm", "fp8q_grad_clip"])
def test_grad_calls(L, name):
    st, at, ws, mem = plan_of(L, (P[0], P[1], 40000, 0, 1), (P[2], None, 10, 1, 0))
    assert st == OK and ws == 4 * 8

    def call(plan=at, scale=1.0, most=1.0, norm=P[3], each=P[4], w=P[5], wb=ws):
        return getattr(L, name)(plan, scale, most, norm, each, w, wb, None)
    for v in (0.0, -1.0, NAN, INF):
        assert call(scale=v) == ERR_SIZE
    for v in (0.0, -1.0, NAN):
        assert call(most=v) == ERR_SIZE
    assert call(plan=None) == ERR_NULL and call(norm=None) == ERR_NULL and call(w=None) == ERR_NULL
    assert call(plan=at + 8) == ERR_ALIGN and call(wb=ws - 1) == ERR_SIZE
    for n in ("norm", "each", "w"):
        assert call(**{n: P[9] + 8}) == ERR_ALIGN
    assert call(each=P[3]) == ERR_ALIAS and call(w=P[3]) == ERR_ALIAS
    for n in ("norm", "each", "w"):                       # over a gradient or over an output
        assert call(**{n: P[0] + 79984}) == ERR_ALIAS and call(**{n: P[2] + 32}) == ERR_ALIAS
        assert call(**{n: P[1] + 159984}) == ERR_ALIAS
    blank = ctypes.create_string_buffer(4096)
    assert call(plan=(ctypes.addressof(blank) + 15) & ~15) == ERR_FORMAT


def test_grad_clip_refuses_overlapping_outputs(L):
    def clip(*tensors):
        st, at, ws, mem = plan_of(L, *tensors)
        assert st == OK
        return L.fp8q_grad_clip(at, 1.0, 1.0, P[10], None, P[11], ws, None)
    assert clip((P[0], P[0] + 16, 100, 0, 0)) == ERR_ALIAS                      # its own input, shifted
    assert clip((P[0], P[0], 100, 0, 1)) == ERR_ALIAS                           # in place in another type
    assert clip((P[0], P[2], 100, 0, 0), (P[1], P[2] + 198, 100, 0, 0)) == ERR_ALIAS
    assert clip((P[0], None, 100, 0, 0), (P[0] + 198, P[2], 100, 0, 0)) == ERR_ALIAS   # another one's input
    assert clip((P[0], None, 100, 0, 0), (P[0], None, 100, 0, 0)) == ERR_ALIAS         # the same one twice, in place
    assert clip((P[0], P[1], 100, 0, 0), (P[3], P[4], 5, 0, 0), (P[1] + 150, None, 100, 0, 0)) == ERR_ALIAS


def test_moe_decode(L):
    need = L.mxfp8_moe_decode_workspace_bytes(4, 2, 64)
    assert need >= 4 * 2 * 64 * 4
    assert L.mxfp8_moe_decode_workspace_bytes(33, 2, 64) == 0 and L.mxfp8_moe_decode_workspace_bytes(4, 2, 48) == 0
    assert L.mxfp8_moe_decode_workspace_bytes(4, 33, 64) == 0

    def call(c=P[0], s=P[1], ids=P[2], ib=8, w=P[3], tokens=4, topk=2, g=P[4], gs=P[5], u=P[6], us=P[7], d=P[8], ds=P[9],
             experts=3, n=64, k=96, out=P[10], ws=P[11], wb=need):
        return L.mxfp8_moe_decode(c, s, ids, ib, w, tokens, topk, g, gs, u, us, d, ds, experts, n, k, out, ws, wb, None)
    assert call(tokens=0) == OK
    assert call(ib=2) == ERR_FORMAT
    assert call(tokens=-1) == ERR_SIZE and call(tokens=33) == ERR_SIZE
    assert call(experts=0) == ERR_SIZE and call(experts=1025) == ERR_SIZE and call(wb=need - 1) == ERR_SIZE
    assert call(topk=0) == ERR_K and call(topk=33) == ERR_K
    for bad in (0, -32, 48, 16416):
        assert call(n=bad) == ERR_K and call(k=bad) == ERR_K
    for name in ("c", "s", "ids", "w", "g", "gs", "u", "us", "d", "ds", "out", "ws"):
        assert call(**{name: None}) == ERR_NULL
        assert call(**{name: P[12] + 8}) == ERR_ALIGN
    assert call(out=P[0]) == ERR_ALIAS and call(ws=P[8] + 64) == ERR_ALIAS and call(out=P[11]) == ERR_ALIAS
    assert call(ws=P[9]) == ERR_ALIAS and call(out=P[3]) == ERR_ALIAS


def test_binding_refuses(L):
    """What the binding itself turns away, on CPU tensors and wrong shapes."""
    import weight_transfer_gb300 as w
    x = torch.zeros(4, 10)
    with pytest.raises(ValueError, match="CUDA tensor"):
        w.fp8q_token_logprobs(x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError, match="CUDA tensor"):
        w.fp8q_token_logprobs_backward(x, None, torch.zeros(4, 2), entropy=torch.zeros(4), dentropy=torch.zeros(4))
    with pytest.raises(ValueError, match="CUDA tensor"):
        w.fp8q_grad_norm([x])
    with pytest.raises(ValueError, match="1 gradients and 2 outputs"):
        w.fp8q_grad_list([x], [x, x])
