"""Refusals of the expert-block operators: every bad argument is answered with
its status before anything is launched (fake addresses are never dereferenced)."""
import ctypes

import pytest

from conftest import build_lib
from test_abi import A, ERR_ALIAS, ERR_ALIGN, ERR_FLAGS, ERR_FORMAT, ERR_K, ERR_NULL, ERR_SIZE, MB, OK

F = ctypes.c_float
P = [A + i * 64 * MB for i in range(16)]


@pytest.fixture(scope="module")
def L():
    build_lib()
    import weight_transfer_gb300 as w
    return w.lib()


def test_rmsnorm(L):
    f, m = L.fp8q_rmsnorm_quantize, L.mxfp8_rmsnorm_quantize
    x, r, w, s, y, c, sc, rs = P[:8]

    def call(fn, x=x, r=r, w=w, rows=4, k=256, eps=1e-6, mode=0, s=s, y=y, c=c, sc=sc, rs=rs):
        return fn(x, r, w, rows, k, eps, mode, s, y, c, sc, rs, None)
    for fn in (f, m):
        assert call(fn, rows=0) == OK
        assert call(fn, rows=-1) == ERR_SIZE
        assert call(fn, rows=1 << 31) == ERR_SIZE
        assert call(fn, k=0) == ERR_K and call(fn, k=-128) == ERR_K and call(fn, k=16512) == ERR_K
        assert call(fn, eps=-1.0) == ERR_SIZE and call(fn, eps=float("nan")) == ERR_SIZE
        assert call(fn, eps=float("inf")) == ERR_SIZE
        for name in ("x", "w", "c", "sc"):
            assert call(fn, **{name: None}) == ERR_NULL
        assert call(fn, r=None) == ERR_NULL                       # a sum without a residual
        for name in ("x", "r", "w", "s", "y", "c", "sc", "rs"):
            assert call(fn, **{name: P[9] + 8}) == ERR_ALIGN
        assert call(fn, y=x) == ERR_ALIAS and call(fn, c=w) == ERR_ALIAS and call(fn, s=w) == ERR_ALIAS
        assert call(fn, s=x + 32) == ERR_ALIAS and call(fn, y=s) == ERR_ALIAS and call(fn, rs=sc) == ERR_ALIAS
    assert call(f, mode=2) == ERR_FORMAT
    assert call(m, mode=2) == ERR_FLAGS
    assert call(f, k=96) == ERR_K and call(m, k=48) == ERR_K


def test_rmsnorm_backward(L):
    fn = L.fp8q_rmsnorm_backward
    need = L.fp8q_rmsnorm_backward_workspace_bytes(4, 256)
    assert need >= 256 * 4 and need % 1024 == 0
    assert L.fp8q_rmsnorm_backward_workspace_bytes(4, 48) == 0

    def call(dy=P[0], h=P[1], w=P[2], rs=P[3], ds=P[4], rows=4, k=256, dx=P[5], dw=P[6], ws=P[7], wb=need):
        return fn(dy, h, w, rs, ds, rows, k, dx, dw, ws, wb, None)
    assert call(rows=-1) == ERR_SIZE and call(k=80) == ERR_K and call(wb=need - 1) == ERR_SIZE
    for name in ("dy", "h", "w", "rs", "dx", "dw", "ws"):
        assert call(**{name: None}) == ERR_NULL
    for name in ("dy", "h", "w", "rs", "ds", "dx", "dw", "ws"):
        assert call(**{name: P[9] + 4}) == ERR_ALIGN
    assert call(dx=P[1]) == ERR_ALIAS and call(dx=P[0] + 16) == ERR_ALIAS and call(dw=P[5]) == ERR_ALIAS
    assert call(ws=P[0]) == ERR_ALIAS and call(dw=P[7]) == ERR_ALIAS


def test_moe_sort(L):
    fn = L.fp8q_moe_sort
    need = L.fp8q_moe_sort_workspace_bytes(100000, 8, 128)
    assert need > 0 and L.fp8q_moe_sort_workspace_bytes(1, 8, 128) == 0
    assert L.fp8q_moe_sort_workspace_bytes(1, 33, 128) == 0

    def call(ids=P[0], b=4, tokens=100000, topk=8, experts=128, off=P[1], order=P[2], slots=P[3], ws=P[4], wb=need):
        return fn(ids, b, tokens, topk, experts, off, order, slots, ws, wb, None)
    assert call(b=2) == ERR_FORMAT
    assert call(tokens=-1) == ERR_SIZE and call(experts=0) == ERR_SIZE and call(experts=1025) == ERR_SIZE
    assert call(topk=0) == ERR_K and call(topk=33) == ERR_K and call(tokens=1 << 28) == ERR_SIZE
    assert call(wb=need - 1) == ERR_SIZE
    for name in ("ids", "off", "order", "slots", "ws"):
        assert call(**{name: None}) == ERR_NULL
        assert call(**{name: P[9] + 4}) == ERR_ALIGN
    assert call(order=P[0]) == ERR_ALIAS and call(slots=P[2]) == ERR_ALIAS and call(ws=P[3]) == ERR_ALIAS


def test_moe_rows(L):
    g, mg, c, cb = L.fp8q_moe_gather, L.mxfp8_moe_gather, L.fp8q_moe_combine, L.fp8q_moe_combine_backward

    def gather(x=P[0], sl=P[1], off=P[2], tokens=4, topk=2, experts=3, k=64, out=P[3]):
        return g(x, sl, off, tokens, topk, experts, k, out, None)

    def mgather(x=P[0], sc=P[4], sl=P[1], off=P[2], tokens=4, topk=2, experts=3, k=64, out=P[3], osc=P[5]):
        return mg(x, sc, sl, off, tokens, topk, experts, k, out, osc, None)

    def combine(x=P[0], sl=P[1], off=P[2], w=P[4], tokens=4, topk=2, experts=3, k=64, out=P[3]):
        return c(x, sl, off, w, tokens, topk, experts, k, out, None)

    def backward(d=P[6], x=P[0], sl=P[1], off=P[2], w=P[4], tokens=4, topk=2, experts=3, k=64, out=P[3], dw=P[5]):
        return cb(d, x, sl, off, w, tokens, topk, experts, k, out, dw, None)
    for fn in (gather, mgather, combine, backward):
        assert fn(tokens=0) == OK and fn(tokens=-1) == ERR_SIZE and fn(tokens=1 << 30) == ERR_SIZE
        assert fn(topk=0) == ERR_K and fn(topk=33) == ERR_K and fn(experts=0) == ERR_SIZE and fn(experts=1025) == ERR_SIZE
        assert fn(k=0) == ERR_K and fn(k=-64) == ERR_K and fn(k=20) == ERR_K and fn(k=(1 << 30) + 32) == ERR_SIZE
        for name in ("x", "sl", "off", "out"):
            assert fn(**{name: None}) == ERR_NULL
            assert fn(**{name: P[9] + 2}) == ERR_ALIGN
        assert fn(out=P[0]) == ERR_ALIAS and fn(out=P[1]) == ERR_ALIAS and fn(out=P[2]) == ERR_ALIAS
    assert mgather(k=40) == ERR_K and mgather(sc=None) == ERR_NULL and mgather(osc=None) == ERR_NULL
    assert mgather(osc=P[3]) == ERR_ALIAS and mgather(osc=P[4]) == ERR_ALIAS
    assert combine(out=P[4]) == ERR_ALIAS
    assert backward(w=None) == ERR_NULL and backward(d=None) == ERR_NULL and backward(dw=None) == ERR_NULL
    assert backward(dw=P[3]) == ERR_ALIAS and backward(dw=P[6]) == ERR_ALIAS


def test_moe_products(L):
    mm, sg = L.mxfp8_moe_matmul, L.mxfp8_moe_swiglu

    def matmul(a=P[0], s=P[1], rows=4, w=P[2], ws=P[3], off=P[4], experts=2, n=64, k=64, out=P[5]):
        return mm(a, s, rows, w, ws, off, experts, n, k, out, None)

    def swiglu(a=P[0], s=P[1], rows=4, w=P[2], ws=P[3], u=P[6], us=P[7], off=P[4], experts=2, n=64, k=64, out=P[5], os=P[8]):
        return sg(a, s, rows, w, ws, u, us, off, experts, n, k, out, os, None)
    for fn in (matmul, swiglu):
        assert fn(rows=0) == OK and fn(n=0) == OK
        assert fn(rows=-1) == ERR_SIZE and fn(rows=1 << 31) == ERR_SIZE and fn(n=-32) == ERR_SIZE
        assert fn(experts=0) == ERR_SIZE and fn(experts=1025) == ERR_SIZE
        assert fn(k=0) == ERR_K and fn(k=48) == ERR_K and fn(n=1 << 30, k=1 << 20) == ERR_SIZE
        for name in ("a", "s", "w", "ws", "off", "out"):
            assert fn(**{name: None}) == ERR_NULL
            assert fn(**{name: P[9] + 8}) == ERR_ALIGN
        for p in (P[0], P[1], P[2], P[3], P[4]):
            assert fn(out=p) == ERR_ALIAS
    assert swiglu(n=48) == ERR_K and swiglu(u=None) == ERR_NULL and swiglu(us=None) == ERR_NULL
    assert swiglu(os=None) == ERR_NULL and swiglu(os=P[5]) == ERR_ALIAS and swiglu(os=P[6]) == ERR_ALIAS


def test_binding_checks_shapes():
    import torch
    import weight_transfer_gb300 as w
    b = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        w.mxfp8_rmsnorm_quantize(b(2, 64), b(64), scales=torch.zeros(4, dtype=torch.uint8))
    with pytest.raises(ValueError, match="weight"):
        w.mxfp8_rmsnorm_quantize(b(2, 64), b(32))
    with pytest.raises(ValueError, match="residual"):
        w.fp8q_rmsnorm_quantize(b(2, 128), b(128), residual=b(2, 64))
    with pytest.raises(ValueError, match="ids"):
        w.fp8q_moe_sort(torch.zeros(4, dtype=torch.int32), 4)
    with pytest.raises(ValueError, match="int32 or int64"):
        w.fp8q_moe_sort(torch.zeros(4, 2), 4)
