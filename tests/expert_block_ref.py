"""Plain 64-bit implementations of the expert-block operators (test infrastructure)."""
import numpy as np
import torch

F8MAX = {"e4m3": 448.0, "e5m2": 57344.0}
F8DT = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}


def decode(codes, fmt="e4m3"):
    return codes.cpu().view(F8DT[fmt]).float().double()


def rne8(v, fmt):
    """float64 -> the 8-bit value it rounds to (saturating), as float64.  The
    double rounding through float32 is avoided by rounding on the format's own grid."""
    mant, emin = (3, -6) if fmt == "e4m3" else (2, -14)
    v = v.clamp(-F8MAX[fmt], F8MAX[fmt])
    e = torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -100))).clamp(min=emin)
    step = torch.pow(torch.tensor(2.0, dtype=torch.float64), e - mant)
    return (torch.round(v / step) * step).clamp(-F8MAX[fmt], F8MAX[fmt])


def e8m0(amax):
    """The MXFP8 exponent byte of float64 block maxima."""
    m, ex = torch.frexp(amax)
    e = (ex - 1 - 8 + 127).clamp(0, 254)
    return torch.where(amax > 0, e, torch.zeros_like(e)).long()


def unswizzle(scales, m, kb):
    r, c = -(-m // 128), -(-kb // 4)
    full = scales.reshape(r, c, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(r * 128, c * 4)
    return full[:m, :kb], full


def check_mx(y, codes, exps, tol):
    """codes [rows, k] and E8M0 bytes [rows, k/32] (long) are a quantization of some y' within a
    relative `tol` of the float64 y."""
    b = y.reshape(y.shape[0], -1, 32)
    top = b.abs().amax(2)
    lo, hi = e8m0(top * (1 - tol)), e8m0(top * (1 + tol))
    exps = exps.reshape(lo.shape)
    bad = (exps < lo) | (exps > hi)
    assert not bad.any(), f"{int(bad.sum())} scales off, first at {bad.nonzero()[0].tolist()}"
    f = torch.pow(torch.tensor(2.0, dtype=torch.float64), (127 - exps).double())[..., None]
    check_codes(b * f, decode(codes).reshape(b.shape), tol, "e4m3")


def check_codes(q, v, tol, fmt):
    """v is the 8-bit rounding of some q' within a relative `tol` of q."""
    a, c = rne8(q * (1 - tol), fmt), rne8(q * (1 + tol), fmt)
    bad = (v < torch.minimum(a, c)) | (v > torch.maximum(a, c))
    assert not bad.any(), f"{int(bad.sum())} codes off, first at {bad.nonzero()[0].tolist()}"


def check_bf16(got, want, tol, scale=None):
    """got (bf16) is the rounding of a value within tol * scale (or tol * |want|) of the float64 want: it lies between
    the roundings of the two ends of that interval (each first brought to binary32, outwards)."""
    slack = tol * (want.abs() if scale is None else scale)
    inf = torch.tensor(float("inf"))
    lo = torch.nextafter((want - slack).float(), -inf).bfloat16().double()
    hi = torch.nextafter((want + slack).float(), inf).bfloat16().double()
    v = got.double().cpu()
    bad = (v < lo) | (v > hi) | v.isnan()
    assert not bad.any(), f"{int(bad.sum())} values off, first at {bad.nonzero()[0].tolist()}"


def sort_ref(ids, experts):
    flat = ids.cpu().reshape(-1).tolist()
    key = [e if 0 <= e < experts else experts for e in flat]
    order = sorted(range(len(key)), key=lambda i: key[i])
    slots = [0] * len(key)
    for s, i in enumerate(order):
        slots[i] = s
    counts = np.bincount(np.asarray(key, dtype=np.int64), minlength=experts + 1)[:experts]
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    return offsets, np.asarray(order, np.int32), np.asarray(slots, np.int32).reshape(ids.shape)
