"""The operators of a mixture-of-experts block, each in its plain form and as the library's calls.

Three operators that a user who moves MXFP8 expert weights needs next to them:

* ``norm`` / ``norm_grad``: residual addition and root-mean-square norm with an output in 8 bits and its scales (and
  the gradient of the norm);
* ``route`` / ``route_grad``: tokens sorted by expert, their rows carried to the experts and the experts' rows summed
  back with weights (and the gradients of both ways);
* ``experts`` / ``swiglu``: the experts' products with MXFP8 weights, either to bf16 rows or through the gated
  activation to MXFP8 rows.

``run`` with ``own`` false computes them with elementary torch operations in 32 bits; with ``own`` true it makes the
calls a user of the package makes.
"""
import math

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
EPS = 1e-6
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
FMAX = {"e4m3": 448.0, "e5m2": 57344.0}

# ---------------------------------------------------------------- cases ----


def listed():
    return [
        # one decode step of four requests: the norm in front of a product with blockwise FP8 activations
        {"name": "norm_step", "op": "norm", "rows": 4, "k": 2048, "fmt": "e4m3", "residual": True, "bf16": False},
        # a prefill batch of a wider model: MXFP8 for the experts, and the bf16 row that the router reads
        {"name": "norm_prompt", "op": "norm", "rows": 16384, "k": 4096, "fmt": "mxfp8", "residual": True, "bf16": True},
        # the norm's gradient on a ragged micro-batch
        {"name": "norm_grad_odd", "op": "norm_grad", "rows": 777, "k": 5120, "residual": True},
        # the norm's gradient on a full training micro-batch
        {"name": "norm_grad_long", "op": "norm_grad", "rows": 16384, "k": 4096, "residual": True},
        # one token to its 8 of 128 experts and back
        {"name": "route_step", "op": "route", "tokens": 1, "topk": 8, "experts": 128, "k": 2048, "form": "mxfp8",
         "id_bits": 32, "drop": False},
        # a prefill batch to its experts and back
        {"name": "route_prompt", "op": "route", "tokens": 8192, "topk": 8, "experts": 128, "k": 2048, "form": "mxfp8",
         "id_bits": 64, "drop": False},
        # training with some choices dropped (capacity), odd counts
        {"name": "route_grad_odd", "op": "route_grad", "tokens": 1531, "topk": 6, "experts": 60, "k": 1408,
         "drop": True},
        # a training micro-batch
        {"name": "route_grad_long", "op": "route_grad", "tokens": 8192, "topk": 8, "experts": 128, "k": 2048,
         "drop": False},
        # the down projection of one token: 8 rows, each of another expert
        {"name": "experts_step", "op": "experts", "rows": 8, "experts": 128, "n": 2048, "k": 768, "drop": False},
        # the down projection of a prefill batch, odd rows, some dropped
        {"name": "experts_prompt", "op": "experts", "rows": 65533, "experts": 128, "n": 2048, "k": 768, "drop": True},
        # the gate and up projections of a decode batch of 64 requests
        {"name": "swiglu_step", "op": "swiglu", "rows": 512, "experts": 128, "n": 768, "k": 2048, "drop": False},
        # the gate and up projections of a prefill batch
        {"name": "swiglu_prompt", "op": "swiglu", "rows": 65536, "experts": 128, "n": 768, "k": 2048, "drop": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi, step):
    w = max(lo, _log(rng, lo, hi) // step * step)
    return w + step if w == 3072 else w


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "route", "route", "route_grad", "experts", "experts", "swiglu", "swiglu"])
    if op == "norm":
        fmt = rng.choice(["mxfp8", "mxfp8", "mxfp8_swizzled", "e4m3", "e5m2"])
        k = _width(rng, 128, 16384, 32 if fmt.startswith("mxfp8") else 128)
        return {"op": op, "rows": _log(rng, 1, max(1, min(40000, (16384 * 4096) // k))), "k": k, "fmt": fmt,
                "residual": rng.random() < 0.75, "bf16": rng.random() < 0.5}
    if op == "norm_grad":
        k = _width(rng, 128, 16384, 32)
        return {"op": op, "rows": _log(rng, 1, max(1, min(40000, (16384 * 4096) // k))), "k": k,
                "residual": rng.random() < 0.75}
    if op in ("route", "route_grad"):
        k = _width(rng, 256, 8192, 32)
        topk = rng.choice([1, 2, 3, 4, 6, 8])
        tokens = _log(rng, 1, max(1, min(60000, (8192 * 8 * 2048) // (k * topk))))
        c = {"op": op, "tokens": tokens, "topk": topk, "experts": max(topk, _log(rng, 4, 384)), "k": k,
             "drop": rng.random() < 0.4}
        if op == "route":
            c.update(form=rng.choice(["mxfp8", "mxfp8", "bf16"]), id_bits=rng.choice([32, 64]))
        return c
    experts = _log(rng, 1, 160)
    n, k = _width(rng, 256, 2560, 32), _width(rng, 256, 2560, 32)
    while experts * n * k > 128 * 768 * 2048:
        experts = max(1, experts // 2)
    rows = _log(rng, 1, max(1, min(60000, 65536 * 768 * 2048 // (n * k))))
    return {"op": op, "rows": rows, "experts": experts, "n": n, "k": k, "drop": rng.random() < 0.3}


def work(c):
    op = c["op"]
    if op in ("norm", "norm_grad"):
        e = c["rows"] * c["k"]
        if op == "norm":
            per = 2 + (4 if c["residual"] else 0) + 1 + (2 if c["bf16"] else 0) + (1 / 32 if c["fmt"].startswith("mx") else 4 / 128)
            return {"bytes": e * per + 2 * c["k"] + 4 * c["rows"], "flops": 8 * e}
        return {"bytes": e * (6 + (2 if c["residual"] else 0)) + 6 * c["k"] + 4 * c["rows"], "flops": 12 * e}
    if op in ("route", "route_grad"):
        t, s, k = c["tokens"], c["tokens"] * c["topk"], c["k"]
        if op == "route":
            # ids in; order, slots, offsets out; each token's row read once and written once per choice; the experts'
            # rows read once, one row a token out
            row = 2 * k if c["form"] == "bf16" else k + k // 32
            return {"bytes": s * (c["id_bits"] // 8 + 8 + 4) + 4 * (c["experts"] + 1) + (t + s) * row + s * 2 * k + t * 2 * k,
                    "flops": 2 * s * k}
        # dout and the experts' rows in, their gradients out; the carried rows' gradients in, one row a token out
        return {"bytes": t * 2 * k + s * (2 * k + 2 * k + 4 + 4) + s * 4 + s * 2 * k + t * 2 * k, "flops": 4 * s * k}
    r, n, k, e = c["rows"], c["n"], c["k"], c["experts"]
    active = e * (1 - (1 - 1 / e) ** r)
    if op == "experts":
        return {"bytes": active * n * k * 33 / 32 + r * k * 33 / 32 + r * n * 2, "flops": 2 * r * n * k}
    return {"bytes": 2 * active * n * k * 33 / 32 + r * k * 33 / 32 + r * n * 33 / 32, "flops": 4 * r * n * k}


# --------------------------------------------------------------- inputs ----


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _hidden(g, rows, k):
    """A residual stream: rows of different size, and a few channels far above the rest."""
    x = _randn(g, rows, k) * torch.exp(0.5 * _randn(g, rows, 1))
    loud = torch.rand(k, generator=g, device=DEV) < 0.01
    return (x * (1 + 19 * loud)).bfloat16()


def _mx_quantize(x):
    """x [..., k] in 32 or 64 bits -> the values before their rounding to e4m3, the E8M0 bytes [..., k/32] (int64)."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax).exponent.to(torch.int64) - 1 - 8 + 127).clamp(0, 254)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    q = torch.ldexp(b, (127 - e).to(torch.int32)[..., None]).clamp(-448, 448)
    return q.flatten(-2), e


def _swizzle(s):
    """E8M0 bytes [..., m, kb] -> the 128 x 4 tiled layout, flat per matrix, padding 0."""
    lead, (m, kb) = s.shape[:-2], s.shape[-2:]
    r, c = -(-m // 128), -(-kb // 4)
    t = torch.zeros(*lead, r * 128, c * 4, dtype=s.dtype, device=s.device)
    t[..., :m, :kb] = s
    t = t.reshape(*lead, r, 4, 32, c, 4)
    n = len(lead)
    return t.permute(*range(n), n, n + 3, n + 2, n + 1, n + 4).reshape(*lead, -1)


def _unswizzle(s, m, kb):
    lead = s.shape[:-1]
    r, c = -(-m // 128), -(-kb // 4)
    n = len(lead)
    t = s.reshape(*lead, r, c, 32, 4, 4).permute(*range(n), n, n + 3, n + 2, n + 1, n + 4)
    return t.reshape(*lead, r * 128, c * 4)[..., :m, :kb]


def _mx_inputs(x):
    q, e = _mx_quantize(x.float())
    return q.to(F8["e4m3"]).view(torch.uint8), e.to(torch.uint8)


def _popular(g, experts):
    return torch.softmax(0.5 * _randn(g, experts), 0)


def _choices(g, tokens, topk, experts, drop):
    """Each token's experts, all different, popular ones more often; with `drop` some choices are taken back (-1)."""
    p = torch.log(_popular(g, experts))
    noise = -torch.log(-torch.log(torch.rand(tokens, experts, generator=g, device=DEV).clamp(1e-9, 1 - 1e-7)))
    score, ids = torch.topk(p + noise, topk, dim=1)
    if drop:
        ids = torch.where(torch.rand(tokens, topk, generator=g, device=DEV) < 0.1, torch.full_like(ids, -1), ids)
        if tokens > 2:
            ids[tokens // 2] = -1          # a token that no expert takes
    return ids, torch.softmax(score, 1)


def _sort_plain(ids, experts):
    """-> offsets [experts + 1], order [n], slots [n]: a stable sort of the choices by expert, dropped ones last."""
    key = torch.where((ids < 0) | (ids >= experts), torch.full_like(ids, experts), ids).reshape(-1)
    order = torch.sort(key, stable=True).indices
    slots = torch.empty_like(order)
    slots[order] = torch.arange(order.numel(), device=order.device)
    count = (key[:, None] == torch.arange(experts, device=key.device)).sum(0) if key.numel() * experts <= 1 << 24 \
        else torch.zeros(experts + 1, dtype=torch.int64, device=key.device).index_add_(0, key.long(), torch.ones_like(key, dtype=torch.int64))[:experts]
    offsets = torch.cat([count.new_zeros(1), torch.cumsum(count, 0)])
    return offsets.to(torch.int32), order.to(torch.int32), slots.to(torch.int32).reshape(ids.shape)


def _groups(g, rows, experts, drop):
    """Rows of each expert, as offsets on the GPU; `cap`, the most that one expert has, is known to the host as a
    capacity would be."""
    routed = rows - rows // 13 if drop else rows
    e = torch.multinomial(_popular(g, experts), max(routed, 1), replacement=True, generator=g)[:routed]
    if rows <= 16 and rows <= experts:      # a token's choices are different experts
        e = torch.randperm(experts, generator=g, device=DEV)[:routed]
    count = torch.bincount(e, minlength=experts)
    offsets = torch.cat([count.new_zeros(1), torch.cumsum(count, 0)]).to(torch.int32)
    return offsets, int(count.max())


def _weights(g, experts, n, k):
    w = _randn(g, experts, n, k) * 0.02
    codes, scales = _mx_inputs(w)
    return codes, _swizzle(scales).reshape(-1)


def prepare(c, seed):
    g, op = _gen(seed), c["op"]
    s = {"case": c}
    if op == "norm":
        s["x"] = _hidden(g, c["rows"], c["k"])
        s["residual"] = _hidden(g, c["rows"], c["k"]) if c["residual"] else None
        s["weight"] = (1 + 0.2 * _randn(g, c["k"])).bfloat16()
    elif op == "norm_grad":
        s["h"] = _hidden(g, c["rows"], c["k"])
        s["dy"] = (_randn(g, c["rows"], c["k"]) * 1e-3).bfloat16()
        s["dsum"] = (_randn(g, c["rows"], c["k"]) * 1e-3).bfloat16() if c["residual"] else None
        s["weight"] = (1 + 0.2 * _randn(g, c["k"])).bfloat16()
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(-1) + EPS)
    elif op in ("route", "route_grad"):
        t, n = c["tokens"], c["tokens"] * c["topk"]
        ids, s["weights"] = _choices(g, t, c["topk"], c["experts"], c["drop"])
        s["y"] = _randn(g, n, c["k"]).bfloat16()
        if op == "route":
            s["ids"] = ids.to(torch.int64 if c["id_bits"] == 64 else torch.int32)
            s["x"] = _hidden(g, t, c["k"])
            if c["form"] == "mxfp8":
                s["codes"], s["scales"] = _mx_inputs(s.pop("x"))
        else:
            s["offsets"], _, s["slots"] = _sort_plain(ids, c["experts"])
            s["dout"] = (_randn(g, t, c["k"]) * 1e-3).bfloat16()
            s["dxs"] = (_randn(g, n, c["k"]) * 1e-3).bfloat16()
    else:
        s["offsets"], s["cap"] = _groups(g, c["rows"], c["experts"], c["drop"])
        s["codes"], s["scales"] = _mx_inputs(_randn(g, c["rows"], c["k"]) * (1 if op == "swiglu" else 0.1))
        if op == "experts":
            s["w"], s["ws"] = _weights(g, c["experts"], c["n"], c["k"])
        else:
            s["gate"], s["gs"] = _weights(g, c["experts"], c["n"], c["k"])
            s["up"], s["us"] = _weights(g, c["experts"], c["n"], c["k"])
    return s


# ----------------------------------------------------------- plain form ----


def _e8(e):
    return e.to(torch.uint8).contiguous().view(torch.float8_e8m0fnu)


def _f8(u8):
    return u8.view(torch.float8_e4m3fn)


def _norm_plain(s):
    c = s["case"]
    h = s["x"].float()
    if s["residual"] is not None:
        h = h + s["residual"].float()
    rstd = torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS)
    y = h * rstd * s["weight"].float()
    out = {"rstd": rstd[:, 0]}
    if c["fmt"].startswith("mx"):
        q, e = _mx_quantize(y)
        out["codes"] = q.to(F8["e4m3"])
        out["scales"] = _e8(_swizzle(e) if c["fmt"] == "mxfp8_swizzled" else e)
    else:
        b = y.unflatten(-1, (-1, 128))
        scale = b.abs().amax(-1) / FMAX[c["fmt"]]
        q = torch.where(scale[..., None] > 0, b / scale[..., None], b).clamp(-FMAX[c["fmt"]], FMAX[c["fmt"]])
        out["codes"], out["scales"] = q.flatten(-2).to(F8[c["fmt"]]), scale
    if s["residual"] is not None:
        out["sum"] = h.bfloat16()
    if c["bf16"]:
        out["y"] = y.bfloat16()
    return out


def _norm_grad_plain(s):
    dy, h, w, r = s["dy"].float(), s["h"].float(), s["weight"].float(), s["rstd"][:, None]
    xhat = h * r
    g = dy * w
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    if s["dsum"] is not None:
        dx = dx + s["dsum"].float()
    return {"dx": dx.bfloat16(), "dweight": (dy * xhat).sum(0)}


def _carry(x, order, topk, routed):
    """Rows of x by slot; the slots of dropped choices are zero."""
    live = torch.arange(order.numel(), device=order.device) < routed
    return x[order.long() // topk] * live[:, None].to(x.dtype)


def _back(y, slots, offsets, weights):
    """Sum over a token's choices of its expert rows (weighted where weights are given), dropped ones left out."""
    live = slots < offsets[-1]
    rows = torch.where(live[..., None], y[slots.long()].float(), 0.0)
    return (rows if weights is None else rows * weights[..., None]).sum(1)


def _route_plain(s):
    c = s["case"]
    offsets, order, slots = _sort_plain(s["ids"], c["experts"])
    out = {"offsets": offsets, "order": order, "slots": slots}
    if c["form"] == "mxfp8":
        out["codes"] = _f8(_carry(s["codes"], order, c["topk"], offsets[-1]))
        out["scales"] = _e8(_carry(s["scales"], order, c["topk"], offsets[-1]))
    else:
        out["rows"] = _carry(s["x"], order, c["topk"], offsets[-1])
    out["out"] = _back(s["y"], slots, offsets, s["weights"]).bfloat16()
    return out


def _route_grad_plain(s):
    live = s["slots"] < s["offsets"][-1]
    dout = s["dout"].float()
    dy = torch.empty_like(s["y"])
    dy[s["slots"].long()] = torch.where(live[..., None], dout[:, None] * s["weights"][..., None], 0.0).bfloat16()
    dw = torch.where(live, (dout[:, None] * s["y"][s["slots"].long()].float()).sum(-1), 0.0)
    return {"dy": dy, "dweights": dw, "dx": _back(s["dxs"], s["slots"], s["offsets"], None).bfloat16()}


def _mx_values(codes, scales, dtype=torch.float32):
    """Codes [..., k] and E8M0 bytes [..., k/32] -> the values they stand for."""
    v = _f8(codes).to(dtype).unflatten(-1, (-1, 32))
    return torch.ldexp(v, (scales.to(torch.int32) - 127)[..., None]).flatten(-2)


def _products_plain(s, weights):
    """Each row's product with its expert's matrix, for each of the weight tensors given; rows of no expert are zero."""
    c = s["case"]
    r, n, k, e = c["rows"], c["n"], c["k"], c["experts"]
    off = s["offsets"].long()
    a = _mx_values(s["codes"], s["scales"])
    outs = []
    if r < e:                 # few rows: each row's own matrix
        at = torch.searchsorted(off[1:], torch.arange(r, device=off.device), right=True)
        live, at = at < e, at.clamp(max=e - 1)
        for w, ws in weights:
            m = _mx_values(w[at], _unswizzle(ws.view(e, -1)[at], n, k // 32))
            outs.append(torch.bmm(m, a[:, :, None])[:, :, 0] * live[:, None])
        return outs
    at = off[:-1, None] + torch.arange(s["cap"], device=off.device)
    live = at < off[1:, None]
    padded = a[at.clamp(max=r - 1)] * live[..., None]
    for w, ws in weights:
        m = _mx_values(w, _unswizzle(ws.view(e, -1), n, k // 32))
        p = torch.bmm(padded, m.transpose(1, 2))
        o = torch.zeros(r + 1, n, device=p.device)
        o[torch.where(live, at, r).reshape(-1)] = p.reshape(-1, n)
        outs.append(o[:r])
    return outs


def _experts_plain(s):
    return _products_plain(s, [(s["w"], s["ws"])])[0].bfloat16()


def _swiglu_plain(s):
    g, u = _products_plain(s, [(s["gate"], s["gs"]), (s["up"], s["us"])])
    q, e = _mx_quantize(g / (1 + torch.exp(-g)) * u)
    return {"codes": q.to(F8["e4m3"]), "scales": _e8(e)}


# ------------------------------------------------------ the library's calls ----


def _norm_own(s):
    import weight_transfer_gb300 as fp8q
    c = s["case"]
    if c["fmt"].startswith("mx"):
        codes, scales, total, y, rstd = fp8q.mxfp8_rmsnorm_quantize(
            s["x"], s["weight"], EPS, residual=s["residual"], swizzled=c["fmt"] == "mxfp8_swizzled", want_bf16=c["bf16"],
            want_rstd=True)
        scales = scales.view(torch.float8_e8m0fnu)
        fmt = "e4m3"
    else:
        fmt = c["fmt"]
        codes, scales, total, y, rstd = fp8q.fp8q_rmsnorm_quantize(
            s["x"], s["weight"], EPS, fmt, residual=s["residual"], want_bf16=c["bf16"], want_rstd=True)
    out = {"rstd": rstd, "codes": codes.view(F8[fmt]), "scales": scales}
    if total is not None:
        out["sum"] = total
    if y is not None:
        out["y"] = y
    return out


def _norm_grad_own(s):
    import weight_transfer_gb300 as fp8q
    dx, dw = fp8q.fp8q_rmsnorm_backward(s["dy"], s["h"], s["weight"], s["rstd"], dsum=s["dsum"])
    return {"dx": dx, "dweight": dw}


def _route_own(s):
    import weight_transfer_gb300 as fp8q
    c = s["case"]
    offsets, order, slots = fp8q.fp8q_moe_sort(s["ids"], c["experts"])
    out = {"offsets": offsets, "order": order, "slots": slots}
    if c["form"] == "mxfp8":
        codes, scales = fp8q.mxfp8_moe_gather(s["codes"], s["scales"], slots, offsets)
        out["codes"], out["scales"] = _f8(codes), scales.view(torch.float8_e8m0fnu)
    else:
        out["rows"] = fp8q.fp8q_moe_gather(s["x"], slots, offsets)
    out["out"] = fp8q.fp8q_moe_combine(s["y"], slots, offsets, s["weights"])
    return out


def _route_grad_own(s):
    import weight_transfer_gb300 as fp8q
    dy, dw = fp8q.fp8q_moe_combine_backward(s["dout"], s["y"], s["slots"], s["offsets"], s["weights"])
    return {"dy": dy, "dweights": dw, "dx": fp8q.fp8q_moe_combine(s["dxs"], s["slots"], s["offsets"])}


def _experts_own(s):
    import weight_transfer_gb300 as fp8q
    return fp8q.mxfp8_moe_matmul(s["codes"], s["scales"], s["w"], s["ws"], s["offsets"])


def _swiglu_own(s):
    import weight_transfer_gb300 as fp8q
    codes, scales = fp8q.mxfp8_moe_swiglu(s["codes"], s["scales"], s["gate"], s["gs"], s["up"], s["us"], s["offsets"])
    return {"codes": _f8(codes), "scales": scales.view(torch.float8_e8m0fnu)}


_PLAIN = {"norm": _norm_plain, "norm_grad": _norm_grad_plain, "route": _route_plain, "route_grad": _route_grad_plain,
          "experts": _experts_plain, "swiglu": _swiglu_plain}
_OWN = {"norm": _norm_own, "norm_grad": _norm_grad_own, "route": _route_own, "route_grad": _route_grad_own,
        "experts": _experts_own, "swiglu": _swiglu_own}


def run(s):
    return (_OWN if own else _PLAIN)[s["case"]["op"]](s)


# ------------------------------------------------------------- in 64 bits ----


def _mx_exact(y):
    """y [rows, k] in 64 bits -> what the codes stand for before their rounding to 8 bits, and the scales."""
    b = y.reshape(y.shape[0], -1, 32)
    top = b.abs().max(dim=2).values
    power = torch.floor(torch.log2(top.clamp(min=2.0 ** -200)))
    power = power + (torch.pow(2.0, power + 1) <= top).double() - (torch.pow(2.0, power) > top).double()
    e = torch.where(top > 0, (power - 8 + 127).clamp(0, 254), 0.0)
    return (b * torch.pow(2.0, 127 - e)[:, :, None]).clamp(-448, 448).reshape(y.shape), e


def _tiled_exact(v):
    """Scale values [m, kb] placed one by one at their positions in the 128 x 4 tiled layout."""
    m, kb = v.shape
    r, j = torch.arange(m, device=v.device)[:, None], torch.arange(kb, device=v.device)[None]
    tiles = -(-kb // 4)
    at = ((r // 128) * tiles + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4
    out = torch.full((-(-m // 128) * tiles * 512,), 2.0 ** -127, dtype=v.dtype, device=v.device)
    out[at.reshape(-1)] = v.reshape(-1)
    return out


def _products_exact(s, w, ws):
    c = s["case"]
    n, kb = c["n"], c["k"] // 32
    r, j = torch.arange(n, device=DEV)[:, None], torch.arange(kb, device=DEV)[None]
    tiles = -(-kb // 4)
    at = ((r // 128) * tiles + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4
    per = -(-n // 128) * tiles * 512
    x = _f8(s["codes"]).double() * torch.pow(2.0, s["scales"].double() - 127).repeat_interleave(32, 1)
    out = torch.zeros(c["rows"], n, dtype=torch.float64, device=DEV)
    off = s["offsets"].tolist()
    for e in range(c["experts"]):
        if off[e + 1] > off[e]:
            scale = torch.pow(2.0, ws[e * per:(e + 1) * per][at].double() - 127)
            m = _f8(w[e]).double() * scale.repeat_interleave(32, 1)
            out[off[e]:off[e + 1]] = x[off[e]:off[e + 1]] @ m.T
    return out


def exact(c, seed):
    s, op = prepare(c, seed), c["op"]
    if op == "norm":
        h = s["x"].double() + (0 if s["residual"] is None else s["residual"].double())
        rstd = 1 / torch.sqrt((h * h).sum(1) / c["k"] + EPS)
        y = h * rstd[:, None] * s["weight"].double()
        out = {"rstd": rstd}
        if c["fmt"].startswith("mx"):
            out["codes"], e = _mx_exact(y)
            v = torch.pow(2.0, e - 127)
            out["scales"] = _tiled_exact(v) if c["fmt"] == "mxfp8_swizzled" else v
        else:
            b = y.reshape(c["rows"], -1, 128)
            v = b.abs().max(dim=2).values / FMAX[c["fmt"]]
            out["codes"] = (b / v.clamp(min=1e-300)[:, :, None]).reshape(y.shape)
            out["scales"] = v
        if s["residual"] is not None:
            out["sum"] = h
        if c["bf16"]:
            out["y"] = y
        return out
    if op == "norm_grad":
        dy, h, w, r = s["dy"].double(), s["h"].double(), s["weight"].double(), s["rstd"].double()[:, None]
        inner = (dy * w * h).sum(1, keepdim=True) * r * r / c["k"]
        dx = r * (dy * w - h * inner) + (0 if s["dsum"] is None else s["dsum"].double())
        return {"dx": dx, "dweight": torch.einsum("rk,rk->k", dy, h * r)}
    if op in ("route", "route_grad"):
        if op == "route":
            ids = s["ids"].cpu()
            kept = (ids >= 0) & (ids < c["experts"])
            flat = torch.where(kept, ids, torch.tensor(c["experts"], dtype=ids.dtype)).reshape(-1).tolist()
            order = sorted(range(len(flat)), key=lambda i: flat[i])
            slot_of = [0] * len(flat)
            for at, i in enumerate(order):
                slot_of[i] = at
            slots, routed = torch.tensor(slot_of, device=DEV).reshape(ids.shape), int(kept.sum())
        else:
            slots, routed = s["slots"].long(), int(s["offsets"][-1])
        live = (slots < routed).double()
        total = torch.zeros(c["tokens"], c["k"], dtype=torch.float64, device=DEV)
        if op == "route":
            for j in range(c["topk"]):
                total += s["y"][slots[:, j]].double() * (live[:, j] * s["weights"][:, j].double())[:, None]
            src = torch.tensor(order, device=DEV) // c["topk"]
            out = {"offsets": None, "order": None, "slots": None, "out": total}
            if c["form"] == "bf16":
                out["rows"] = s["x"][src].double()
                out["rows"][routed:] = 0
            else:
                out["codes"], out["scales"] = _f8(s["codes"])[src].double(), torch.pow(2.0, s["scales"][src].double() - 127)
                out["codes"][routed:] = 0
                out["scales"][routed:] = 2.0 ** -127
            return out
        dout, dy = s["dout"].double(), torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)
        dw = torch.zeros(slots.shape, dtype=torch.float64, device=DEV)
        for j in range(c["topk"]):
            dy[slots[:, j]] = dout * (live[:, j] * s["weights"][:, j].double())[:, None]
            dw[:, j] = (dout * s["y"][slots[:, j]].double()).sum(1) * live[:, j]
            total += s["dxs"][slots[:, j]].double() * live[:, j, None]
        return {"dy": dy, "dweights": dw, "dx": total}
    if op == "experts":
        return _products_exact(s, s["w"], s["ws"])
    g, u = _products_exact(s, s["gate"], s["gs"]), _products_exact(s, s["up"], s["us"])
    codes, e = _mx_exact(g * torch.sigmoid(g) * u)
    return {"codes": codes, "scales": torch.pow(2.0, e - 127)}
