"""Operators around the transfer of gradients and weights, each in its plain form and as the library's calls.

What stands on the two sides of a weight transfer in reinforcement learning: the trainer scores the sampled tokens, takes
the gradient of that score, bounds the gradient's norm and sends it; the inference engine decodes a few tokens with the
expert weights that it was sent and reports the log probabilities of what it sampled, with the alternatives.

* ``score`` / ``score_grad``: log probabilities of given tokens with entropy and top alternatives, and the gradient;
* ``norm`` / ``clip``: the global norm of many gradient tensors, and the gradients clipped by it;
* ``moe``: a whole mixture-of-experts layer on MXFP8 weights for a few tokens.

``run`` with ``own`` false computes them with elementary torch operations in 32 bits; with ``own`` true it makes the
calls a user of the package makes.
"""
import math
import random

import torch

own = False

DEV = "cuda" if torch.cuda.is_available() else "cpu"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
NORM_EPS = 1e-6

# ---------------------------------------------------------------- cases ----


def listed():
    return [
        # one decode step of four requests: the sampled tokens' log probabilities and the twenty best alternatives
        {"name": "score_step", "op": "score", "rows": 4, "vocab": 151936, "stride": 151936, "type": "bf16", "top": 20,
         "entropy": False, "stats": False, "temperature": 1.0, "id_bits": 64},
        # a decode step of a large batch: logits in 32 bits, a padded vocabulary, sampled at another temperature
        {"name": "score_batch", "op": "score", "rows": 256, "vocab": 151669, "stride": 151936, "type": "fp32", "top": 5,
         "entropy": True, "stats": False, "temperature": 0.7, "id_bits": 64},
        # a trainer scores a micro-batch of rollouts: log probabilities, entropy and what the gradient needs
        {"name": "score_rollouts", "op": "score", "rows": 4096, "vocab": 151936, "stride": 151936, "type": "bf16", "top": 0,
         "entropy": True, "stats": True, "temperature": 1.0, "id_bits": 64},
        # the policy's gradient on a short ragged batch with an odd vocabulary and an entropy bonus
        {"name": "score_grad_odd", "op": "score_grad", "rows": 777, "vocab": 50257, "stride": 50257, "type": "fp32",
         "bonus": True, "temperature": 0.7, "id_bits": 32},
        # the policy's gradient on a micro-batch of rollouts
        {"name": "score_grad_long", "op": "score_grad", "rows": 4096, "vocab": 151936, "stride": 151936, "type": "bf16",
         "bonus": True, "temperature": 1.0, "id_bits": 64},
        # the gradients of an adapter's few small matrices
        {"name": "norm_few", "op": "norm", "tensors": 14, "elements": 1 << 20, "layout": "even", "type": "fp32",
         "scale": 1.0, "each": False},
        # one layer of 128 experts: three expert batches, four attention matrices, router and norms, each norm reported
        {"name": "norm_layer", "op": "norm", "tensors": 12, "elements": 623120640, "layout": "layer", "type": "bf16",
         "scale": 0.125, "each": True},
        # the sums of eight ranks' buckets, averaged and clipped into the buffers that go on
        {"name": "clip_buckets", "op": "clip", "tensors": 8, "elements": 8 * 13107200, "layout": "even", "type": "bf16",
         "out": "bf16", "scale": 0.125, "each": False},
        # a thousand ragged views of flat buffers, some in 16 and some in 32 bits, clipped into the optimizer's 32 bits
        {"name": "clip_ragged", "op": "clip", "tensors": 1000, "elements": 60000000, "layout": "ragged", "type": "mixed",
         "out": "fp32", "scale": 1.0, "each": True},
        # a single request's next token
        {"name": "moe_one", "op": "moe", "tokens": 1, "topk": 8, "experts": 128, "n": 768, "k": 2048, "drop": False,
         "id_bits": 64},
        # eight requests, some choices taken by other ranks
        {"name": "moe_eight", "op": "moe", "tokens": 8, "topk": 8, "experts": 128, "n": 768, "k": 2048, "drop": True,
         "id_bits": 32},
        # thirty-two requests
        {"name": "moe_batch", "op": "moe", "tokens": 32, "topk": 8, "experts": 128, "n": 768, "k": 2048, "drop": False,
         "id_bits": 64},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(max(hi, lo))))))))


def draw(rng):
    op = rng.choice(["score", "score", "score_grad", "norm", "clip", "clip", "moe", "moe", "moe"])
    if op in ("score", "score_grad"):
        vocab = _log(rng, 1000, 200000)
        kind = rng.choice(["bf16", "bf16", "fp32"])
        cap = 4096 * 151936 // (2 if kind == "fp32" else 1)
        stride = vocab if rng.random() < 0.6 else vocab + rng.choice([1, 8, 64 - vocab % 64, 267])
        c = {"op": op, "rows": _log(rng, 1, max(1, min(60000, cap // stride))), "vocab": vocab, "stride": stride,
             "type": kind, "temperature": rng.choice([1.0, 1.0, 0.6, 1.3]), "id_bits": rng.choice([32, 64])}
        if op == "score":
            c.update(top=rng.choice([0, 0, 1, 5, 8, 20, 32]), entropy=rng.random() < 0.6, stats=rng.random() < 0.5)
            if c["top"]:          # alternatives are asked for where tokens are generated
                c["rows"] = min(c["rows"], _log(rng, 1, 1024))
        else:
            c["bonus"] = rng.random() < 0.5
        return c
    if op in ("norm", "clip"):
        tensors = _log(rng, 1, 1500)
        c = {"op": op, "tensors": tensors, "elements": max(_log(rng, 10000, 200000000), 40 * tensors),
             "layout": rng.choice(["ragged", "ragged", "even"]), "type": rng.choice(["bf16", "fp32", "mixed"]),
             "scale": rng.choice([1.0, 0.125, 1 / 3]), "each": rng.random() < 0.4}
        if op == "clip":
            c["out"] = rng.choice(["bf16", "fp32"])
        return c
    k, n = (max(256, _log(rng, 256, 2560) // 32 * 32) for _ in range(2))
    topk = rng.choice([1, 2, 4, 6, 8])
    experts = max(topk, _log(rng, 4, 160))
    while experts * n * k > 128 * 768 * 2048:
        experts = max(topk, experts // 2)
    return {"op": op, "tokens": _log(rng, 1, max(1, min(32, 32 * 8 * 768 * 2048 // (topk * n * k)))), "topk": topk,
            "experts": experts, "n": n, "k": k, "drop": rng.random() < 0.3, "id_bits": rng.choice([32, 64])}


def work(c):
    op = c["op"]
    if op in ("score", "score_grad"):
        e, b = c["rows"] * c["vocab"], 2 if c["type"] == "bf16" else 4
        if op == "score":
            out = 4 + (4 if c["entropy"] else 0) + (8 if c["stats"] else 0) + 8 * c["top"]
            return {"bytes": e * b + c["rows"] * (c["id_bits"] // 8 + out), "flops": (6 if c["entropy"] else 4) * e}
        return {"bytes": 2 * e * b + c["rows"] * (c["id_bits"] // 8 + 12 + (8 if c["bonus"] else 0)), "flops": 6 * e}
    if op in ("norm", "clip"):
        size = {"bf16": 2, "fp32": 4}
        read = sum(n * size[t] for n, t in _shapes(c))
        write = sum(n for n, _ in _shapes(c)) * size[c["out"]] if op == "clip" else 0
        return {"bytes": read + write + 8 + (4 * c["tensors"] if c["each"] else 0),
                "flops": (3 if op == "clip" else 2) * c["elements"]}
    t, j, e, n, k = c["tokens"], c["topk"], c["experts"], c["n"], c["k"]
    active = e * (1 - (1 - j / e) ** t)
    return {"bytes": active * 3 * n * k * 33 / 32 + t * k * 33 / 32 + t * j * (c["id_bits"] // 8 + 4) + t * k * 2,
            "flops": 6 * t * j * n * k}


def _shapes(c):
    """Elements and type of each gradient tensor, the same for every seed."""
    count, total = c["tensors"], c["elements"]
    if c["layout"] == "layer":      # gate, up, down; q, k, v, o; router; norms of the rows, of queries and of keys
        sizes = [128 * 768 * 2048] * 3 + [4096 * 2048, 512 * 2048, 512 * 2048, 2048 * 4096, 128 * 2048, 2048, 2048, 128, 128]
    elif c["layout"] == "even":
        sizes = [total // count] * count
    else:                           # a few large matrices, many small ones, vectors; odd sizes
        rng = random.Random(total * 31 + count)
        share = [math.exp(rng.gauss(0, 2)) for _ in range(count)]
        sizes = [max(1, int(total * s / sum(share))) for s in share]
    kinds = ["bf16", "fp32"]
    return [(n, kinds[i % 3 == 2] if c["type"] == "mixed" else c["type"]) for i, n in enumerate(sizes)]


# --------------------------------------------------------------- inputs ----


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV)


def _logits(g, c):
    """Rows of a language model's last product: a broad bulk and some tokens far above it, in some rows one that takes
    nearly all; the last columns of some rows are masked, as a grammar does it."""
    rows, vocab, stride = c["rows"], c["vocab"], c["stride"]
    x = torch.empty(rows, stride, dtype=TYPES[c["type"]], device=DEV)
    step = max(1, (1 << 27) // stride)
    for r in range(0, rows, step):
        x[r:r + step] = _randn(g, min(step, rows - r), stride) * 2.5
    part = vocab // 24
    at = torch.arange(24, device=DEV) * part + torch.randint(0, part, (rows, 24), generator=g, device=DEV)
    x.scatter_(1, at, (6 + 4 * _randn(g, rows, 24) + 8 * (torch.rand(rows, 1, generator=g, device=DEV) < 0.2)).to(x.dtype))
    masked = (torch.rand(rows, generator=g, device=DEV) < 0.1).nonzero()[:, 0]
    x[masked, vocab // 2:] = float("-inf")
    best = x[:, :vocab].argmax(1, keepdim=True)
    likely = torch.rand(rows, 1, generator=g, device=DEV) < 0.6
    pick = torch.where(likely, best, at[:, 3:4])[:, 0]
    ignored = torch.rand(rows, generator=g, device=DEV) < 0.1
    ids = torch.where(ignored, torch.full_like(pick, -100), pick)
    return x[:, :vocab], ids.to(torch.int64 if c["id_bits"] == 64 else torch.int32)


def _stats64(x, temperature, step=256):
    """(largest logit, log of the sum of exp((x - largest) / T), entropy) of each row, in 64 bits."""
    m, s, h = [], [], []
    for r in range(0, x.shape[0], step):
        v = x[r:r + step].double()
        top = v.max(1).values
        z = (v - top[:, None]) / temperature
        e = torch.exp(z)
        total = e.sum(1)
        m.append(top)
        s.append(torch.log(total))
        h.append(torch.log(total) - (e * z.clamp(min=-1e4)).sum(1) / total)
    return torch.cat(m), torch.cat(s), torch.cat(h)


def _gradients(g, c):
    """The tensors as views of one flat buffer per type, each of its own magnitude, some values far above the rest."""
    shapes = _shapes(c)
    flat, views = {}, []
    for t in ("bf16", "fp32"):
        total = sum(n for n, kind in shapes if kind == t)
        flat[t] = torch.empty(total, dtype=TYPES[t], device=DEV)
        for r in range(0, total, 1 << 26):
            part = _randn(g, min(1 << 26, total - r)) * 1e-4
            part[::1009] *= 30
            flat[t][r:r + (1 << 26)] = part
    at = {"bf16": 0, "fp32": 0}
    for i, (n, t) in enumerate(shapes):
        v = flat[t][at[t]:at[t] + n]
        if i % 4 == 1:
            v.mul_(4.0)
        views.append(v)
        at[t] += n
    return views


def _mx_quantize(x):
    """x [..., k] -> e4m3 codes and E8M0 bytes [..., k/32] by the rules of MXFP8 (uint8)."""
    b = x.unflatten(-1, (-1, 32))
    amax = b.abs().amax(-1)
    e = (torch.frexp(amax).exponent.to(torch.int64) - 1 - 8 + 127).clamp(0, 254)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    q = torch.ldexp(b, (127 - e).to(torch.int32)[..., None]).clamp(-448, 448).flatten(-2)
    return q.to(torch.float8_e4m3fn).view(torch.uint8), e.to(torch.uint8)


def _tile(s):
    """E8M0 bytes [experts, m, kb] -> the 128 x 4 tiled layout of block-scaled products, flat, padding 0."""
    e, m, kb = s.shape
    r, c = -(-m // 128), -(-kb // 4)
    t = torch.zeros(e, r * 128, c * 4, dtype=s.dtype, device=s.device)
    t[:, :m, :kb] = s
    return t.reshape(e, r, 4, 32, c, 4).permute(0, 1, 4, 3, 2, 5).reshape(-1)


def _untile(s, experts, m, kb):
    r, c = -(-m // 128), -(-kb // 4)
    t = s.reshape(experts, r, c, 32, 4, 4).permute(0, 1, 4, 3, 2, 5).reshape(experts, r * 128, c * 4)
    return t[:, :m, :kb]


def _expert_weights(g, experts, n, k):
    codes, scales = zip(*(_mx_quantize(_randn(g, n, k) * (0.7 / k ** 0.5)) for _ in range(experts)))
    return torch.stack(codes), _tile(torch.stack(scales))


def prepare(c, seed):
    g, op = _gen(seed), c["op"]
    s = {"case": c}
    if op in ("score", "score_grad"):
        s["logits"], s["ids"] = _logits(g, c)
        if op == "score_grad":
            m, total, h = _stats64(s["logits"], c["temperature"])
            s["stats"] = torch.stack([m, total], 1).float()
            s["dlogprobs"] = _randn(g, c["rows"]) / c["rows"] ** 0.5
            s["entropy"], s["dentropy"] = (h.float(), torch.full((c["rows"],), -0.01, device=DEV)) if c["bonus"] else (None, None)
    elif op in ("norm", "clip"):
        s["grads"] = _gradients(g, c)
        # about twice as large as allowed, as a clipped step is
        size = math.sqrt(sum(n * (16 if i % 4 == 1 else 1) for i, (n, _) in enumerate(_shapes(c)))) * 1e-4 * c["scale"]
        s["max_norm"] = 0.5 * size
        if op == "clip":
            # one flat buffer, the tensors one after the other
            s["flat"] = torch.empty(sum(t.numel() for t in s["grads"]), dtype=TYPES[c["out"]], device=DEV)
            s["outs"] = list(s["flat"].split([t.numel() for t in s["grads"]]))
        if own:
            import weight_transfer_gb300 as fp8q
            s["list"] = fp8q.fp8q_grad_list(s["grads"], s.get("outs"))
    else:
        t, j, e = c["tokens"], c["topk"], c["experts"]
        noise = -torch.log(-torch.log(torch.rand(t, e, generator=g, device=DEV).clamp(1e-9, 1 - 1e-7)))
        score, ids = torch.topk(torch.log_softmax(0.5 * _randn(g, e), 0) + noise, j, dim=1)
        if c["drop"]:
            ids = torch.where(torch.rand(t, j, generator=g, device=DEV) < 0.15, torch.full_like(ids, -1), ids)
            if t > 2:
                ids[t // 2] = -1          # a token that none of these experts takes
        s["ids"] = ids.to(torch.int64 if c["id_bits"] == 64 else torch.int32)
        s["weights"] = torch.softmax(score, 1)
        loud = 1 + 19 * (torch.rand(c["k"], generator=g, device=DEV) < 0.01)
        s["codes"], s["scales"] = _mx_quantize(_randn(g, t, c["k"]) * loud)
        s["gate"], s["up"] = (_expert_weights(g, e, c["n"], c["k"]) for _ in range(2))
        s["down"] = _expert_weights(g, e, c["k"], c["n"])
    return s


# ----------------------------------------------------------- plain form ----


def _pick(z, ids):
    """z[r, ids[r]], and whether ids[r] names a column."""
    live = (ids >= 0) & (ids < z.shape[1])
    return z.gather(1, torch.where(live, ids, 0).long()[:, None])[:, 0], live


def _score_plain(s):
    c = s["case"]
    x = s["logits"].float()
    m = x.amax(1, keepdim=True)
    z = (x - m) / c["temperature"]
    e = torch.exp(z)
    total = e.sum(1)
    log_total = torch.log(total)
    at, live = _pick(z, s["ids"])
    out = {"logprobs": torch.where(live, at - log_total, 0.0)}
    if c["entropy"]:
        out["entropy"] = log_total - torch.where(e > 0, e * z, 0.0).sum(1) / total
    if c["stats"]:
        out["stats"] = torch.stack([m[:, 0], log_total], 1)
    if c["top"]:
        bits = (x + 0.0).contiguous().view(torch.int32)
        rank = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).long()
        key = (rank << 32) | (0x7FFFFFFF - torch.arange(c["vocab"], device=x.device))     # ties to the lowest index
        ids = 0x7FFFFFFF - (torch.topk(key, c["top"], dim=1).values & 0x7FFFFFFF)
        out["top_ids"] = ids.to(torch.int32)
        out["top_logprobs"] = z.gather(1, ids) - log_total[:, None]
    return out


def _score_grad_plain(s):
    c = s["case"]
    m, log_total = s["stats"][:, :1], s["stats"][:, 1:]
    logp = (s["logits"].float() - m) / c["temperature"] - log_total
    p = torch.exp(logp)
    live = (s["ids"] >= 0) & (s["ids"] < c["vocab"])
    dlogp = torch.where(live, s["dlogprobs"], 0.0)
    d = p * -dlogp[:, None]
    if c["bonus"]:
        d = d - torch.where(p > 0, p * (logp + s["entropy"][:, None]), 0.0) * s["dentropy"][:, None]
    d.scatter_add_(1, torch.where(live, s["ids"], 0).long()[:, None], dlogp[:, None])
    return (d / c["temperature"]).to(s["logits"].dtype)


def _norm_plain(s):
    c = s["case"]
    squares = torch.stack([t.float().square().sum() for t in s["grads"]])
    norm = torch.sqrt(squares.sum()) * c["scale"]
    coefficient = torch.clamp(s["max_norm"] / (norm + NORM_EPS), max=1.0)
    out = {"norm": torch.stack([norm, coefficient])}
    if c["each"]:
        out["each"] = torch.sqrt(squares) * c["scale"]
    return out


def _clip_plain(s):
    out = _norm_plain(s)
    factor = out["norm"][1] * s["case"]["scale"]
    for t, o in zip(s["grads"], s["outs"]):
        o.copy_(t.float() * factor)
    out["flat"] = s["flat"]
    return out


def _mx_values(codes, scales):
    v = codes.view(torch.float8_e4m3fn).float().unflatten(-1, (-1, 32))
    return torch.ldexp(v, (scales.to(torch.int32) - 127)[..., None]).flatten(-2)


def _moe_plain(s):
    c = s["case"]
    t, j, e, n, k = c["tokens"], c["topk"], c["experts"], c["n"], c["k"]
    x = _mx_values(s["codes"], s["scales"]).repeat_interleave(j, 0)
    ids = s["ids"].reshape(-1).long()
    live = (ids >= 0) & (ids < e)
    scales = [_untile(s[w][1], e, *shape) for w, shape in (("gate", (n, k // 32)), ("up", (n, k // 32)), ("down", (k, n // 32)))]
    y = []
    for r in range(0, t * j, 32):             # 32 choices' matrices at a time
        at = torch.where(live, ids, 0)[r:r + 32]
        gate, up, down = (_mx_values(s[w][0][at], sc[at]) for w, sc in zip(("gate", "up", "down"), scales))
        a = x[r:r + 32, :, None]
        g, u = torch.bmm(gate, a), torch.bmm(up, a)
        y.append(torch.bmm(down, g / (1 + torch.exp(-g)) * u)[:, :, 0])
    y = torch.where(live[:, None], torch.cat(y) * s["weights"].reshape(-1, 1), 0.0)
    return y.view(t, j, k).sum(1).bfloat16()


# ------------------------------------------------------ the library's calls ----


def _score_own(s):
    import weight_transfer_gb300 as fp8q
    c = s["case"]
    logprobs, entropy, top_logprobs, top_ids, stats = fp8q.fp8q_token_logprobs(
        s["logits"], s["ids"], temperature=c["temperature"], top=c["top"], want_entropy=c["entropy"], want_stats=c["stats"])
    out = {"logprobs": logprobs}
    if c["entropy"]:
        out["entropy"] = entropy
    if c["stats"]:
        out["stats"] = stats
    if c["top"]:
        out["top_ids"], out["top_logprobs"] = top_ids, top_logprobs
    return out


def _score_grad_own(s):
    import weight_transfer_gb300 as fp8q
    return fp8q.fp8q_token_logprobs_backward(s["logits"], s["ids"], s["stats"], s["dlogprobs"], entropy=s["entropy"],
                                             dentropy=s["dentropy"], temperature=s["case"]["temperature"])


def _norm_own(s):
    import weight_transfer_gb300 as fp8q
    c = s["case"]
    norm, each = fp8q.fp8q_grad_norm(s["list"], s["max_norm"], scale=c["scale"], want_each=c["each"])
    return {"norm": norm, "each": each} if c["each"] else {"norm": norm}


def _clip_own(s):
    import weight_transfer_gb300 as fp8q
    c = s["case"]
    norm, each = fp8q.fp8q_grad_clip(s["list"], s["max_norm"], scale=c["scale"], want_each=c["each"])
    out = {"norm": norm, "each": each} if c["each"] else {"norm": norm}
    return {**out, "flat": s["flat"]}


def _moe_own(s):
    import weight_transfer_gb300 as fp8q
    return fp8q.mxfp8_moe_decode(s["codes"], s["scales"], s["ids"], s["weights"], *s["gate"], *s["up"], *s["down"])


_PLAIN = {"score": _score_plain, "score_grad": _score_grad_plain, "norm": _norm_plain, "clip": _clip_plain, "moe": _moe_plain}
_OWN = {"score": _score_own, "score_grad": _score_grad_own, "norm": _norm_own, "clip": _clip_own, "moe": _moe_own}


def run(s):
    return (_OWN if own else _PLAIN)[s["case"]["op"]](s)


# ------------------------------------------------------------- in 64 bits ----


def _score_exact(c, s):
    x, ids = s["logits"], s["ids"].long()
    m, log_total, h = _stats64(x, c["temperature"])
    rows = torch.arange(c["rows"], device=DEV)
    named = (ids >= 0) & (ids < c["vocab"])
    own_logit = x[rows, ids.clamp(0, c["vocab"] - 1)].double()
    out = {"logprobs": torch.where(named, (own_logit - m) / c["temperature"] - log_total, 0.0)}
    if c["entropy"]:
        out["entropy"] = h
    if c["stats"]:
        out["stats"] = torch.stack([m, log_total], 1)
    if c["top"]:
        best = [torch.sort(x[r:r + 64].double(), dim=1, descending=True, stable=True) for r in range(0, c["rows"], 64)]
        values = torch.cat([b.values[:, :c["top"]] for b in best])
        out["top_ids"] = torch.cat([b.indices[:, :c["top"]] for b in best]).to(torch.int32)
        out["top_logprobs"] = (values - m[:, None]) / c["temperature"] - log_total[:, None]
    return out


def _score_grad_exact(c, s):
    # d logp[t] / dz_j = [j = t] - p_j,  d entropy / dz_j = -p_j * (log p_j + entropy),  z = x / T
    out = torch.empty(c["rows"], c["vocab"], dtype=torch.float64, device=DEV)
    for r in range(0, c["rows"], 256):
        cut = slice(r, min(r + 256, c["rows"]))
        z = s["logits"][cut].double() / c["temperature"]
        lse = s["stats"][cut, :1].double() / c["temperature"] + s["stats"][cut, 1:].double()
        p = torch.exp(z - lse)
        ids = s["ids"][cut].long()
        named = (ids >= 0) & (ids < c["vocab"])
        up = s["dlogprobs"][cut].double() * named
        d = -p * up[:, None]
        d[torch.arange(d.shape[0], device=DEV)[named], ids[named]] += up[named]
        if c["bonus"]:
            d -= s["dentropy"][cut].double()[:, None] * p * ((z - lse).clamp(min=-1e4) + s["entropy"][cut].double()[:, None])
        out[cut] = d / c["temperature"]
    return out


def _norm_exact(c, s):
    squares = []
    for t in s["grads"]:
        parts = [t[r:r + (1 << 26)].double() for r in range(0, t.numel(), 1 << 26)]
        squares.append(sum(torch.dot(p, p) for p in parts))
    squares = torch.stack(squares)
    norm = torch.sqrt(squares.sum()) * c["scale"]
    coefficient = torch.minimum(s["max_norm"] / (norm + NORM_EPS), torch.ones_like(norm))
    out = {"norm": torch.stack([norm, coefficient])}
    if c["each"]:
        out["each"] = torch.sqrt(squares) * c["scale"]
    if c["op"] == "clip":
        out["flat"] = torch.cat([t.double() * (coefficient * c["scale"]) for t in s["grads"]])
    return out


def _moe_exact(c, s):
    def matrix(name, expert, rows, cols):
        kb = cols // 32
        r, j = torch.arange(rows, device=DEV)[:, None], torch.arange(kb, device=DEV)[None]
        tiles = -(-kb // 4)
        at = ((r // 128) * tiles + j // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + j % 4
        per = -(-rows // 128) * tiles * 512
        scale = torch.pow(2.0, s[name][1][expert * per:(expert + 1) * per][at].double() - 127)
        return s[name][0][expert].view(torch.float8_e4m3fn).double() * scale.repeat_interleave(32, 1)

    x = s["codes"].view(torch.float8_e4m3fn).double() * torch.pow(2.0, s["scales"].double() - 127).repeat_interleave(32, 1)
    ids, n, k = s["ids"].tolist(), c["n"], c["k"]
    out = torch.zeros(c["tokens"], k, dtype=torch.float64, device=DEV)
    for e in sorted({i for row in ids for i in row if 0 <= i < c["experts"]}):
        who = [(t, j) for t, row in enumerate(ids) for j, i in enumerate(row) if i == e]
        rows = x[[t for t, _ in who]]
        g, u = rows @ matrix("gate", e, n, k).T, rows @ matrix("up", e, n, k).T
        y = (g * torch.sigmoid(g) * u) @ matrix("down", e, k, n).T
        for (t, j), row in zip(who, y):
            out[t] += row * s["weights"][t, j].double()
    return out


_EXACT = {"score": _score_exact, "score_grad": _score_grad_exact, "norm": _norm_exact, "clip": _norm_exact, "moe": _moe_exact}


def exact(c, seed):
    return _EXACT[c["op"]](c, prepare(c, seed))
