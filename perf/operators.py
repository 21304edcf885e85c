"""Measured cases of the finetuning operators that run around the NF4 + LoRA linear layers.

Causal or full attention over dense or packed batches (forward with the row statistics, and the backward pass that recomputes
the probabilities from them), layer norm and root-mean-square norm (forward, and backward with the weight's gradient), and the
clipping of all adapters' gradients by their global norm.

`run` has every operator twice: in plain torch operations held in 32 bits (`own` false) and through this package's entry points
(`own` true).  `exact` is the same in 64 bits, written from the definitions.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}


# ---------------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------------

def _attn(op, seqs, lq, lk, heads, kv_heads, dim, causal=True, fused=False):
    """A dense batch: `seqs` sequences of lq queries and lk keys.  `fused`: q, k and v are views of one projection's output."""
    return {"op": op, "layout": "dense", "seqs": seqs, "lq": lq, "lk": lk, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "causal": causal, "fused": fused}


def _packed(op, seqs, tokens, heads, kv_heads, dim, causal=True, fused=False):
    """A packed batch: `tokens` tokens in `seqs` sequences of unequal length, one after the other."""
    return {"op": op, "layout": "packed", "seqs": seqs, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "causal": causal, "fused": fused}


def _norm(op, rows, width, dtype, rms=False):
    return {"op": op, "rows": rows, "width": width, "dtype": dtype, "rms": rms}


def _clip(layers, hidden, inner, rank, dtype, max_norm):
    """The adapter gradients of `layers` decoder blocks: A [rank, K] and B [N, rank] of q, k, v, o, gate, up and down."""
    return {"op": "clip", "layers": layers, "hidden": hidden, "inner": inner, "rank": rank, "dtype": dtype, "max_norm": max_norm}


def listed():
    return [
        # the 4096-token step (8 x 512) of the 32-head, 4096-wide layers that the benchmark times
        dict(_attn("attn_fwd", 8, 512, 512, 32, 32, 128), name="attn_fwd_8x512"),
        # one long document with shared key/value heads, straight from a fused projection
        dict(_attn("attn_fwd", 1, 8192, 8192, 32, 8, 128, fused=True), name="attn_fwd_1x8192_gqa"),
        # a short instruction of odd length: the time of a call
        dict(_attn("attn_bwd", 1, 67, 67, 16, 16, 64), name="attn_bwd_1x67"),
        # the same step's backward pass
        dict(_attn("attn_bwd", 8, 512, 512, 32, 32, 128), name="attn_bwd_8x512"),
        # examples of unequal length packed into one row, 40 heads as in the 5120-wide block
        dict(_packed("attn_bwd", 17, 8191, 40, 40, 128), name="attn_bwd_packed_8191"),
        # the long document's backward pass
        dict(_attn("attn_bwd", 1, 8192, 8192, 32, 8, 128), name="attn_bwd_1x8192_gqa"),
        # one token: the smallest call there is
        dict(_norm("norm_fwd", 1, 4096, "bf16"), name="norm_fwd_1x4096"),
        # the benchmark's step, in the residual stream's type
        dict(_norm("norm_fwd", 4096, 4096, "bf16"), name="norm_fwd_4096x4096"),
        # norms kept in 32 bits, as finetuning of quantized bases commonly does, an odd count of tokens
        dict(_norm("norm_bwd", 2047, 5120, "fp32"), name="norm_bwd_2047x5120_fp32"),
        # the widest layers of the benchmark, root-mean-square form
        dict(_norm("norm_bwd", 8192, 8192, "bf16", rms=True), name="norm_bwd_8192x8192_rms"),
        # one small block with rank 8: the time of a call over 14 tensors
        dict(_clip(1, 1024, 2730, 8, "fp32", 0.3), name="clip_1_block_r8"),
        # every adapter of a 32-block model at rank 64: 448 tensors
        dict(_clip(32, 4096, 11008, 64, "bf16", 0.3), name="clip_32_blocks_r64"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        c = _draw(rng)
        if _cost(c) <= top and _memory(c) <= 12e9:
            return c


def _draw(rng):
    op = rng.choice(["attn_fwd", "attn_fwd", "attn_bwd", "attn_bwd", "norm_fwd", "norm_bwd", "clip"])
    if op.startswith("attn"):
        kv = rng.choice([1, 2, 4, 5, 8, 16, 32])
        heads = kv * rng.choice([g for g in (1, 1, 2, 4, 8) if kv * g <= 40])
        dim, causal, fused = rng.choice([64, 80, 96, 128, 128]), rng.random() < 0.75, rng.random() < 0.5
        shape = rng.choice(["square", "square", "packed", "packed", "cross"])
        if shape == "packed":
            tokens = _log(rng, 64, 16384)
            return _packed(op, _log(rng, 1, min(128, tokens)), tokens, heads, kv, dim, causal, fused)
        lq = _log(rng, 1, 8192)
        # "cross": queries that are the end of a longer sequence, or that look at another one
        # (two keys at least, and two tokens: over one key the gradients of q and k are zero but for rounding)
        lq = max(lq, 2) if shape == "square" else lq
        lk = lq if shape == "square" else _log(rng, 2, 8192)
        return _attn(op, max(1, min(64, int(rng.uniform(0.2, 1.0) * 16384 / max(lq, lk)))), lq, lk, heads, kv, dim, causal,
                     fused and lq == lk)
    if op.startswith("norm"):
        return _norm(op, _log(rng, 1, 16384), _log(rng, 33, 16384), rng.choice(["bf16", "fp32"]), rng.random() < 0.5)
    hidden = _log(rng, 128, 8192)
    return _clip(_log(rng, 1, 48), hidden, int(hidden * rng.uniform(2.0, 4.0)), _log(rng, 1, 128),
                 rng.choice(["bf16", "fp32"]), rng.choice([0.3, 1.0, 1e6]))


def _lengths(case):
    """The lengths of a packed batch's sequences: cut points that follow from the case alone."""
    rng = random.Random("%d tokens in %d" % (case["tokens"], case["seqs"]))
    cuts = sorted(rng.randrange(case["tokens"] + 1) for _ in range(case["seqs"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["tokens"]])]


def _pairs(lq, lk, causal):
    """Query/key pairs that the mask leaves: the last query sees the last key."""
    if not causal:
        return lq * lk
    first = max(0, lq - lk)  # queries before this one see nothing
    n = lq - first
    return n * (lk - lq + first + 1) + n * (n - 1) // 2


def _adapters(case):
    h, m, r = case["hidden"], case["inner"], case["rank"]
    block = []
    for n, k in ((h, h), (h, h), (h, h), (h, h), (m, h), (m, h), (h, m)):
        block += [(r, k), (n, r)]
    return block * case["layers"]


def work(case):
    op = case["op"]
    if op == "clip":
        n = sum(a * b for a, b in _adapters(case))
        return {"bytes": 2 * n * BYTES[case["dtype"]], "flops": 3 * n}
    if op.startswith("norm"):
        n, e = case["rows"] * case["width"], BYTES[case["dtype"]]
        if op == "norm_fwd":
            return {"bytes": 2 * n * e + 8 * case["rows"] + 2 * case["width"] * e, "flops": 8 * n}
        return {"bytes": 3 * n * e + 8 * case["rows"] + 3 * case["width"] * e, "flops": 14 * n}
    if case["layout"] == "packed":
        lens = _lengths(case)
        tq = tk = case["tokens"]
        pairs = sum(_pairs(n, n, case["causal"]) for n in lens)
    else:
        tq, tk = case["seqs"] * case["lq"], case["seqs"] * case["lk"]
        pairs = case["seqs"] * _pairs(case["lq"], case["lk"], case["causal"])
    rows_q, rows_k = tq * case["heads"] * case["dim"] * 2, tk * case["kv_heads"] * case["dim"] * 2
    stats = tq * case["heads"] * 4
    if op == "attn_fwd":
        return {"bytes": 2 * rows_q + 2 * rows_k + stats, "flops": 4 * pairs * case["dim"] * case["heads"]}
    return {"bytes": 4 * rows_q + 4 * rows_k + stats, "flops": 10 * pairs * case["dim"] * case["heads"]}


def _cost(case):
    w = work(case)
    return w["bytes"] / 4e12 + w["flops"] / 400e12


def _memory(case):
    """Bytes of one 32-bit score matrix of the plain form."""
    if not case["op"].startswith("attn"):
        return 0
    if case["layout"] == "packed":
        return case["seqs"] * case["heads"] * max(_lengths(case)) ** 2 * 4
    return case["seqs"] * case["heads"] * case["lq"] * case["lk"] * 4


# ---------------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    if case["op"] == "clip":
        dt = DTYPES[case["dtype"]]
        # gradients of very unequal size, as A's and B's are
        s["grads"] = [normal(a, b, std=3e-4 * (1 + i % 5), dtype=dt) for i, (a, b) in enumerate(_adapters(case))]
        # the optimizer's flat buffer that takes them, one after the other
        s["flat"] = torch.empty(sum(t.numel() for t in s["grads"]), dtype=dt, device="cuda")
        return s
    if case["op"].startswith("norm"):
        dt = DTYPES[case["dtype"]]
        rows, width = case["rows"], case["width"]
        # a residual stream: a common offset, and a few channels that are much larger than the rest
        chan = 1.0 + 9.0 * (torch.rand(width, generator=g, device="cuda") < 0.01).float()
        s["x"] = (torch.randn(rows, width, generator=g, device="cuda") * 2.0 * chan + 0.25).to(dt)
        s["weight"] = (1.0 + 0.2 * torch.randn(width, generator=g, device="cuda")).to(dt)
        s["bias"] = None if case["rms"] else normal(width, std=0.1, dtype=dt)
        s["eps"] = 1e-5
        if case["op"] == "norm_bwd":
            s["dy"] = normal(rows, width, std=1e-2, dtype=dt)
            _, s["mean"], s["rstd"] = _plain_norm_fwd(s["x"], s["weight"], s["bias"], s["eps"], case["rms"])
        return s
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["layout"] == "packed":
        lens = _lengths(case)
        s["lens"] = lens
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
        lead_q = lead_k = (case["tokens"],)
    else:
        s["cu"] = None
        lead_q, lead_k = (case["seqs"], case["lq"]), (case["seqs"], case["lk"])
    if case["fused"]:
        qkv = normal(*lead_q, h + 2 * hk, d)
        s["q"], s["k"], s["v"] = qkv.split([h, hk, hk], dim=-2)
    else:
        s["q"], s["k"], s["v"] = normal(*lead_q, h, d), normal(*lead_k, hk, d), normal(*lead_k, hk, d)
    s["q"].mul_(1.5)  # scores with a spread of 1.5: some keys matter much more than others
    s["scale"] = 1.0 / math.sqrt(d)
    if case["op"] == "attn_bwd":
        s["do"] = normal(*lead_q, h, d, std=1e-2)
        o, lse = _plain_attn_fwd(s)
        s["o"], s["lse"] = o, lse
    return s


# ---------------------------------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------------------------------

def _rows(s):
    """Packed batches: the padded [sequence, position] -> token index and which of those positions exist."""
    lens = (s["cu"][1:] - s["cu"][:-1]).long()
    pos = torch.arange(max(s["lens"]), device="cuda")
    there = pos[None, :] < lens[:, None]
    return torch.where(there, s["cu"][:-1, None].long() + pos[None, :], 0), there


def _heads(t, kv_heads, index):
    """[batch, kv head, group, position, dim] in 32 bits."""
    t = t.float()
    if index is not None:
        t = t[index]
    b, n, h, d = t.shape
    return t.reshape(b, n, kv_heads, h // kv_heads, d).permute(0, 2, 3, 1, 4)


def _back(s, t, heads, there):
    """The other way, rounded once."""
    b, hk, g, n, d = t.shape
    t = t.permute(0, 3, 1, 2, 4).reshape(b, n, heads, d)
    return (t if there is None else t[there]).to(torch.bfloat16)


def _scores(s, q, k, there):
    x = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    lq, lk = q.shape[-2], k.shape[-2]
    if there is not None:
        # queries and keys of a packed batch are the same tokens
        x = x.masked_fill(~there[:, None, None, None, :], -math.inf)
    if s["case"]["causal"]:
        i, j = torch.arange(lq, device="cuda"), torch.arange(lk, device="cuda")
        x = x.masked_fill(j[None, :] > i[:, None] + (lk - lq), -math.inf)
    return x


def _plain_attn_fwd(s):
    hk = s["case"]["kv_heads"]
    index, there = _rows(s) if s["cu"] is not None else (None, None)
    q, k, v = (_heads(s[n], hk, index) for n in ("q", "k", "v"))
    x = _scores(s, q, k, there)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x, v) / torch.where(total == 0, 1.0, total)
    lse = (top + torch.log(total)).squeeze(-1)
    b, _, g, n = lse.shape
    lse = lse.reshape(b, hk * g, n)
    if there is not None:
        lse = lse.transpose(0, 1)[:, there]
    return _back(s, o, hk * g, there), lse.contiguous()


def _plain_attn_bwd(s):
    hk, heads = s["case"]["kv_heads"], s["case"]["heads"]
    index, there = _rows(s) if s["cu"] is not None else (None, None)
    q, k, v, o, do = (_heads(s[n], hk, index) for n in ("q", "k", "v", "o", "do"))
    lse = s["lse"] if there is None else s["lse"][:, index].transpose(0, 1)
    lse = lse.reshape(lse.shape[0], hk, heads // hk, -1, 1)
    p = torch.exp(_scores(s, q, k, there) - torch.where(lse == -math.inf, 0.0, lse))
    if there is not None:
        p = p.masked_fill(~there[:, None, None, :, None], 0.0)
    dv = torch.matmul(p.transpose(-1, -2), do).sum(2, keepdim=True)
    ds = p * (torch.matmul(do, v.transpose(-1, -2)) - (do * o).sum(-1, keepdim=True)) * s["scale"]
    dq = torch.matmul(ds, k)
    dk = torch.matmul(ds.transpose(-1, -2), q).sum(2, keepdim=True)
    return _back(s, dq, heads, there), _back(s, dk, hk, there), _back(s, dv, hk, there)


def _plain_norm_fwd(x, weight, bias, eps, rms):
    x32 = x.float()
    mean = None if rms else x32.mean(-1)
    c = x32 if rms else x32 - mean[:, None]
    rstd = torch.rsqrt((c * c).mean(-1) + eps)
    y = c * rstd[:, None] * weight.float()
    return (y if bias is None else y + bias.float()).to(x.dtype), mean, rstd


def _plain_norm_bwd(dy, x, weight, mean, rstd, rms):
    xhat = (x.float() if rms else x.float() - mean[:, None]) * rstd[:, None]
    dy32 = dy.float()
    g = dy32 * weight.float()
    dx = g - xhat * (g * xhat).mean(-1, keepdim=True)
    if not rms:
        dx = dx - g.mean(-1, keepdim=True)
    dx = dx * rstd[:, None]
    dw = (dy32 * xhat).sum(0)
    return dx.to(x.dtype), dw.to(weight.dtype), None if rms else dy32.sum(0).to(weight.dtype)


def _plain_clip(grads, max_norm):
    flat = torch.cat([g.flatten() for g in grads]).float()
    norm = (flat * flat).sum().sqrt().reshape(1)
    return norm, (flat * torch.clamp(max_norm / (norm + 1e-6), max=1.0)).to(grads[0].dtype)


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import quantized_base_lora_nf4_amd as qn
        if op == "attn_fwd":
            o, lse = qn.attention_fwd(s["q"], s["k"], s["v"], causal=case["causal"], scale=s["scale"], cu_seqlens=s["cu"])
            return {"o": o, "lse": lse}
        if op == "attn_bwd":
            dq, dk, dv = qn.attention_bwd(s["q"], s["k"], s["v"], s["o"], s["lse"], s["do"], causal=case["causal"],
                                          scale=s["scale"], cu_seqlens=s["cu"])
            return {"dq": dq, "dk": dk, "dv": dv}
        if op == "norm_fwd":
            y, mean, rstd = qn.norm_fwd(s["x"], s["weight"], s["bias"], eps=s["eps"], rms=case["rms"])
            return {"y": y, "rstd": rstd} if case["rms"] else {"y": y, "mean": mean, "rstd": rstd}
        if op == "norm_bwd":
            dx, dw, db = qn.norm_bwd(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], rms=case["rms"])
            return {"dx": dx, "dw": dw} if case["rms"] else {"dx": dx, "dw": dw, "db": db}
        norm = qn.clip_grad_norm(s["grads"], case["max_norm"], out=s["flat"])
        return {"norm": norm, "grads": s["flat"]}
    if op == "attn_fwd":
        o, lse = _plain_attn_fwd(s)
        return {"o": o, "lse": lse}
    if op == "attn_bwd":
        dq, dk, dv = _plain_attn_bwd(s)
        return {"dq": dq, "dk": dk, "dv": dv}
    if op == "norm_fwd":
        y, mean, rstd = _plain_norm_fwd(s["x"], s["weight"], s["bias"], s["eps"], case["rms"])
        return {"y": y, "rstd": rstd} if case["rms"] else {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        dx, dw, db = _plain_norm_bwd(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"], case["rms"])
        return {"dx": dx, "dw": dw} if case["rms"] else {"dx": dx, "dw": dw, "db": db}
    norm, grads = _plain_clip(s["grads"], case["max_norm"])
    return {"norm": norm, "grads": grads}


# ---------------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        flat = torch.cat([t.double().flatten() for t in s["grads"]])
        norm = torch.linalg.vector_norm(flat)
        factor = min(1.0, case["max_norm"] / (float(norm) + 1e-6))
        return {"norm": norm.reshape(1), "grads": flat * factor}
    if op.startswith("norm"):
        x, w = s["x"].double(), s["weight"].double()
        mu = torch.zeros_like(x[:, :1]) if case["rms"] else x.sum(1, keepdim=True) / case["width"]
        sigma = ((x - mu).square().sum(1, keepdim=True) / case["width"] + s["eps"]).sqrt()
        z = (x - mu) / sigma
        if op == "norm_fwd":
            y = z * w if s["bias"] is None else z * w + s["bias"].double()
            return {"y": y, "rstd": 1 / sigma[:, 0]} if case["rms"] else {"y": y, "mean": mu[:, 0], "rstd": 1 / sigma[:, 0]}
        dy = s["dy"].double()
        dz = dy * w
        # the Jacobian of z: (1 - z z^T / n - [1 1^T / n]) / sigma
        dx = dz - z * (z * dz).sum(1, keepdim=True) / case["width"]
        if not case["rms"]:
            dx -= dz.sum(1, keepdim=True) / case["width"]
        out = {"dx": dx / sigma, "dw": (dy * z).sum(0)}
        return out if case["rms"] else {**out, "db": dy.sum(0)}
    return _exact_attn(case, s)


def _exact_attn(case, s):
    """One sequence and one head after the other."""
    h, d = case["heads"], case["dim"]
    share = h // case["kv_heads"]
    if case["layout"] == "packed":
        ends = s["cu"].tolist()
        spans = [(slice(a, b),) * 2 for a, b in zip(ends, ends[1:]) if b > a]
        flat = {n: s[n] for n in ("q", "k", "v", "do") if n in s}
    else:
        spans = [(slice(i * case["lq"], (i + 1) * case["lq"]), slice(i * case["lk"], (i + 1) * case["lk"])) for i in range(case["seqs"])]
        flat = {n: s[n].reshape(-1, *s[n].shape[2:]) for n in ("q", "k", "v", "do") if n in s}
    if len(spans) * h > 6000:
        return None
    new = lambda t: torch.zeros(t.shape, dtype=torch.float64, device="cuda")  # noqa: E731
    o, dq, dk, dv = new(flat["q"]), new(flat["q"]), new(flat["k"]), new(flat["v"])
    lse = torch.full((h, flat["q"].shape[0]), -math.inf, dtype=torch.float64, device="cuda")
    for a, b in spans:
        n, m = a.stop - a.start, b.stop - b.start
        hide = torch.ones(n, m, dtype=torch.bool, device="cuda").triu(m - n + 1) if case["causal"] else None
        for i in range(h):
            q, k, v = flat["q"][a, i].double(), flat["k"][b, i // share].double(), flat["v"][b, i // share].double()
            z = q @ k.T / math.sqrt(d)
            if hide is not None:
                z[hide] = -math.inf
            r = torch.logsumexp(z, 1)
            p = torch.exp(z - r[:, None])
            p[r == -math.inf] = 0.0
            y = p @ v
            if case["op"] == "attn_fwd":
                o[a, i], lse[i, a] = y, r
                continue
            w = flat["do"][a, i].double()
            dv[b, i // share] += p.T @ w
            dz = p * (w @ v.T - (w * y).sum(1, keepdim=True)) / math.sqrt(d)
            dq[a, i] = dz @ k
            dk[b, i // share] += dz.T @ q
    if case["op"] == "attn_fwd":
        if case["layout"] == "dense":
            lse = lse.reshape(h, case["seqs"], case["lq"]).transpose(0, 1).contiguous()
        return {"o": o.reshape(s["q"].shape), "lse": lse}
    return {"dq": dq.reshape(s["q"].shape), "dk": dk.reshape(s["k"].shape), "dv": dv.reshape(s["v"].shape)}
