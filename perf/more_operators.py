"""Measured cases of rotary positions, the AdamW step, and many adapters beside one NF4 projection.

Rotary positions of q and k (forward, and backward through the same rotation), in halves or interleaved, over part of a head, at
far and scaled positions; the AdamW step over all adapters at once with its states in 32 or in 8 bits; and the NF4 linear layer
whose rows belong to different requests, each with an adapter of its own, from one token to a batch of prompts.

`run` has every operator twice: in plain torch operations held in 32 bits (`own` false) and through this package's entry points
(`own` true).  `exact` is the same in 64 bits, written from the definitions.
"""

import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BLOCK = 256  # elements of a tensor that share the scales of their 8-bit optimizer states


# ---------------------------------------------------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------------------------------------------------

def _rope(op, seqs, rows, heads, kv_heads, dim, rot=None, layout="dense", interleaved=False, fused=False, far=0, factor=1.0):
    """`seqs` sequences of `rows` tokens; packed: `rows` tokens in `seqs` sequences of unequal length.  `rot` rotated elements of
    each head; `far`: the tokens stand somewhere before this position (0: at 0, 1, ...); `factor`: positions stretched beyond the
    trained length; `fused`: q and k are views of one projection's output."""
    return {"op": op, "layout": layout, "seqs": seqs, "rows": rows, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": dim if rot is None else rot, "interleaved": interleaved, "fused": fused, "far": far, "factor": factor}


def _adamw(bits, layers, hidden, inner, rank, types, clipped, step):
    """The adapters of `layers` decoder blocks: A [rank, K] and B [N, rank] of q, k, v, o, gate, up and down.  `types`: of the
    parameters and gradients, or "mixed": parameters in 32 bits with a copy and gradients in bf16."""
    return {"op": "adamw", "bits": bits, "layers": layers, "hidden": hidden, "inner": inner, "rank": rank, "types": types,
            "clipped": clipped, "step": step}


def _multi(tokens, n, k, rank, adapters, order):
    """`tokens` rows over an [n, k] weight.  `order`: "each" (row after row another adapter, as when every request gives one
    token), "runs" (prompts one after the other), "some" (as "each", a third of the rows without an adapter)."""
    return {"op": "multi", "tokens": tokens, "n": n, "k": k, "rank": rank, "adapters": adapters, "order": order}


def listed():
    return [
        # one token of each of 16 requests deep in long contexts, shared key/value heads: the time of a call
        dict(_rope("rope_fwd", 16, 1, 32, 8, 128, far=131072, factor=8.0), name="rope_fwd_16x1_far"),
        # the 4096-token step (8 x 512) of the 32-head, 4096-wide layers that the benchmark times, from a fused projection
        dict(_rope("rope_fwd", 8, 512, 32, 32, 128, fused=True), name="rope_fwd_8x512"),
        # a short instruction of odd length, half of each head rotated, neighbours as pairs
        dict(_rope("rope_bwd", 1, 67, 16, 16, 64, rot=32, interleaved=True), name="rope_bwd_1x67_part"),
        # examples of unequal length packed into one row, 40 heads as in the 5120-wide block
        dict(_rope("rope_bwd", 17, 8191, 40, 40, 128, layout="packed"), name="rope_bwd_packed_8191"),
        # one small block with rank 8: the time of a call over 14 tensors
        dict(_adamw(32, 1, 1024, 2730, 8, "fp32", False, 1), name="adamw32_1_block_r8"),
        # every adapter of a 32-block model at rank 64: 448 tensors, clipped on the way
        dict(_adamw(32, 32, 4096, 11008, 64, "bf16", True, 100), name="adamw32_32_blocks_r64"),
        # the same two with states in 8 bits, the small one with its parameters in 32 bits beside bf16 copies
        dict(_adamw(8, 1, 1024, 2730, 8, "mixed", True, 10), name="adamw8_1_block_r8"),
        dict(_adamw(8, 32, 4096, 11008, 64, "bf16", True, 100), name="adamw8_32_blocks_r64"),
        # a single request
        dict(_multi(1, 4096, 4096, 16, 8, "each"), name="multi_1_4096x4096"),
        # one token of each of 16 requests over the widest projection of the benchmark
        dict(_multi(16, 28672, 8192, 16, 16, "each"), name="multi_16_28672x8192"),
        # a decoding batch, some of it on the base model
        dict(_multi(61, 8192, 8192, 32, 24, "some"), name="multi_61_8192x8192"),
        # prompts of a few requests together, 4096 tokens in all
        dict(_multi(4096, 11008, 4096, 64, 5, "runs"), name="multi_4096_11008x4096"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    top = max(_cost(c) for c in listed())
    while True:
        c = _draw(rng)
        if _cost(c) <= top:
            return c


def _draw(rng):
    op = rng.choice(["rope_fwd", "rope_bwd", "adamw", "adamw", "multi", "multi", "multi"])
    if op.startswith("rope"):
        kv = rng.choice([1, 2, 4, 5, 8, 16, 32])
        heads = kv * rng.choice([g for g in (1, 1, 2, 4, 8) if kv * g <= 40])
        dim = rng.choice([64, 80, 96, 128, 128])
        rot = rng.choice([dim, dim, dim // 2, dim // 4, 2 * rng.randint(1, dim // 2)])
        layout = rng.choice(["dense", "dense", "packed"])
        rows = _log(rng, 1, 16384)
        seqs = _log(rng, 1, min(128, rows)) if layout == "packed" else max(1, int(rng.uniform(0.05, 1.0) * 16384 / rows))
        return _rope(op, min(seqs, 512), rows, heads, kv, dim, rot, layout, rng.random() < 0.4, rng.random() < 0.5,
                     rng.choice([0, 4096, 131072, 1 << 24]) if layout == "dense" else 0, rng.choice([1.0, 1.0, 4.0, 32.0]))
    if op == "adamw":
        hidden = _log(rng, 128, 8192)
        return _adamw(rng.choice([8, 8, 32]), _log(rng, 1, 48), hidden, int(hidden * rng.uniform(2.0, 4.0)), _log(rng, 1, 128),
                      rng.choice(["bf16", "fp32", "mixed"]), rng.random() < 0.5, _log(rng, 1, 10000))
    return _multi(_log(rng, 1, 4096), 8 * _log(rng, 8, 3584), 64 * _log(rng, 1, 172), rng.choice([8, 16, 16, 32, 64, _log(rng, 1, 128)]),
                  _log(rng, 1, 64), rng.choice(["each", "runs", "some"]))


def _lengths(case):
    """The lengths of a packed batch's sequences: cut points that follow from the case alone."""
    rng = random.Random("%d tokens in %d" % (case["rows"], case["seqs"]))
    cuts = sorted(rng.randrange(case["rows"] + 1) for _ in range(case["seqs"] - 1))
    return [b - a for a, b in zip([0] + cuts, cuts + [case["rows"]])]


def _adapters(case):
    h, m, r = case["hidden"], case["inner"], case["rank"]
    block = []
    for n, k in ((h, h), (h, h), (h, h), (h, h), (m, h), (m, h), (h, m)):
        block += [(r, k), (n, r)]
    return block * case["layers"]


def _owners(case):
    """The adapter of each row, -1 for none."""
    rng = random.Random("%(tokens)d rows of %(adapters)d, %(order)s" % case)
    m, n = case["tokens"], case["adapters"]
    if case["order"] == "runs":
        cuts = sorted(rng.randrange(m + 1) for _ in range(n - 1))
        return [a for a, (b, e) in enumerate(zip([0] + cuts, cuts + [m])) for _ in range(e - b)]
    first = rng.randrange(n)
    return [-1 if case["order"] == "some" and rng.random() < 1 / 3 else (first + i) % n for i in range(m)]


def work(case):
    op = case["op"]
    if op.startswith("rope"):
        tokens = case["rows"] * (1 if case["layout"] == "packed" else case["seqs"])
        heads = case["heads"] + case["kv_heads"]
        return {"bytes": 4 * tokens * heads * case["dim"] + (8 * tokens if case["far"] else 0) + 4 * case["rot"],
                "flops": 3 * tokens * heads * case["rot"]}
    if op == "adamw":
        n = sum(a * b for a, b in _adapters(case))
        param = {"bf16": 2 + 2 + 2, "fp32": 4 + 4 + 4, "mixed": 4 + 4 + 2 + 2}[case["types"]]
        # 8 bits: two codes read and written, a scale of each for every block; the values they stand for are returned in 32
        state = 16 if case["bits"] == 32 else 2 * (2 + 8 / BLOCK) + 8
        return {"bytes": int(n * (param + state)), "flops": (15 if case["bits"] == 32 else 45) * n}
    m, n, k, r = case["tokens"], case["n"], case["k"], case["rank"]
    rows = [a for a in _owners(case) if a >= 0]
    return {"bytes": n * k // 2 + n * k // 64 + n * k // 4096 + 2 * m * (n + k) + 2 * len(set(rows)) * r * (n + k) + 4 * m,
            "flops": 2 * m * n * k + 2 * len(rows) * r * (n + k)}


def _cost(case):
    w = work(case)
    return w["bytes"] / 4e12 + w["flops"] / 400e12


# ---------------------------------------------------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------------------------------------------------

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)

    if case["op"] == "adamw":
        return _prepare_adamw(case, g, normal)
    s = {"case": case}
    if case["op"] == "multi":
        m, n, k, r, a = (case[x] for x in ("tokens", "n", "k", "rank", "adapters"))
        blocks = n * k // 64
        # each of the 16 levels stands for an equal share of the weights; block constants as of a trained layer
        s["codes"] = torch.randint(0, 256, (n * k // 2,), generator=g, dtype=torch.uint8, device="cuda")
        s["q8"] = torch.randint(96, 256, (blocks,), generator=g, dtype=torch.uint8, device="cuda")
        s["step"] = (1.0 + torch.rand(-(-blocks // 256), generator=g, device="cuda")) * (k ** -0.5 / 100.0)
        s["x"] = normal(m, k)
        s["a"], s["b"] = normal(a, r, k, std=k ** -0.5), normal(a, n, r, std=0.3)
        s["s"] = 2.0 ** torch.randint(0, 3, (a,), generator=g, device="cuda").float() / 2.0
        s["index"] = torch.tensor(_owners(case), dtype=torch.int32, device="cuda")
        return s
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["layout"] == "packed":
        lens = _lengths(case)
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")
        s["rows"] = torch.cat([torch.arange(n, device="cuda") for n in lens])
        lead = (case["rows"],)
    else:
        s["cu"] = None
        lead = (case["seqs"], case["rows"])
        s["rows"] = torch.arange(case["rows"], device="cuda").expand(lead)
    s["positions"] = None
    if case["far"]:
        start = torch.randint(0, max(1, case["far"] - case["rows"]), (case["seqs"], 1), generator=g, device="cuda")
        s["positions"] = s["rows"] = start + s["rows"]
    if case["fused"]:
        s["q"], s["k"] = normal(*lead, h + 2 * hk, d).split([h, hk, hk], dim=-2)[:2]
    else:
        s["q"], s["k"] = normal(*lead, h, d), normal(*lead, hk, d)
    s["inv_freq"], s["scale"] = _frequencies(case["rot"], case["factor"])
    s["inv_freq"] = s["inv_freq"].cuda()
    return s


def _frequencies(rot, factor, base=10000.0, length=4096):
    """Radians per position in 64 bits.  A factor above 1 stretches the slow pairs (less than one turn within the trained length)
    by it, leaves the fast ones (more than 32 turns), and blends between."""
    f = base ** -(torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    if factor == 1.0:
        return f, 1.0
    keep = ((length * f / (2 * math.pi) - 1.0) / 31.0).clamp(0.0, 1.0)
    return f * keep + f / factor * (1.0 - keep), 0.1 * math.log(factor) + 1.0


def _prepare_adamw(case, g, normal):
    shapes = _adapters(case)
    sizes = [a * b for a, b in shapes]
    spans = [-(-n // BLOCK) * BLOCK for n in sizes]
    total = sum(spans)
    low = torch.float32 if case["types"] == "fp32" else torch.bfloat16
    s = {"case": case, "pads": [b - n for n, b in zip(sizes, spans)], "lr": 2e-4, "betas": (0.9, 0.999), "eps": 1e-8, "decay": 0.01}
    # the parameters lie one after the other in the program's flat buffer, each from a multiple of a block on
    at = _starts(spans)
    s["flat"] = normal(total, std=0.02, dtype=low if case["types"] == "bf16" else torch.float32)
    s["copy"] = s["flat"].to(low) if case["types"] == "mixed" else None
    inside = torch.ones(total, dtype=torch.bool, device="cuda")
    for a, n, b in zip(at, sizes, spans):
        inside[a + n:a + b] = False
    s["flat"].mul_(inside)

    def views(t):
        return None if t is None else [t[a:a + n].view(shape) for a, n, shape in zip(at, sizes, shapes)]
    s["params"], s["copies"] = views(s["flat"]), views(s["copy"])
    # gradients of very unequal size, as A's and B's are; the states of some steps over such gradients
    scale = [3e-4 * (1 + i % 5) for i in range(len(shapes))]
    s["grads"] = [normal(a, b, std=c, dtype=low) for (a, b), c in zip(shapes, scale)]
    each = torch.repeat_interleave(torch.tensor(scale), torch.tensor(spans)).cuda() * inside
    m = torch.randn(total, generator=g, device="cuda") * 0.3 * each
    v = (0.5 + torch.rand(total, generator=g, device="cuda")) * (torch.randn(total, generator=g, device="cuda") * 0.5).exp() * each * each
    s["m"], s["v"], s["m_scale"], s["v_scale"] = (m, v, None, None) if case["bits"] == 32 else _to8(m, v)
    s["norm"] = torch.linalg.vector_norm(torch.cat([t.flatten().float() for t in s["grads"]])).reshape(1)
    s["max_norm"] = float(s["norm"]) * 0.7 if case["clipped"] else None
    return s


def _starts(spans):
    at = [0]
    for n in spans[:-1]:
        at.append(at[-1] + n)
    return at


# ---------------------------------------------------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------------------------------------------------

def _plain_rope(s, sign):
    case = s["case"]
    angle = s["rows"].double().unsqueeze(-1) * s["inv_freq"]
    c = (torch.cos(angle) * s["scale"]).float().unsqueeze(-2)
    n = (torch.sin(angle) * (sign * s["scale"])).float().unsqueeze(-2)
    r = case["rot"]

    def turn(t):
        x32 = t[..., :r].float()
        x, y = (x32[..., 0::2], x32[..., 1::2]) if case["interleaved"] else (x32[..., :r // 2], x32[..., r // 2:])
        a, b = x * c - y * n, y * c + x * n
        z = torch.stack([a, b], -1).flatten(-2) if case["interleaved"] else torch.cat([a, b], -1)
        return torch.cat([z.to(t.dtype), t[..., r:]], -1)
    return turn(s["q"]), turn(s["k"])


def _to8(m, v):
    """The states' codes and scales: one scale for each block, its largest magnitude; square law for m, fourth power for v."""
    mb, vb = m.view(-1, BLOCK), v.view(-1, BLOCK)
    ms, vs = mb.abs().amax(1, keepdim=True), vb.amax(1, keepdim=True)
    ms, vs = (torch.where(t < 2.0 ** -96, 0.0, t) for t in (ms, vs))
    edge = (torch.arange(1, 256, device=m.device) - 0.5).square()  # between code c - 1 and code c
    cm = torch.bucketize(torch.where(ms > 0, mb.abs() * (torch.full_like(ms, 127.0 ** 2) / ms), 0.0), edge[:127], right=True)
    cv = torch.bucketize(torch.where(vs > 0, vb * (torch.full_like(vs, 255.0 ** 4) / vs), 0.0), edge * edge, right=True)
    cv = torch.where((vb > 0) & (vs > 0), cv.clamp(min=1), cv)  # what is not 0 does not become 0
    return torch.where(mb < 0, -cm, cm).to(torch.int8).view(-1), cv.to(torch.uint8).view(-1), ms.view(-1), vs.view(-1)


def _from8(m, v, ms, vs):
    c, d = m.view(-1, BLOCK).float(), v.view(-1, BLOCK).float()
    d = d * d
    return (c * c.abs() * (1 / 16129) * ms.view(-1, 1)).view(-1), (d * d * (1 / 255 ** 4) * vs.view(-1, 1)).view(-1)


def _plain_adamw(s):
    b1, b2 = s["betas"]
    t, lr = s["case"]["step"], s["lr"]
    eight = s["case"]["bits"] == 8
    m, v = _from8(s["m"], s["v"], s["m_scale"], s["v_scale"]) if eight else (s["m"], s["v"])
    grad = torch.cat([torch.nn.functional.pad(x.flatten(), (0, n)) for x, n in zip(s["grads"], s["pads"])]).float()
    if s["max_norm"] is not None:
        grad = grad * torch.clamp(s["max_norm"] / (s["norm"].double() + 1e-6), max=1.0).float()
    m = m * b1 + grad * (1 - b1)
    v = v * b2 + (grad * grad) * (1 - b2)
    p = s["flat"].float() * (1 - lr * s["decay"]) - m * (lr / (1 - b1 ** t)) / (torch.sqrt(v) / math.sqrt(1 - b2 ** t) + s["eps"])
    s["flat"].copy_(p)
    if s["copy"] is not None:
        s["copy"].copy_(p)
    if not eight:
        s["m"].copy_(m)
        s["v"].copy_(v)
        return m, v
    for name, t in zip(("m", "v", "m_scale", "v_scale"), _to8(m, v)):
        s[name].copy_(t)
    return _from8(s["m"], s["v"], s["m_scale"], s["v_scale"])


def _levels():
    """The 16 NF4 levels: normal quantiles with an exact zero, the outermost at -1 and 1."""
    top = 1.0 - 0.5 * (1.0 / 30.0 + 1.0 / 32.0)
    up = torch.special.ndtri(torch.linspace(top, 0.5, 9, dtype=torch.float64)[:8])
    down = torch.special.ndtri(torch.linspace(top, 0.5, 8, dtype=torch.float64)[:7])
    return torch.cat([-down, torch.zeros(1, dtype=torch.float64), up.flip(0)]) / up[0]


LEVELS = _levels()


def _weight(s):
    """W [n, k]: bf16 values of level times block constant."""
    case = s["case"]
    codes = torch.stack([s["codes"] & 15, s["codes"] >> 4], -1).flatten().int()
    const = s["q8"].float() * s["step"].repeat_interleave(256)[:s["q8"].numel()]
    w = LEVELS.float().cuda()[codes].view(-1, 64) * const.unsqueeze(1)
    return w.bfloat16().view(case["n"], case["k"])


def _plain_multi(s):
    case = s["case"]
    a, r = case["adapters"], case["rank"]
    x = s["x"].float()
    u = torch.matmul(x, s["a"].float().flatten(0, 1).t()).view(-1, a, r)
    mine = s["index"].unsqueeze(1) == torch.arange(a, device="cuda")
    u = torch.where(mine.unsqueeze(2), u * s["s"].view(1, a, 1), 0.0).flatten(1)
    y = torch.matmul(x, _weight(s).float().t()) + torch.matmul(u, s["b"].float().transpose(0, 1).flatten(1).t())
    return y.bfloat16()


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        import quantized_base_lora_nf4_amd as qn
        if op in ("rope_fwd", "rope_bwd"):
            q, k = (qn.rope_fwd if op == "rope_fwd" else qn.rope_bwd)(
                s["q"], s["k"], s["inv_freq"], positions=s["positions"], cu_seqlens=s["cu"], interleaved=case["interleaved"],
                scale=s["scale"])
            return {"q": q, "k": k}
        if op == "adamw":
            st = qn.AdamWState(s["m"], s["v"], s["m_scale"], s["v_scale"])
            if s["copy"] is not None and "ends" not in s:
                # the program's own padding between the copies, which the step does not write, cleared before the first one
                s["ends"] = [t[t.numel() - n:] for t, n in zip(s["copy"].split([x.numel() + n for x, n in zip(s["grads"], s["pads"])]),
                                                               s["pads"]) if n]
                torch._foreach_zero_(s["ends"])
            qn.adamw_step(s["params"], s["grads"], st, case["step"], s["lr"], betas=s["betas"], eps=s["eps"],
                          weight_decay=s["decay"], norm=None if s["max_norm"] is None else s["norm"], max_norm=s["max_norm"],
                          copies=s["copies"])
            m, v = qn.adamw_values(st)
            return {"p": s["flat"], "copy": s["copy"], "m": m, "v": v}
        w = qn.NF4Weight(s["codes"], s["q8"], s["step"], case["n"], case["k"])
        return {"y": qn.qlora_linear_multi_fwd(w, s["x"], s["a"], s["b"], s["s"], s["index"])}
    if op in ("rope_fwd", "rope_bwd"):
        q, k = _plain_rope(s, 1.0 if op == "rope_fwd" else -1.0)
        return {"q": q, "k": k}
    if op == "adamw":
        m, v = _plain_adamw(s)
        return {"p": s["flat"], "copy": s["copy"], "m": m, "v": v}
    return {"y": _plain_multi(s)}


# ---------------------------------------------------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "multi":
        x, w = s["x"].double(), _weight(s).double()
        y = x @ w.T
        del w
        for i in sorted(set(_owners(case)) - {-1}):
            mine = s["index"] == i
            y[mine] += float(s["s"][i]) * ((x[mine] @ s["a"][i].double().T) @ s["b"][i].double().T)
        return {"y": y}
    if case["op"] == "adamw":
        return _exact_adamw(s)
    # a pair is a complex number, the backward pass its rotation by the negative angle
    turn = torch.polar(torch.full_like(s["inv_freq"], s["scale"]).expand(*s["rows"].shape, -1),
                       (1 if case["op"] == "rope_fwd" else -1) * s["rows"].double().unsqueeze(-1) * s["inv_freq"]).unsqueeze(-2)
    out = {}
    for name in ("q", "k"):
        z = s[name].double()
        part = z[..., :case["rot"]]
        pairs = part.unflatten(-1, (-1, 2)) if case["interleaved"] else part.unflatten(-1, (2, -1)).transpose(-1, -2)
        pairs = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        part = pairs.flatten(-2) if case["interleaved"] else pairs.transpose(-1, -2).flatten(-2)
        out[name] = torch.cat([part, z[..., case["rot"]:]], -1)
    return out


def _exact_adamw(s):
    """Tensor after tensor.  The values that 8-bit states stand for have no 64-bit form: which code is nearest is settled by the
    32-bit arithmetic."""
    case = s["case"]
    (b1, b2), lr, t = s["betas"], s["lr"], case["step"]
    m8 = v8 = None
    if case["bits"] == 8:
        m8 = s["m"].double() * s["m"].double().abs() / 127 ** 2 * s["m_scale"].double().repeat_interleave(BLOCK)
        v8 = (s["v"].double() / 255) ** 4 * s["v_scale"].double().repeat_interleave(BLOCK)
    m_all, v_all = (s["m"].double(), s["v"].double()) if m8 is None else (m8, v8)
    p_all = s["flat"].double()
    at = 0
    for grad, pad in zip(s["grads"], s["pads"]):
        here = slice(at, at + grad.numel())
        d = grad.double().flatten()
        if s["max_norm"] is not None:
            d = d * min(1.0, s["max_norm"] / (float(s["norm"]) + 1e-6))
        m_all[here] += (1 - b1) * (d - m_all[here])
        v_all[here] += (1 - b2) * (d.square() - v_all[here])
        way = (m_all[here] / (1 - b1 ** t)) / ((v_all[here] / (1 - b2 ** t)).sqrt() + s["eps"])
        p_all[here] -= lr * (s["decay"] * p_all[here] + way)
        at += grad.numel() + pad
    eight = case["bits"] == 8
    return {"p": p_all, "copy": p_all if s["copy"] is not None else None, "m": None if eight else m_all, "v": None if eight else v_all}
