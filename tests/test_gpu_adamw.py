"""The AdamW step against the fp64 oracle, and its 8-bit states bit for bit.

Tolerances (u = 2^-24, half an fp32 step, relative): beta and 1 - beta are
rounded to fp32, and each product and sum, so m and v are off by at most
4 u (b |m| + (1 - b) |g|) (v: one product more, 5 u).  The update divides m by
sqrt(v) / sqrt(1 - b2^t) + eps: half of v's error, and at most 2 u each for
two constants, the square root, the reciprocal (1 unit in the last place each),
the fused sum and two products: 20 u of the update beside m's share.  The
parameter is scaled (2 u) and summed (1 u), and rounded to its type.
"""

import math

import numpy as np
import pytest
import torch

import quantized_base_lora_nf4_amd as qn
from gpu_util import say
from oracle import adamw as oracle

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
U = 2.0 ** -24
SIZES = [1, 2048, 255, 256, 257, 0, 2049, 4097, 31, 8 * 1024]
HYPER = dict(lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.02)


def host(t):
    return t.detach().float().cpu().numpy()


class Case:
    """Tensors, some steps' worth of states, and what the oracle says."""

    def __init__(self, sizes, p_types, g_types, bits, seed=0, off=0, spread=1.0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def randn(n, dt, std=1.0):
            # `off` elements into an allocation: only the elements' alignment
            return (torch.randn(n + off, generator=g, device="cuda") * std).to(dt)[off:]
        self.sizes = sizes
        self.params = [randn(n, p_types[i % len(p_types)], 0.05) for i, n in enumerate(sizes)]
        self.grads = [randn(n, g_types[i % len(g_types)], 1e-3) *
                      (10.0 ** (spread * torch.rand(n, generator=g, device="cuda") - spread)).to(g_types[i % len(g_types)])
                      for i, n in enumerate(sizes)]
        self.state = qn.adamw_init(self.params, bits, device="cuda")
        self.spans = [-(-n // 256) * 256 for n in sizes]
        self.at = np.cumsum([0] + self.spans)[:-1]
        m = [1e-4 * torch.randn(n, generator=g, device="cuda") for n in sizes]
        v = [1e-7 * torch.rand(n, generator=g, device="cuda") for n in sizes]
        for i, n in enumerate(sizes):
            self.put(i, host(m[i]), host(v[i]))

    def parts(self, i):
        a, b = self.at[i], self.at[i] + self.spans[i]
        return a, b, a // 256, b // 256

    def put(self, i, m, v):
        a, b, c, d = self.parts(i)
        s = self.state
        if s.bits == 32:
            s.m[a:a + len(m)], s.v[a:a + len(v)] = torch.from_numpy(m).cuda(), torch.from_numpy(v).cuda()
            return
        for t, x, lo, hi in zip((s.m, s.v, s.m_scale, s.v_scale), oracle.pack(m, v), (a, a, c, c), (b, b, d, d)):
            t[lo:hi] = torch.from_numpy(x).cuda()

    def get(self, i):
        """fp32 m and v of tensor i, padded."""
        a, b, c, d = self.parts(i)
        s = self.state
        if s.bits == 32:
            return host(s.m[a:b]), host(s.v[a:b])
        return oracle.unpack(s.m[a:b].cpu().numpy(), s.v[a:b].cpu().numpy(), host(s.m_scale[c:d]), host(s.v_scale[c:d]))

    def raw(self, i):
        a, b, c, d = self.parts(i)
        s = self.state
        return [t[lo:hi].cpu().numpy().copy() for t, lo, hi in
                zip((s.m, s.v, s.m_scale, s.v_scale), (a, a, c, c), (b, b, d, d)) if t is not None]

    def check(self, step, factor=1.0, copies=None, left=(), run=None, **hyper):
        h = {**HYPER, **hyper}
        (b1, b2), lr, eps, decay = h["betas"], h["lr"], h["eps"], h["weight_decay"]
        before = [(host(p).astype(np.float64), *self.get(i)) for i, p in enumerate(self.params)]
        raw = [self.raw(i) for i in range(len(self.params))]
        run()
        torch.cuda.synchronize()
        worst = 0.0
        for i, (n, p, g) in enumerate(zip(self.sizes, self.params, self.grads)):
            p0, m0, v0 = before[i]
            if i in left:
                assert np.array_equal(host(p), p0.astype(np.float32))
                assert all(np.array_equal(x, y, equal_nan=x.dtype.kind == "f") for x, y in zip(self.raw(i), raw[i]))
                continue
            g64 = host(g).astype(np.float64)
            ref, m, v = oracle.step64(p0, g64, m0[:n], v0[:n], step, lr, b1, b2, eps, decay, factor)
            em = 4 * U * (b1 * np.abs(m0[:n]) + (1 - b1) * np.abs(factor * g64))
            ev = 5 * U * v
            d = np.sqrt(v / (1 - b2 ** step)) + eps
            way = lr / (1 - b1 ** step) / d
            tol = way * em + 20 * U * np.abs(way * m) + 3 * U * np.abs(p0) + U * np.abs(ref)
            if p.dtype == BF:
                tol = tol + 2.0 ** -8 * (np.abs(ref) + tol)
            err = np.abs(host(p) - ref)
            assert (err <= tol).all(), f"tensor {i}: {float((err / tol).max())} of the bound"
            worst = max(worst, float((err / np.maximum(tol, 1e-300)).max(initial=0.0)))
            if copies is not None and copies[i] is not None:
                assert torch.equal(copies[i], p.to(BF))
            if self.state.bits == 32:
                x, y = self.get(i)
                assert (np.abs(x[:n] - m) <= em).all() and (np.abs(y[:n] - v) <= ev).all()
                assert not x[n:].any() and not y[n:].any()
            else:
                expect = oracle.pack(*oracle.states32(host(g), m0[:n], v0[:n], b1, b2, factor))
                for what, x, y in zip(("m", "v", "m scale", "v scale"), self.raw(i), expect):
                    assert np.array_equal(x, y), f"tensor {i}: {what} differs in {int((x != y).sum())} of {y.size}"
        say(f"    parameters: {worst:.3f} of the bound")


def step(c, n, **kw):
    h = {**HYPER, **kw}
    return lambda: qn.adamw_step(c.params, c.grads, c.state, n, h.pop("lr"), **h)


TYPES = [([BF], [BF]), ([F32], [F32]), ([F32], [BF]), ([BF], [F32]), ([BF, F32, F32], [F32, BF])]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("types", TYPES, ids=lambda t: "-".join(str(x).split(".")[-1] for x in t[0] + t[1]))
@pytest.mark.parametrize("off", [0, 1])
def test_types_and_sizes(bits, types, off):
    say(f"[adamw] {bits} bits, {types}, offset {off}")
    c = Case(SIZES, *types, bits, seed=bits + off, off=off)
    for n in (3, 4):
        c.check(n, run=step(c, n))


@pytest.mark.parametrize("bits", [32, 8])
def test_first_step_from_new_states(bits):
    c = Case(SIZES, [BF], [BF], bits)
    c.state = qn.adamw_init(c.params, bits)
    c.check(1, run=step(c, 1))
    # from zeros the update is lr sign(g), but for eps
    c = Case([512], [F32], [F32], bits)
    c.state = qn.adamw_init(c.params, bits)
    p = c.params[0].clone()
    qn.adamw_step(c.params, c.grads, c.state, 1, 0.5, eps=0.0, weight_decay=0.0)
    there = c.grads[0] != 0
    way = (p - c.params[0])[there]
    assert torch.allclose(way, 0.5 * c.grads[0][there].sign(), rtol=1e-4)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("hyper", [dict(betas=(0.0, 0.0)), dict(betas=(0.5, 0.9), lr=0.3), dict(weight_decay=0.0),
                                   dict(lr=0.0), dict(eps=1e-3), dict(betas=(0.95, 0.9999), weight_decay=1.5)])
def test_settings(bits, hyper):
    say(f"[adamw] {bits} bits, {hyper}")
    c = Case([300, 2048], [F32, BF], [BF], bits, seed=3)
    for n in (1, 1000):
        c.check(n, run=step(c, n, **hyper), **hyper)


@pytest.mark.parametrize("bits", [32, 8])
def test_many_tensors(bits):
    """More than a launch's table, with some gradients missing."""
    say(f"[adamw] {bits} bits, many tensors")
    rng = np.random.default_rng(5)
    sizes = [int(n) for n in rng.integers(1, 3000, 450)]
    c = Case(sizes, [BF, F32], [BF], bits)
    left = [i for i in range(450) if i % 7 == 3]
    for i in left:
        c.grads[i] = None
    c.check(2, left=left, run=step(c, 2))


@pytest.mark.parametrize("bits", [32, 8])
def test_copies(bits):
    c = Case(SIZES * 12, [F32, BF], [BF], bits, off=1)
    copies = [torch.zeros_like(p, dtype=BF) if i % 3 else None for i, p in enumerate(c.params)]
    c.check(2, copies=copies, run=step(c, 2, copies=copies))


def test_copies_of_all():
    """Every parameter with a copy, and each way in which one of them does not fit."""
    c = Case([300, 64, 7], [F32], [F32], 32)
    copies = [torch.zeros_like(p, dtype=BF) for p in c.params]
    c.check(2, copies=copies, run=step(c, 2, copies=copies))
    before = [p.clone() for p in c.params]
    for bad, error in ((copies[1].float(), TypeError), (copies[1].cpu(), ValueError), (copies[1].view(8, 8), ValueError),
                       (torch.zeros(64, 2, dtype=BF, device="cuda")[:, 0], ValueError), (3, TypeError)):
        with pytest.raises(error):
            step(c, 3, copies=[copies[0], bad, copies[2]])()
    assert all(torch.equal(a, b) for a, b in zip(before, c.params))


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("norm,max_norm", [(2.0, 0.3), (0.1, 0.3), (2.0, 0.0), (1e-20, 1e-20), (float("inf"), 1.0),
                                           (float("inf"), float("inf"))])
def test_clipping(bits, norm, max_norm):
    c = Case([1000, 64], [F32], [BF], bits)
    factor = float(np.float32(oracle.clip_factor(np.float32(norm), max_norm)))
    t = torch.tensor([norm], device="cuda")
    before = [g.clone() for g in c.grads]
    c.check(5, factor=factor, run=step(c, 5, norm=t, max_norm=max_norm))
    assert all(torch.equal(a, b) for a, b in zip(before, c.grads))


def test_clipping_factor_is_rounded_once():
    """From the limit as it is given: its own rounding to fp32 would move the
    factor by a step for about half of the norms."""
    p, g = torch.zeros(1, device="cuda"), torch.ones(1, device="cuda")
    rng = np.random.default_rng(7)
    for n in rng.uniform(1.0, 20.0, 64).astype(np.float32):
        st, limit = qn.adamw_init([p], bits=32), float(n) * 0.7
        qn.adamw_step([p], [g], st, 1, 0.0, betas=(0.0, 0.0), norm=torch.tensor([n], device="cuda"), max_norm=limit)
        assert float(st.m[0]) == np.float32(oracle.clip_factor(n, limit))


def test_clipping_with_grad_norm_is_clip_then_step():
    """fp32 gradients: scaled in the step as clip_grad_norm scales them."""
    for bits in (32, 8):
        a, b = (Case([5000, 33], [F32], [F32], bits) for _ in range(2))
        norm = qn.grad_norm(a.grads)
        limit = float(norm) / 2
        step(a, 3, norm=norm, max_norm=limit)()
        qn.clip_grad_norm(b.grads, limit)
        step(b, 3)()
        # the factor comes from the norm in fp32 here, in fp64 there: one step of it
        for x, y in zip(a.params, b.params):
            assert torch.allclose(x, y, rtol=1e-6, atol=1e-9)


def test_nan_and_infinite_gradients():
    say("[adamw] NaN and infinities")
    c = Case([1024, 300], [F32], [F32], 8)
    c.grads[0][5], c.grads[0][300], c.grads[0][301] = float("nan"), float("inf"), -1.0
    qn.adamw_step(c.params, c.grads, c.state, 2, 1e-3)
    p = c.params[0]
    assert p[5].isnan() and p[300].isnan() and p[[0, 1, 301, 600]].isfinite().all()
    m, v = qn.adamw_values(c.state)
    assert m[:512].isnan().all() and v[:512].isnan().all()      # the two blocks, as a whole
    assert m[512:].isfinite().all() and v[512:].isfinite().all()
    assert c.params[1].isfinite().all()
    c = Case([1024], [F32], [F32], 32)
    c.grads[0][5] = float("nan")
    qn.adamw_step(c.params, c.grads, c.state, 2, 1e-3)
    assert int(c.params[0].isnan().sum()) == 1 and int(c.state.m.isnan().sum()) == 1
    c = Case([1024], [F32], [F32], 8)
    t = torch.tensor([float("nan")], device="cuda")
    qn.adamw_step(c.params, c.grads, c.state, 2, 1e-3, norm=t, max_norm=1.0)
    assert c.params[0].isnan().all()


def test_zero_and_tiny_gradients():
    c = Case([700], [F32], [F32], 8)
    c.state = qn.adamw_init(c.params, 8)
    c.grads[0].zero_()
    c.check(1, run=step(c, 1))
    assert not c.state.m.any() and not c.state.v.any() and not c.state.m_scale.any()
    c.grads[0].fill_(1e-30)     # below the smallest scale: stored as zeros
    c.check(2, run=step(c, 2))
    assert not c.state.m.any() and not c.state.v_scale.any()
    c.grads[0].copy_(torch.logspace(-18, 3, 700, device="cuda"))
    for n in (3, 4, 5):
        c.check(n, run=step(c, n))


def test_codes_at_their_thresholds():
    """Values on and next to every threshold (beta = 0: the states are the
    gradient and its square)."""
    edges = (np.arange(1, 128) - 0.5) ** 2 / 127.0 ** 2
    near = np.concatenate([np.nextafter(edges.astype(np.float32), np.float32(2 * s)) if s >= 0 else edges
                           for s in (0, 1)] + [edges.astype(np.float32)])
    rng = np.random.default_rng(1)
    vals = np.concatenate([near, -near, np.sqrt(((np.arange(1, 256) - 0.5) / 255) ** 4)]).astype(np.float32)
    rows = []
    for top in (1.0, 0.37, 3e-7, 1.7e4):
        for part in np.array_split(vals, -(-len(vals) // 255)):
            x = np.zeros(256, np.float32)
            x[0] = top
            x[1:1 + len(part)] = part * np.float32(top)
            rows.append(x)
    g = np.concatenate(rows)
    c = Case([len(g)], [F32], [F32], 8)
    c.grads = [torch.from_numpy(g).cuda()]
    c.check(1, run=step(c, 1, betas=(0.0, 0.0)), betas=(0.0, 0.0))
    g = (rng.standard_normal(1 << 20) * 10.0 ** rng.uniform(-3, 0, 1 << 20)).astype(np.float32)
    c = Case([len(g)], [F32], [F32], 8)
    c.grads = [torch.from_numpy(g).cuda()]
    c.check(7, run=step(c, 7))


def test_values():
    c = Case(SIZES, [BF], [BF], 8)
    step(c, 1)()
    m, v = qn.adamw_values(c.state)
    for i in range(len(SIZES)):
        a, b, _, _ = c.parts(i)
        x, y = c.get(i)
        assert np.array_equal(host(m[a:b]), x) and np.array_equal(host(v[a:b]), y)
    c = Case(SIZES, [BF], [BF], 32)
    m, v = qn.adamw_values(c.state)
    assert m is c.state.m and v is c.state.v


@pytest.mark.parametrize("bits", [32, 8])
def test_step_and_rate_on_the_device(bits):
    """A captured step, replayed with a new step and rate each time."""
    say(f"[adamw] {bits} bits, captured")
    a, b = (Case([3000, 77], [BF], [BF], bits) for _ in range(2))
    n = torch.zeros(1, dtype=torch.int64, device="cuda")
    lr = torch.zeros(1, device="cuda")
    norm = torch.ones(1, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        n.add_(1)
        qn.adamw_step(a.params, a.grads, a.state, n, lr, norm=norm, max_norm=0.5)
    for i in range(1, 6):
        g = torch.Generator(device="cuda").manual_seed(i)
        for x, y in zip(a.grads, b.grads):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda") * 1e-3)
            y.copy_(x)
        norm.fill_(0.25 * i)
        lr.fill_(1e-2 / i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        qn.adamw_step(b.params, b.grads, b.state, i, float(lr), norm=norm, max_norm=0.5)
        torch.cuda.synchronize()
        assert int(n) == i
        # 1 - beta^t comes from other functions: one step of it
        for x, y in zip(a.params, b.params):
            assert torch.allclose(x.float(), y.float(), rtol=2.0 ** -7, atol=1e-7)
        assert torch.equal(a.state.m, b.state.m) and torch.equal(a.state.v, b.state.v)


def test_other_stream_and_rerun():
    for bits in (32, 8):
        a, b = (Case([30000], [BF], [BF], bits) for _ in range(2))
        step(a, 2)()
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        step(b, 2, stream=s)()
        s.synchronize()
        assert torch.equal(a.params[0], b.params[0])
        assert all(torch.equal(x, y) for x, y in zip(a.state.__dict__.values(), b.state.__dict__.values()) if x is not None)


def test_nothing_outside_is_touched():
    buf = torch.full((3, 1003), 9.0, dtype=BF, device="cuda")
    p = buf[1, 1:1000]
    s = qn.adamw_init([p], 8)
    big = [torch.zeros(1024 + 512, dtype=t.dtype, device="cuda") for t in (s.m, s.v)]
    scales = [torch.zeros(6, device="cuda") for _ in range(2)]
    for t in (*big, *scales):
        t.fill_(3)
        t[:1024 if t.numel() > 6 else 4] = 0
    qn.adamw_step([p], [torch.ones(999, device="cuda")], qn.AdamWState(*big, *scales), 1, 0.1)
    assert (buf[0] == 9).all() and (buf[2] == 9).all() and buf[1, 0] == 9 and (buf[1, 1000:] == 9).all()
    assert (p != 9).all()
    for t in big:
        assert (t[1024:] == 3).all() and not t[999:1024].any()
    for t in scales:
        assert (t[4:] == 3).all()


def test_past_32_bits():
    say("[adamw] 2^31 elements and more")
    n = (1 << 31) + 5000
    g = torch.zeros(n, dtype=BF, device="cuda")
    p = torch.zeros(n, dtype=BF, device="cuda")
    tail = torch.linspace(-1, 1, 4000, device="cuda").bfloat16()
    g[-4000:] = tail
    s = qn.adamw_init([p], 8)
    qn.adamw_step([p], [g], s, 1, 0.5, eps=1e-8, weight_decay=0.0)
    assert torch.allclose(p[-4000:].float(), -0.5 * tail.float().sign(), rtol=2.0 ** -7, atol=1e-6)
    assert not p[:-4000].any() and s.m[-5000:].any() and not s.m[:-5000].any()


# ---- the optimizer ----

def _module(seed=0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.nn.Parameter((0.1 * torch.randn(*s, generator=g, device="cuda")).to(dtype)) for s in ((8, 300), (77,), (0,))]


def _train(ps, opt, steps, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for _ in range(steps):
        opt.zero_grad()
        for p in ps:
            p.grad = torch.randn(p.shape, generator=g, device="cuda").to(p.dtype)
        opt.step()


def test_optimizer_follows_torch():
    for clip in (None, 0.5):
        a, b = _module(dtype=F32), _module(dtype=F32)
        x = qn.AdamW(a, lr=1e-2, weight_decay=0.1, max_norm=clip)
        y = torch.optim.AdamW(b, lr=1e-2, weight_decay=0.1)
        g = torch.Generator(device="cuda").manual_seed(1)
        for i in range(10):
            for p, q in zip(a, b):
                p.grad = torch.randn(p.shape, generator=g, device="cuda")
                q.grad = p.grad.clone()
            x.param_groups[0]["lr"] = y.param_groups[0]["lr"] = 1e-2 / (i + 1)
            if clip:
                norm = torch.nn.utils.clip_grad_norm_(b, clip)
            x.step()
            y.step()
            if clip:
                assert float(x.last_norm) == pytest.approx(float(norm), rel=1e-6)
        for p, q in zip(a, b):
            assert torch.allclose(p, q, rtol=1e-5, atol=1e-7)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("masters", [False, True])
def test_optimizer_state_comes_back(bits, masters):
    kw = dict(lr=1e-2, bits=bits, masters=masters, max_norm=1.0)
    a, b = _module(), _module()
    x = qn.AdamW(a, **kw)
    _train(a, x, 3)
    saved = {k: v for k, v in x.state_dict().items()}
    import copy
    saved = copy.deepcopy(saved)
    with torch.no_grad():
        for p, q in zip(a, b):
            q.copy_(p)
    y = qn.AdamW(b, **{**kw, "lr": 1.0})
    y.load_state_dict(saved)
    assert y.param_groups[0]["lr"] == 1e-2
    _train(a, x, 3, seed=2)
    _train(b, y, 3, seed=2)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    with pytest.raises(ValueError, match="other"):
        qn.AdamW(_module()[:1], **kw).load_state_dict(saved)
    with pytest.raises(ValueError, match="other"):
        qn.AdamW(_module(), **{**kw, "bits": 40 - bits}).load_state_dict(saved)


def test_masters_keep_small_updates():
    """Steps of 2^-12 of a parameter of 1: lost in bf16, kept in the master."""
    a, b = (torch.nn.Parameter(torch.ones(64, dtype=BF, device="cuda")) for _ in range(2))
    x = qn.AdamW([a], lr=2.0 ** -12, weight_decay=0.0, masters=True)
    y = qn.AdamW([b], lr=2.0 ** -12, weight_decay=0.0)
    for _ in range(64):
        a.grad = b.grad = torch.ones_like(a)
        x.step()
        y.step()
    assert (b == 1).all() and torch.allclose(a.float(), torch.full((64,), 1 - 64 * 2.0 ** -12, device="cuda"), atol=2.0 ** -8)


def test_masters_follow_loaded_parameters():
    a = [torch.nn.Parameter(torch.ones(300, dtype=BF, device="cuda"))]
    opt = qn.AdamW(a, lr=0.0, weight_decay=0.0, masters=True)
    with torch.no_grad():
        a[0].fill_(5.0)
    opt.take_masters()
    a[0].grad = torch.ones_like(a[0])
    opt.step()
    assert (a[0] == 5).all()


def test_optimizer_copies():
    import copy
    a = _module()
    x = qn.AdamW(a, lr=1e-2, bits=8, masters=True)
    _train(a, x, 2)
    b, y = copy.deepcopy((a, x))
    assert y.param_groups[0]["params"][0] is b[0]
    _train(a, x, 2, seed=3)
    _train(b, y, 2, seed=3)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_optimizer_with_a_schedule():
    a = _module()
    opt = qn.AdamW(a, lr=1.0, weight_decay=0.0)
    sched = torch.optim.lr_scheduler.LambdaLR(opt, lambda i: 0.0 if i else 1.0)
    _train(a, opt, 1)
    sched.step()
    before = [p.detach().clone() for p in a]
    _train(a, opt, 1)
    assert all(torch.equal(p, q) for p, q in zip(a, before))


def test_optimizer_groups_and_missing_gradients():
    a = _module()
    opt = qn.AdamW([{"params": a[:1], "lr": 0.0}, {"params": a[1:], "lr": 0.1}], weight_decay=0.0, bits=8)
    opt.step()                       # no gradients at all
    before = [p.detach().clone() for p in a]
    a[1].grad = torch.ones_like(a[1])
    opt.step()
    assert torch.equal(a[0], before[0]) and not torch.equal(a[1], before[1])
    a[0].grad = torch.ones_like(a[0])
    opt.step()
    assert torch.equal(a[0], before[0])


@pytest.mark.parametrize("make,error,match", [
    (lambda p, g, s: qn.adamw_step([], [], s, 1, 0.1), ValueError, "no parameters"),
    (lambda p, g, s: qn.adamw_step(p, g[:1], s, 1, 0.1), ValueError, "1 gradients for 2"),
    (lambda p, g, s: qn.adamw_step([p[0], p[0]], [g[0], g[0]], s, 1, 0.1), ValueError, "twice"),
    (lambda p, g, s: qn.adamw_step(p, [g[1], g[0]], s, 1, 0.1), ValueError, "another size"),
    (lambda p, g, s: qn.adamw_step(p, [g[1], None], s, 1, 0.1), ValueError, "another size"),
    (lambda p, g, s: qn.adamw_step(p, [g[0].half(), g[1]], s, 1, 0.1), TypeError, "grads must be"),
    (lambda p, g, s: qn.adamw_step([p[0].half(), p[1]], g, s, 1, 0.1), TypeError, "params must be"),
    (lambda p, g, s: qn.adamw_step(p, [x.cpu() for x in g], s, 1, 0.1), ValueError, "is on cpu"),
    (lambda p, g, s: qn.adamw_step([x.cpu() for x in p], g, s, 1, 0.1), ValueError, "is on cpu"),
    (lambda p, g, s: qn.adamw_step([p[0].view(20, 15).t(), p[1]], g, s, 1, 0.1), ValueError, "contiguous"),
    (lambda p, g, s: qn.adamw_step(p, g, qn.adamw_init(p[:1]), 1, 0.1), ValueError, "too few"),
    (lambda p, g, s: qn.adamw_step(p, g, qn.AdamWState(s.m[:100], s.v[:100]), 1, 0.1), ValueError, "multiple of 256"),
    (lambda p, g, s: qn.adamw_step(p, g, qn.AdamWState(s.m, s.v[:256]), 1, 0.1), ValueError, "state.v has shape"),
    (lambda p, g, s: qn.adamw_step(p, g, qn.AdamWState(s.m.to(torch.int8), s.v.to(torch.uint8)), 1, 0.1), TypeError, "m_scale"),
    (lambda p, g, s: qn.adamw_step(p, g, qn.AdamWState(s.m, s.v, s.m[:3], s.v[:3]), 1, 0.1), ValueError, "no scales"),
    (lambda p, g, s: qn.adamw_step(p, g, None, 1, 0.1), TypeError, "AdamWState"),
    (lambda p, g, s: qn.adamw_step(p, g, s, 1, 0.1, copies=[None]), ValueError, "1 copies"),
    (lambda p, g, s: qn.adamw_step(p, g, s, 1, 0.1, copies=[p[0], None]), TypeError, "copy has dtype"),
    (lambda p, g, s: qn.adamw_step(p, g, s, 1, 0.1, max_norm=1.0), ValueError, "together"),
    (lambda p, g, s: qn.adamw_step(p, g, s, 1, 0.1, norm=p[1][:2], max_norm=1.0), ValueError, "norm must be"),
    (lambda p, g, s: qn.adamw_step(p, g, s, 1, 0.1, norm=p[1][:1], max_norm=-1.0), ValueError, "max_norm"),
    (lambda p, g, s: qn.adamw_step(p, g, s, torch.ones(1, device="cuda"), 0.1), ValueError, "step must be"),
    (lambda p, g, s: qn.adamw_step(p, g, s, 1, torch.ones(2, device="cuda")), ValueError, "lr must be"),
    (lambda p, g, s: qn.adamw_step(p, g, s, 0, 0.1), qn.QloraError, "invalid"),
    (lambda p, g, s: qn.adamw_step(p, g, s, 1, -0.1), qn.QloraError, "invalid"),
    (lambda p, g, s: qn.adamw_step(p, g, s, 1, 0.1, betas=(1.0, 0.9)), qn.QloraError, "invalid"),
    (lambda p, g, s: qn.adamw_step(p, g, s, 1, 0.1, eps=-1.0), qn.QloraError, "invalid"),
])
def test_refusals(make, error, match):
    p = [torch.zeros(300, device="cuda"), torch.zeros(7, device="cuda")]
    g = [torch.ones_like(t) for t in p]
    with pytest.raises(error, match=match):
        make(p, g, qn.adamw_init(p))
    assert not p[0].any() and not p[1].any()


def test_tensor_lists():
    """The compiled reader of lists of tensors: what torch says of each, and
    None for whatever is not a contiguous tensor of the two types."""
    from quantized_base_lora_nf4_amd.train_ops import _TYPES, _describe
    base = torch.zeros(1000, device="cuda")
    ok = [base, base[3:9], base.view(10, 100)[2:4], torch.nn.Parameter(torch.zeros(5, 7, dtype=BF, device="cuda")),
          torch.zeros(0, 4, device="cuda"), base[7], base.view(1000, 1)[::2][:1], torch.zeros(3, 4, dtype=BF, device="cuda")[1:]]
    dev, ptrs, sizes, types = _describe(ok)
    assert dev == base.device and ptrs.tolist() == [t.data_ptr() for t in ok]
    assert sizes.tolist() == [t.numel() for t in ok] and types.tolist() == [_TYPES[t.dtype] for t in ok]
    for bad in (base[::2], base.view(10, 100).t(), base.half(), base.double(), base.cpu(), None, 3, base.to_sparse(),
                torch.zeros(2, device="meta")):
        assert _describe([base, bad]) is None and _describe([bad, base]) is None
    from quantized_base_lora_nf4_amd._lib import tensors
    fits, kinds = tensors().fits, {"s": [BF, torch.int16, torch.uint16], "f": [F32], "i": [torch.int32], "b": [torch.uint8],
                                   "c": [torch.int8]}
    x = torch.zeros(4, 6, device="cuda")
    every = [t for ts in kinds.values() for t in ts] + [torch.int64, torch.float64, torch.bool, torch.float16]
    for kind, types in kinds.items():
        for t in every:
            assert fits(0, kind, (x.to(t),), ((4, 6),)) == (t in types)
    assert fits(0, "fi", (x, x.int()[0]), ((4, 6), (6,)))
    for bad in ((1, "f", (x,), ((4, 6),)), (0, "f", (x,), ((6, 4),)), (0, "f", (x,), ((24,),)), (0, "f", (x,), ((4, 6, 1),)),
                (0, "f", (x.t(),), ((6, 4),)), (0, "f", (x.cpu(),), ((4, 6),)), (0, "ff", (x, None), ((4, 6), (4, 6))),
                (0, "z", (x,), ((4, 6),))):
        assert not fits(*bad)
    with pytest.raises(TypeError):
        fits(0, "f", (x,), ((4, "6"),))
