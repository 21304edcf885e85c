"""Tensors that a call writes into count a new version in torch, so that a
backward pass through a graph that saved them before raises instead of taking
the new values."""

import pytest
import torch

import quantized_base_lora_nf4_amd as qn

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def randn(*shape, seed=0, dtype=BF):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


@pytest.mark.parametrize("bits,masters", [(32, False), (8, True)])
def test_backward_after_a_step(bits, masters):
    """A retained graph over the adapter's old values."""
    layer = qn.QLoRALinear(randn(64, 128, dtype=F32), 8, 16.0)
    opt = qn.AdamW([layer.A, layer.B], lr=1e-2, bits=bits, masters=masters)
    x = randn(5, 128, seed=1)
    y = layer(x)
    y.sum().backward(retain_graph=True)
    y.sum().backward(retain_graph=True)   # nothing has changed: fine
    opt.step()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    layer(x).sum().backward()             # a new graph


def test_backward_after_rotation_in_place():
    f, _ = qn.rope_frequencies(64)
    q, w = randn(1, 5, 4, 64), randn(1, 5, 4, 64, seed=1).requires_grad_()
    y = q * w                             # saves q
    qn.rope_fwd(q, None, f, out=(q, None))
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def _calls():
    """(name, call, tensors written, tensors read)."""
    f, _ = qn.rope_frequencies(64)
    q, k, v = (randn(1, 5, h, 64, seed=h) for h in (4, 2, 2))
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    for call in (qn.rope_fwd, qn.rope_bwd):
        yield call.__name__, lambda: call(q, k, f, out=(qo, ko)), (qo, ko), (q, k, f)
        yield f"{call.__name__} of q", lambda: call(q, None, f, out=(qo, None)), (qo,), (q, f)
    o, lse = qn.attention_fwd(q, k, v)
    yield "attention_fwd", lambda: qn.attention_fwd(q, k, v, out=qo), (qo,), (q, k, v)
    do, vo = randn(1, 5, 4, 64, seed=9), torch.empty_like(v)
    yield ("attention_bwd", lambda: qn.attention_bwd(q, k, v, o, lse, do, out=(qo, ko, vo)), (qo, ko, vo),
           (q, k, v, o, lse, do))
    x, wt = randn(7, 128), torch.ones(128, device="cuda")
    xo = torch.empty_like(x)
    yield "norm_fwd", lambda: qn.norm_fwd(x, wt, rms=True, out=xo), (xo,), (x, wt)
    g, h = [randn(300, seed=3), randn(7, seed=4)], [torch.empty(300, dtype=BF, device="cuda"),
                                                    torch.empty(7, dtype=BF, device="cuda")]
    flat = torch.empty(307, dtype=BF, device="cuda")
    yield "clip_grad_norm", lambda: qn.clip_grad_norm(g, 0.5, out=h), h, g
    yield "clip_grad_norm flat", lambda: qn.clip_grad_norm(g, 0.5, out=flat), (flat,), g
    yield "grad_norm", lambda: qn.grad_norm(g), (), g
    i = [t.clone() for t in g]
    yield "clip_grad_norm in place", lambda: qn.clip_grad_norm(i, 0.5), i, ()
    p, c = [randn(300, dtype=F32), randn(7, dtype=F32)], [torch.empty(300, dtype=BF, device="cuda"), None]
    for bits in (32, 8):
        s = qn.adamw_init(p, bits)
        own = [t for t in (s.m, s.v, s.m_scale, s.v_scale) if t is not None]
        yield (f"adamw_step {bits}", lambda: qn.adamw_step(p, [g[0], None], s, 1, 0.1, copies=c),
               (p[0], c[0], *own), (p[1], *g))
    W = randn(64, 128, dtype=F32)
    w = qn.nf4_quantize(W)
    X, A, B, Y = randn(5, 128), randn(8, 128), randn(64, 8), torch.empty(5, 64, dtype=BF, device="cuda")
    U = torch.empty(5, 8, dtype=BF, device="cuda")
    state = (w.codes, w.q8, w.step)
    yield "qlora_linear_fwd", lambda: qn.qlora_linear_fwd(w, X, A, B, 2.0, Y=Y, U_out=U), (Y, U), (X, A, B, *state)
    yield ("qlora_linear_fwd_noalloc", lambda: qn.qlora_linear_fwd_noalloc(w, X, A, B, 2.0, Y, U_out=U), (Y, U),
           (X, A, B, *state))
    grads = [torch.empty_like(t) for t in (X, A, B)]
    dY = randn(5, 64, seed=5)
    yield ("qlora_linear_bwd", lambda: qn.qlora_linear_bwd(w, X, dY, A, B, 2.0, out=tuple(grads)), grads,
           (X, A, B, dY, *state))
    index, sc = torch.zeros(5, dtype=torch.int32, device="cuda"), torch.ones(1, device="cuda")
    yield ("qlora_linear_multi_fwd", lambda: qn.qlora_linear_multi_fwd(w, X, A[None], B[None], sc, index, Y=Y), (Y,),
           (X, A, B, sc, index, *state))
    full = torch.empty(64, 128, dtype=BF, device="cuda")
    yield "nf4_dequantize", lambda: qn.nf4_dequantize(w, out=full), (full,), state
    into = qn.alloc_nf4(64, 128)
    yield "nf4_quantize", lambda: qn.nf4_quantize(W, out=into), (into.codes, into.q8, into.step), (W,)
    e = torch.empty(1, dtype=torch.float64, device="cuda")
    yield "quant_error", lambda: qn.quant_error(W, out=e), (e,), (W,)


def test_written_tensors_count_a_version():
    for name, call, written, read in _calls():
        before = [t._version for t in written], [t._version for t in read]
        call()
        assert all(t._version > b for t, b in zip(written, before[0])), name
        assert [t._version for t in read] == before[1], name


def test_a_refused_call_counts_none():
    f, _ = qn.rope_frequencies(64)
    q = randn(1, 5, 4, 64)
    before = q._version
    with pytest.raises(qn.QloraError):
        qn.rope_fwd(q, None, f, scale=float("inf"), out=(q, None))
    p = [randn(300, dtype=F32)]
    with pytest.raises(qn.QloraError):
        qn.adamw_step(p, p, qn.adamw_init(p), 1, -1.0)
    assert q._version == before and p[0]._version == 0


def test_inference_tensors():
    """They have no version: the calls take them as before, inside and outside
    of inference mode."""
    f, _ = qn.rope_frequencies(64)

    def both(p, q):
        qn.adamw_step([p], [p.clone()], qn.adamw_init([p]), 1, 1e-2)
        qn.rope_fwd(q, None, f, out=(q, None))
        qn.clip_grad_norm([p], 0.5)
        return p.clone(), q.clone()
    want = both(randn(300, dtype=F32), randn(1, 5, 4, 64))
    with torch.inference_mode():
        p, q = randn(300, dtype=F32), randn(1, 5, 4, 64)
        assert p.is_inference()
        r, t = p.clone(), q.clone()
        got = both(p, q)
    after = both(r, t)
    for other in (got, after):
        assert all(torch.equal(a, b) for a, b in zip(want, other))
