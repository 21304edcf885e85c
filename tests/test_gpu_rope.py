"""Rotary positions against the oracle in extended precision.

Tolerance per element: the output is rounded once to bf16 (2^-8 of its value at
most); before that come cos and sin in fp32 (2 units in the last place and the
product with scale), a product and a fused multiply-add: 2^-20 of t (|x| + |y|)
covers them; and the angle, in fp64, is off by at most 2^-51 of its size.
"""

import numpy as np
import pytest
import torch

import quantized_base_lora_nf4_amd as qn
from gpu_util import say
from oracle import rope as oracle

pytestmark = pytest.mark.gpu


def randn(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def check(name, got, x, positions, f, interleaved, scale, inverse):
    """got, x [rows, heads, dim]."""
    f = f.cpu().numpy()
    ref = oracle.rotate(host(x), positions, f, interleaved, scale, inverse)
    n = len(f)
    size = np.zeros_like(ref)
    far = max([abs(int(p)) for p in positions if p is not None], default=0)
    a = np.abs(host(x))
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
    both = abs(scale) * (a[..., first] + a[..., second])
    size[..., first] = size[..., second] = both * (2.0 ** -20 + far * f * 2.0 ** -51)
    rot = np.array([p is not None for p in positions])[:, None, None]
    tol = np.where(rot, np.abs(ref) * 2.0 ** -8 * (1 + 2.0 ** -8) + size, 0.0)
    tol[..., 2 * n:] = 0.0   # copied
    err = np.abs(host(got) - ref)
    say(f"    {name}: {float((err / np.maximum(tol, 1e-30)).max(initial=0)):.3f} of the bound")
    assert (err <= tol).all(), name


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 128), (128, 64), (96, 96), (80, 20), (80, 80),
                                     (8, 2), (8, 8), (136, 34), (128, 126), (1024, 1024), (256, 2)])
def test_head_sizes(dim, rot, interleaved):
    say(f"[rope] heads of {dim}, {rot} rotated, interleaved {interleaved}")
    f, scale = qn.rope_frequencies(rot, scaling="parts" if rot > 8 else None, factor=4.0)
    q, k = randn(2, 19, 5, dim), randn(2, 19, 1, dim, seed=1)
    for inverse, call in ((False, qn.rope_fwd), (True, qn.rope_bwd)):
        a, b = call(q, k, f, interleaved=interleaved, scale=scale)
        assert a.is_contiguous() and a.shape == q.shape and b.shape == k.shape
        pos = list(range(19)) * 2
        check("q", a.flatten(0, 1), q.flatten(0, 1), pos, f, interleaved, scale, inverse)
        check("k", b.flatten(0, 1), k.flatten(0, 1), pos, f, interleaved, scale, inverse)


@pytest.mark.parametrize("rows", [1, 2, 63, 700, 5000])
@pytest.mark.parametrize("heads,kv", [(1, 1), (32, 8), (40, 40)])
def test_lengths(rows, heads, kv):
    say(f"[rope] {rows} rows, {heads}/{kv} heads")
    f, _ = qn.rope_frequencies(64)
    qkv = randn(1, rows, heads + 2 * kv, 64)
    q, k, v = qkv.split([heads, kv, kv], 2)
    a, b = qn.rope_fwd(q, k, f)
    check("q", a[0], q[0], range(rows), f, False, 1.0, False)
    check("k", b[0], k[0], range(rows), f, False, 1.0, False)
    # in place: the same bits, and v as it was
    before = v.clone()
    c, d = qn.rope_fwd(q, k, f, out=(q, k))
    assert c is q and d is k
    assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(v, before)


def test_no_rows():
    f, _ = qn.rope_frequencies(64)
    for lead in ((0, 5), (3, 0)):
        a, b = qn.rope_fwd(randn(*lead, 2, 64), randn(*lead, 1, 64), f)
        assert a.shape == (*lead, 2, 64) and b.shape == (*lead, 1, 64)
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    a, _ = qn.rope_fwd(randn(0, 2, 64), None, f, cu_seqlens=cu)
    assert a.shape == (0, 2, 64)
    x = randn(5, 2, 64)   # rows, but no sequence
    a, _ = qn.rope_fwd(x, None, f, cu_seqlens=cu)
    assert torch.equal(a, x)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_given_positions(dtype):
    say(f"[rope] positions {dtype}")
    f, scale = qn.rope_frequencies(128, scaling="bands", factor=8.0, high=4.0)
    g = torch.Generator().manual_seed(2)
    q, k = randn(3, 7, 4, 128), randn(3, 7, 2, 128, seed=1)
    top = 2 ** 31 - 1 if dtype == torch.int32 else 2 ** 40
    pos = torch.randint(-top, top, (3, 7), generator=g).to(dtype)
    pos[0, 0] = top
    pos[0, 1] = -1

    def one(p, flat):
        a, b = qn.rope_fwd(q, k, f, positions=p, scale=scale)
        check("q", a.flatten(0, 1), q.flatten(0, 1), flat, f, False, scale, False)
        check("k", b.flatten(0, 1), k.flatten(0, 1), flat, f, False, scale, False)
    one(pos.cuda(), pos.flatten().tolist())
    one(pos[0].cuda(), pos[0].tolist() * 3)                      # for all sequences
    one(pos[:1].cuda(), pos[0].tolist() * 3)
    one(pos[:, :1].cuda().expand(3, 7), pos[:, :1].expand(3, 7).flatten().tolist())  # stride 0
    one(pos.t().contiguous().cuda().t(), pos.flatten().tolist())
    # packed
    a, b = qn.rope_fwd(q.flatten(0, 1), None, f, positions=pos.flatten().cuda(), scale=scale)
    assert b is None
    check("packed", a, q.flatten(0, 1), pos.flatten().tolist(), f, False, scale, False)


@pytest.mark.parametrize("cu", [[0, 5], [0, 0, 3, 3, 40, 41, 41], [0, 20, 60], [0] + list(range(1, 61)), [0, 0]])
def test_packed(cu):
    say(f"[rope] offsets {cu[:8]}")
    f, _ = qn.rope_frequencies(64)
    rows = 60
    q, k = randn(rows, 6, 64), randn(rows, 3, 64, seed=1)
    c = torch.tensor(cu, dtype=torch.int32, device="cuda")
    pos = oracle.packed_positions(rows, cu)
    for inverse, call in ((False, qn.rope_fwd), (True, qn.rope_bwd)):
        a, b = call(q, k, f, cu_seqlens=c)
        check("q", a, q, pos, f, False, 1.0, inverse)
        check("k", b, k, pos, f, False, 1.0, inverse)
    p, _ = qn.rope_fwd(q, None, f, interleaved=True, cu_seqlens=c)
    check("interleaved", p, q, pos, f, True, 1.0, False)
    qn.rope_fwd(q, k, f, cu_seqlens=c, out=(q, k))   # in place: rows of no sequence as they were
    a, b = qn.rope_bwd(q, k, f, cu_seqlens=c)
    assert a.shape == q.shape


def test_wrong_offsets_stay_inside():
    f, _ = qn.rope_frequencies(64)
    buf = randn(80, 2, 64)
    x = buf[10:70]
    out = torch.full_like(buf, 7.0)
    for cu in ([5, 2, 90], [0, 1 << 30], [-9, 30, 20], [100, 200]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        a, _ = qn.rope_fwd(x, None, f, cu_seqlens=c, out=(out[10:70], None))
        assert (out[:10] == 7).all() and (out[70:] == 7).all()
        # a rotation by any angle keeps a pair's length: two roundings
        n = a.float().unflatten(-1, (2, 32)).square().sum(-2).sqrt()
        m = x.float().unflatten(-1, (2, 32)).square().sum(-2).sqrt()
        assert torch.allclose(n, m, rtol=2.0 ** -7, atol=0)


def test_infinities_and_nan_stay_in_their_pair():
    f, _ = qn.rope_frequencies(32)
    x = randn(1, 4, 2, 64)
    for interleaved in (False, True):
        y, _ = qn.rope_fwd(x, None, f, interleaved=interleaved)
        z = x.clone()
        z[0, 2, 1, 3], z[0, 2, 1, 40] = float("nan"), float("inf")
        w, _ = qn.rope_fwd(z, None, f, interleaved=interleaved)
        pair = (3, 2 if interleaved else 3 + 16)
        odd = torch.zeros_like(x, dtype=torch.bool)
        odd[0, 2, 1, list(pair)] = True
        assert w[odd].isnan().all() and w[0, 2, 1, 40] == float("inf")
        odd[0, 2, 1, 40] = True
        assert torch.equal(w[~odd], y[~odd])


def test_strided_views_and_layouts():
    f, _ = qn.rope_frequencies(48)
    base = randn(3, 4, 9, 72)                       # [batch, head, row, 72]
    q = base[..., 8:72].transpose(1, 2)             # heads before rows, offset inside
    k = randn(1, 9, 2, 64, seed=3).expand(3, 9, 2, 64)   # one key for every sequence
    out = torch.full((3, 4, 9, 72), 3.0, dtype=torch.bfloat16, device="cuda")
    qo = out[..., :64].transpose(1, 2)
    a, b = qn.rope_fwd(q, k, f, out=(qo, torch.empty(3, 9, 2, 64, dtype=torch.bfloat16, device="cuda")))
    check("q", a.reshape(27, 4, 64), q.reshape(27, 4, 64), list(range(9)) * 3, f, False, 1.0, False)
    check("k", b.reshape(27, 2, 64), k.reshape(27, 2, 64), list(range(9)) * 3, f, False, 1.0, False)
    assert (out[..., 64:] == 3).all()


def test_gradients_against_differences():
    """The rotation is linear: the gradient of <w, rope(x)> at x is rope_bwd(w),
    and <w, rope(d)> = <rope_bwd(w), d> for any d (roundings of 2^-8 of each
    element, independent, over 2560 terms)."""
    f, scale = qn.rope_frequencies(64, scaling="parts", factor=2.0)
    q = randn(2, 5, 4, 64).requires_grad_()
    k = randn(2, 5, 2, 64, seed=1).requires_grad_()
    wq, wk = randn(2, 5, 4, 64, seed=2), randn(2, 5, 2, 64, seed=3)
    for interleaved in (False, True):
        a, b = qn.rope(q, k, f, interleaved=interleaved, scale=scale)
        gq, gk = torch.autograd.grad([a, b], [q, k], [wq, wk])
        x, y = qn.rope_bwd(wq, wk, f, interleaved=interleaved, scale=scale)
        assert torch.equal(gq, x) and torch.equal(gk, y)
        for t, g, w, o in ((q, gq, wq, a), (k, gk, wk, b)):
            left = (w.double() * o.detach().double())
            right = (g.double() * t.detach().double())
            slack = 2.0 ** -8 * float(torch.sqrt(left.square().sum() + right.square().sum())) * 4
            assert abs(float(left.sum() - right.sum())) <= slack
    # one of the two alone
    a, b = qn.rope(q, k, f)
    only, = torch.autograd.grad(b, [k], wk, retain_graph=True)
    assert torch.equal(only, qn.rope_bwd(wk, None, f)[0])
    only, = torch.autograd.grad(a, [q], wq)
    assert torch.equal(only, qn.rope_bwd(wq, None, f)[0])
    a, _ = qn.rope(q, None, f)
    only, = torch.autograd.grad(a, [q], wq)
    assert torch.equal(only, qn.rope_bwd(wq, None, f)[0])


def test_broadcast_gradient():
    """A gradient of strides the kernels do not take (sum's is one number)."""
    f, _ = qn.rope_frequencies(64)
    q = randn(2, 5, 4, 64).requires_grad_()
    a, _ = qn.rope(q, None, f)
    a.sum().backward()
    assert torch.equal(q.grad, qn.rope_bwd(torch.ones_like(q), None, f)[0])


def test_other_stream_and_rerun():
    f, _ = qn.rope_frequencies(128)
    q, k = randn(1, 300, 8, 128), randn(1, 300, 8, 128, seed=1)
    a, b = qn.rope_fwd(q, k, f)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    c, d = qn.rope_fwd(q, k, f, stream=s)
    s.synchronize()
    assert torch.equal(a, c) and torch.equal(b, d)


def test_captured():
    f, _ = qn.rope_frequencies(64)
    q, k = randn(4, 1, 8, 64), randn(4, 1, 2, 64, seed=1)
    pos = torch.zeros(4, 1, dtype=torch.int64, device="cuda")
    qn.rope_fwd(q, k, f, positions=pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a, b = qn.rope_fwd(q, k, f, positions=pos)
    for i in range(4):
        pos.fill_(100 * i + 7)
        q.copy_(randn(4, 1, 8, 64, seed=10 + i))
        c, d = qn.rope_fwd(q, k, f, positions=pos)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, c) and torch.equal(b, d)


def test_offsets_past_32_bits():
    """Rows that lie more than 2^32 bytes into a tensor."""
    say("[rope] 2^31 elements and more")
    f, _ = qn.rope_frequencies(128)
    rows = (1 << 31) // (8 * 128) + 300
    x = torch.zeros(1, rows, 8, 128, dtype=torch.bfloat16, device="cuda")
    tail = randn(1, 200, 8, 128)
    x[:, -200:] = tail
    y, _ = qn.rope_fwd(x, None, f)
    check("tail", y[0, -200:], tail[0], range(rows - 200, rows), f, False, 1.0, False)
    assert not y[0, :-200].any()


@pytest.mark.parametrize("make,error,match", [
    (lambda q, k, f: qn.rope_fwd(q[0, 0], k, f), ValueError, "dimensions"),
    (lambda q, k, f: qn.rope_fwd(q, k[0], f), ValueError, "dimensions"),
    (lambda q, k, f: qn.rope_fwd(q, k[:, :3], f), ValueError, "k has shape"),
    (lambda q, k, f: qn.rope_fwd(q.float(), k, f), TypeError, "q must be bf16"),
    (lambda q, k, f: qn.rope_fwd(q, k.cpu(), f), ValueError, "k is on cpu"),
    (lambda q, k, f: qn.rope_fwd(q, k, f.float()), TypeError, "inv_freq has dtype"),
    (lambda q, k, f: qn.rope_fwd(q, k, f.cpu()), ValueError, "inv_freq is on cpu"),
    (lambda q, k, f: qn.rope_fwd(q, k, torch.cat([f, f])), ValueError, "inv_freq has 64"),
    (lambda q, k, f: qn.rope_fwd(q, k, f[:0]), ValueError, "inv_freq has 0"),
    (lambda q, k, f: qn.rope_fwd(q, k, f, positions=torch.zeros(2, 5, device="cuda")), TypeError, "positions has dtype"),
    (lambda q, k, f: qn.rope_fwd(q, k, f, positions=torch.zeros(2, 4, dtype=torch.int64, device="cuda")), ValueError, "positions has shape"),
    (lambda q, k, f: qn.rope_fwd(q, k, f, positions=torch.zeros(2, 5, dtype=torch.int64)), ValueError, "positions is on cpu"),
    (lambda q, k, f: qn.rope_fwd(q, k, f, cu_seqlens=torch.zeros(2, dtype=torch.int32, device="cuda")), ValueError, "3 dimensions"),
    (lambda q, k, f: qn.rope_fwd(q[0], k[0], f, cu_seqlens=torch.zeros(2, device="cuda")), TypeError, "cu_seqlens has dtype"),
    (lambda q, k, f: qn.rope_fwd(q, k, f, out=(q, q[:, :, :2])), qn.QloraError, "invalid"),
    (lambda q, k, f: qn.rope_fwd(q, k, f, out=(k.new_empty(2, 5, 4, 64), q[:, :, :2])), qn.QloraError, "invalid"),
    (lambda q, k, f: qn.rope_fwd(q, k, f, out=(k.new_empty(1, 5, 4, 64).expand(2, 5, 4, 64), k)), qn.QloraError, "invalid"),
    (lambda q, k, f: qn.rope_fwd(q, k, f, out=(k, k)), ValueError, "out.0. has shape"),
    (lambda q, k, f: qn.rope_fwd(q, k, f, scale=float("inf")), qn.QloraError, "invalid"),
    (lambda q, k, f: qn.rope_fwd(torch.cat([q] * 17, -1), None, f), qn.QloraError, "unsupported"),
    (lambda q, k, f: qn.rope_fwd(q[..., :60], k[..., :60], f[:30]), qn.QloraError, "unsupported"),
])
def test_refusals(make, error, match):
    f, _ = qn.rope_frequencies(64)
    q, k = randn(2, 5, 4, 64), randn(2, 5, 2, 64)
    with pytest.raises(error, match=match):
        make(q, k, f)
