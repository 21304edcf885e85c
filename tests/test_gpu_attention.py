"""Attention on the GPU against the fp64 oracle on the same bf16 inputs.

Tolerances follow from the roundings the kernels state (probabilities, dS and
outputs to bf16, everything else fp32).  Per element, the error is at most the
oracle's budget `lim` (every rounding at its worst) plus 1 % of it and an fp32
share: sums of n fp32 terms and the exponentials are within 2^-14 of the sum of
the terms' magnitudes, which `lim` / U bounds.  Over a whole tensor, the
Frobenius norm of the error is at most the root of the summed variances (every
rounding counted with the largest variance that its relative error can have,
twice the average over the significands), again with the fp32 share.
lse: scores within (D + 2) 2^-24 of scale sum |q k|, the sum of exponentials
within (n + 64) 2^-24, the logarithm within 2^-21 of itself and of 1.
"""

import numpy as np
import pytest
import torch

import quantized_base_lora_nf4_amd as qn
from oracle import attention as oracle
from gpu_util import say

pytestmark = pytest.mark.gpu

F32_SHARE = 2.0 ** -14 / oracle.U   # of the budget


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    qn.lib()


def draw(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(torch.bfloat16).cuda()


def host(t):
    return t.detach().double().cpu().numpy()


def flat(t, packed):
    """[rows, heads, dim] in fp64."""
    h = host(t)
    return h if packed else h.reshape(-1, *h.shape[2:])


def close(name, got, ref, budget):
    lim, var = budget
    assert np.all(np.isfinite(got)), f"{name}: non-finite output"
    err = np.abs(got - ref)
    allowed = lim * (1.01 + F32_SHARE) + 1e-30
    worst = float((err / allowed).max(initial=0.0))
    off = float(np.sqrt((err ** 2).sum()))
    may = float(np.sqrt(var.sum())) + F32_SHARE * float(np.sqrt((lim ** 2).sum())) + 1e-30
    say(f"    {name}: worst element {worst:.3f} of its bound, Frobenius {off / may:.3f} of its")
    assert worst <= 1.0, f"{name}: an element is {worst:.3g} times its bound off"
    assert off <= may, f"{name}: Frobenius error {off:.3g}, at most {may:.3g}"


def check_lse(got, ref, q, k, seqs, scale, D):
    assert np.array_equal(np.isneginf(got), np.isneginf(ref))
    H, share = q.shape[1], q.shape[1] // k.shape[1]
    for a, b in seqs:
        n = b.stop - b.start
        for h in range(H):
            if n == 0 or a.stop == a.start:
                continue
            s = (np.abs(q[a, h]) @ np.abs(k[b, h // share]).T).max(1) * scale
            tol = (D + 2) * 2.0 ** -24 * s + (n + 64) * 2.0 ** -24
            r = ref[h, a]
            fine = np.isfinite(r)
            tol = tol + 2.0 ** -21 * (1 + np.abs(np.where(fine, r, 0.0)))
            assert np.all(np.abs(got[h, a][fine] - r[fine]) <= tol[fine])


def check_all(q, k, v, do, causal, scale=None, cu=None, cu_k=None, out=None, fwd_out=None,
              stream=None):
    """Forward and backward against the oracle; returns the outputs."""
    packed = cu is not None
    D = q.shape[-1]
    sc = 1.0 / np.sqrt(D) if scale is None else scale
    o, lse = qn.attention_fwd(q, k, v, causal, scale, cu, cu_k, out=fwd_out, stream=stream)
    dq, dk, dv = qn.attention_bwd(q, k, v, o, lse, do, causal, scale, cu, cu_k, out=out,
                                  stream=stream)
    torch.cuda.synchronize()
    if packed:
        cq = cu.tolist()
        ck = cq if cu_k is None else cu_k.tolist()
        seqs = oracle.sequences(0, 0, cq, ck)
    else:
        seqs = oracle.sequences(q.shape[1], k.shape[1], batch=q.shape[0])
    fq, fk, fv, fdo = (flat(t, packed) for t in (q, k, v, do))
    if packed:  # what lies outside every sequence is not looked at
        fq, fk, fv, fdo = (np.where(np.isfinite(t), t, 0.0) for t in (fq, fk, fv, fdo))
    r = oracle.run(fq, fk, fv, seqs, sc, causal, fdo)
    close("o", flat(o, packed), r.o, r.budget["o"])
    got = host(lse)
    if not packed:
        got = got.transpose(1, 0, 2).reshape(q.shape[2], -1)
    check_lse(got, r.lse, fq, fk, seqs, sc, D)
    for name, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        close(name, flat(t, packed), getattr(r, name), r.budget[name])
    return o, lse, dq, dk, dv


# batch, queries, keys, heads, key/value heads, dim, causal
DENSE = [
    (1, 1, 1, 1, 1, 64, True),
    (1, 1, 1, 1, 1, 128, False),
    (2, 5, 5, 2, 1, 64, True),
    (1, 31, 31, 1, 1, 128, True),
    (1, 33, 33, 2, 2, 64, True),
    (1, 64, 64, 2, 2, 128, True),
    (3, 65, 65, 2, 1, 128, True),
    (1, 128, 128, 1, 1, 128, False),
    (1, 127, 129, 4, 2, 128, True),      # the diagonal lies two keys to the right
    (1, 129, 127, 4, 1, 128, True),      # two queries see nothing
    (1, 200, 3, 2, 2, 64, True),         # most queries see nothing
    (1, 300, 130, 2, 1, 128, True),      # whole tiles of queries see nothing
    (2, 33, 300, 8, 2, 80, False),
    (2, 33, 300, 8, 2, 80, True),        # a chunk at the end of a longer sequence
    (1, 1, 515, 4, 4, 128, True),        # one query
    (1, 1, 700, 8, 1, 64, False),
    (1, 300, 1, 2, 1, 96, False),        # one key
    (1, 257, 257, 3, 3, 8, True),
    (1, 400, 400, 5, 5, 40, True),
    (2, 193, 193, 6, 2, 72, False),
    (1, 640, 640, 2, 1, 128, True),
    (1, 511, 1025, 2, 2, 128, True),
    (1, 1025, 511, 2, 2, 64, False),
    (5, 97, 97, 7, 7, 120, True),
    # walks that several workgroups share
    (1, 1, 5000, 2, 1, 128, True),
    (1, 40, 3001, 1, 1, 64, False),
    (1, 3001, 40, 4, 1, 128, False),
    (1, 3001, 40, 4, 1, 128, True),
    (1, 1500, 1500, 4, 1, 128, True),
    (2, 777, 1300, 2, 1, 40, True),
]


@pytest.mark.parametrize("case", DENSE, ids=lambda c: "x".join(map(str, c)))
def test_dense(case):
    B, lq, lk, H, Hk, D, causal = case
    say(f"[attention] {case}")
    q, do = draw(1, B, lq, H, D, std=1.5), draw(2, B, lq, H, D, std=1e-2)
    k, v = draw(3, B, lk, Hk, D), draw(4, B, lk, Hk, D)
    check_all(q, k, v, do, causal)


def test_probabilities_that_are_almost_one_hot():
    """Scores spread over hundreds: every row's reference moves many times."""
    say("[attention] large scores")
    q, do = draw(1, 1, 300, 2, 64, std=30.0), draw(2, 1, 300, 2, 64)
    k, v = draw(3, 1, 300, 2, 64, std=3.0), draw(4, 1, 300, 2, 64)
    # the fp32 share of the scores' error here is |scores| (D + 2) 2^-24 <= 2^-9 of a
    # probability only where scores exceed 500; the forward is checked on that share
    o, lse = qn.attention_fwd(q, k, v, True)
    torch.cuda.synchronize()
    r = oracle.run(flat(q, False), flat(k, False), flat(v, False), oracle.sequences(300, 300),
                   1 / 8, True)
    lim, _ = r.budget["o"]
    s = (np.abs(flat(q, False)) @ np.abs(flat(k, False)).transpose(1, 2, 0).max(-1).T).max() / 8
    share = 66 * 2.0 ** -24 * s / oracle.U
    assert np.all(np.abs(flat(o, False) - r.o) <= lim * (1.01 + F32_SHARE + 2 * share))


def test_rising_scores_move_the_reference_in_every_tile():
    """Keys along the queries' direction, growing with the position: the
    running maximum grows in every tile, by more and by less than the slack."""
    say("[attention] rising scores")
    n, D = 400, 64
    base = torch.randn(D, generator=torch.Generator().manual_seed(5))
    base = base / base.norm() * 8
    ramp = torch.linspace(0.0, 6.0, n)[:, None, None]
    q = (base + 0.1 * torch.randn(n, 1, D, generator=torch.Generator().manual_seed(6)))
    k = base * ramp + 0.1 * torch.randn(n, 1, D, generator=torch.Generator().manual_seed(7))
    q, k = (t.to(torch.bfloat16).cuda()[None] for t in (q, k))
    check_all(q, k, draw(8, 1, n, 1, D), draw(9, 1, n, 1, D, std=1e-2), False)
    check_all(q, k.flip(1).contiguous(), draw(8, 1, n, 1, D), draw(9, 1, n, 1, D, std=1e-2), True)


PACKED = [
    # lengths, heads, key/value heads, dim, causal, rows past the last sequence
    ([1], 1, 1, 64, True, 0),
    ([5, 0, 130, 1, 64, 0, 63, 300], 2, 1, 128, True, 0),
    ([64, 64, 128], 4, 2, 64, False, 0),
    ([100, 29], 2, 2, 128, True, 200),          # the tail is a tile and more
    ([0, 0, 0], 2, 1, 64, True, 70),
    ([3] * 150, 1, 1, 64, True, 5),             # more sequences than lanes
    ([129, 257, 511], 5, 5, 80, True, 1),
    ([900, 3, 1100], 4, 1, 128, True, 150),     # shared walks
    ([2, 1700, 1, 140, 1, 300], 2, 2, 64, True, 0),  # tile counts far apart
]


@pytest.mark.parametrize("case", PACKED, ids=lambda c: f"{len(c[0])}seqs-{sum(c[0])}-{c[1:]}")
def test_packed(case):
    lens, H, Hk, D, causal, tail = case
    say(f"[attention] packed {case}")
    T = sum(lens) + tail
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    ts = [draw(i, T, h, D, std=s) for i, (h, s) in enumerate(((H, 1.5), (Hk, 1), (Hk, 1), (H, 1e-2)))]
    for t in ts:   # nothing of the tail may reach an output
        t[sum(lens):] = float("nan")
    o, lse, dq, dk, dv = check_all(*ts, causal, cu=cu)
    n = sum(lens)
    assert not o[n:].any() and not dq[n:].any() and not dk[n:].any() and not dv[n:].any()
    assert torch.isneginf(lse[:, n:]).all()


def test_packed_with_other_keys():
    """Queries and keys of different lengths, one side or both empty."""
    say("[attention] packed, two offset arrays")
    lq, lk = [70, 0, 5, 200, 40], [100, 9, 0, 130, 41]
    cq, ck = (torch.tensor(np.cumsum([0] + n), dtype=torch.int32, device="cuda") for n in (lq, lk))
    q, do = draw(1, sum(lq), 4, 64, std=1.5), draw(2, sum(lq), 4, 64, std=1e-2)
    k, v = draw(3, sum(lk), 2, 64), draw(4, sum(lk), 2, 64)
    for causal in (True, False):
        check_all(q, k, v, do, causal, cu=cq, cu_k=ck)


def test_packed_without_sequences():
    say("[attention] packed, no sequences")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, k = draw(1, 200, 2, 64), draw(2, 200, 1, 64)
    o, lse = qn.attention_fwd(q, k, k, cu_seqlens=cu)
    dq, dk, dv = qn.attention_bwd(q, k, k, o, lse, q, cu_seqlens=cu)
    torch.cuda.synchronize()
    assert not o.any() and torch.isneginf(lse).all()
    assert not dq.any() and not dk.any() and not dv.any()


def test_offsets_that_are_wrong_stay_inside_the_tensors():
    """Negative, descending and too large offsets: outputs are undefined, but
    every access stays within the rows (the kernels clamp)."""
    say("[attention] wrong offsets")
    q, k = draw(1, 300, 2, 64), draw(2, 300, 1, 64)
    for bad in ([0, 400, 300], [-5, 100, 300], [0, 200, 100], [250, 20, 299], [0, 1 << 30, -(1 << 30)]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        o, lse = qn.attention_fwd(q, k, k, cu_seqlens=cu)
        qn.attention_bwd(q, k, k, o, lse, q, cu_seqlens=cu)
    torch.cuda.synchronize()


def test_neighbours_of_a_sequence_never_reach_it():
    """NaN in the sequence before and after: the one between is unaffected."""
    say("[attention] NaN next door")
    lens = [50, 77, 60]
    cu = torch.tensor(np.cumsum([0] + lens), dtype=torch.int32, device="cuda")
    ts = [draw(i, sum(lens), 2, 128) for i in range(4)]
    ref = [t[50:127].clone().contiguous() for t in ts]
    for t in ts:
        t[:50] = float("nan")
        t[127:] = float("inf")
    o, lse = qn.attention_fwd(*ts[:3], True, cu_seqlens=cu)
    got = qn.attention_bwd(*ts[:3], o, lse, ts[3], True, cu_seqlens=cu)
    one = torch.tensor([0, 77], dtype=torch.int32, device="cuda")
    o1, lse1 = qn.attention_fwd(*ref[:3], True, cu_seqlens=one)
    exp = qn.attention_bwd(*ref[:3], o1, lse1, ref[3], True, cu_seqlens=one)
    torch.cuda.synchronize()
    assert torch.equal(o[50:127], o1) and torch.equal(lse[:, 50:127], lse1)
    for a, b in zip(got, exp):
        assert torch.equal(a[50:127], b)


def test_views_of_one_projection_and_outputs_into_one():
    say("[attention] strided")
    B, S, H, Hk, D = 2, 150, 4, 2, 64
    qkv = draw(1, B, S, H + 2 * Hk, D)
    q, k, v = qkv.split([H, Hk, Hk], dim=2)
    dqkv = torch.full_like(qkv, 7.0)
    out = dqkv.split([H, Hk, Hk], dim=2)
    wide = torch.full((B, S, H, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
    _, _, dq, dk, dv = check_all(q, k, v, draw(2, B, S, H, D, std=1e-2), True, out=out,
                                 fwd_out=wide[..., :D])
    assert dq.data_ptr() == dqkv.data_ptr()
    assert torch.all(wide[..., D:] == 7.0)
    # [batch, head, row, dim] storage
    q2, k2, v2 = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (q, k, v))
    check_all(q2, k2, v2, draw(2, B, S, H, D, std=1e-2).transpose(1, 2).contiguous().transpose(1, 2),
              True)


def test_a_key_head_broadcast_over_the_batch():
    say("[attention] stride 0")
    q, do = draw(1, 3, 70, 2, 64), draw(2, 3, 70, 2, 64, std=1e-2)
    k = draw(3, 1, 90, 2, 64).expand(3, -1, -1, -1)
    v = draw(4, 1, 90, 1, 64).expand(3, -1, 2, -1)
    check_all(q, k, v, do, True)


def test_scale_and_another_stream():
    say("[attention] scale, stream")
    q, do = draw(1, 1, 100, 2, 64), draw(2, 1, 100, 2, 64, std=1e-2)
    k, v = draw(3, 1, 100, 2, 64), draw(4, 1, 100, 2, 64)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    a = check_all(q, k, v, do, True, scale=0.5, stream=st)
    with torch.cuda.stream(st):
        b = check_all(q, k, v, do, True, scale=0.5)
    for x, y in zip(a, b):   # and the same bits on every run
        assert torch.equal(x, y)


def test_shared_walks_are_the_same_on_every_run():
    say("[attention] shared walks, determinism")
    q, do = draw(1, 1, 1000, 4, 128), draw(2, 1, 1000, 4, 128)
    k, v = draw(3, 1, 1000, 1, 128), draw(4, 1, 1000, 1, 128)
    c = qn.train_ops._AttnCall(q, k, v, True, None, None, None).c
    assert qn.lib().qlora_attention_fwd_workspace_size(c) > 0
    assert qn.lib().qlora_attention_bwd_workspace_size(c) > 4000 * 4
    runs = []
    for _ in range(2):
        o, lse = qn.attention_fwd(q, k, v)
        runs.append((o, lse, *qn.attention_bwd(q, k, v, o, lse, do)))
    for a, b in zip(*runs):
        assert torch.equal(a, b)


@pytest.mark.parametrize("lq,lk,n", [(0, 5, 1), (5, 0, 2), (0, 0, 1), (4, 4, 0)])
def test_nothing_on_one_side(lq, lk, n):
    say(f"[attention] empty {lq} {lk} {n}")
    q, do = draw(1, n, lq, 2, 64), draw(2, n, lq, 2, 64)
    k, v = draw(3, n, lk, 1, 64), draw(4, n, lk, 1, 64)
    o, lse = qn.attention_fwd(q, k, v)
    dq, dk, dv = qn.attention_bwd(q, k, v, o, lse, do)
    torch.cuda.synchronize()
    assert not o.any() and torch.isneginf(lse).all()
    for t, like in ((dq, q), (dk, k), (dv, v)):
        assert t.shape == like.shape and not t.any()


def test_offsets_past_32_bits():
    """A row stride that puts the last heads' rows beyond 4 GB."""
    say("[attention] 64-bit offsets")
    S, D = 600, 64
    big = torch.zeros(S, 1 << 22, dtype=torch.bfloat16, device="cuda")   # 5 GB
    at = (1 << 22) - 4 * D
    big[:, at:] = draw(1, S, 4 * D)
    t = big[:, at:].unflatten(1, (4, D))
    q, k, v, do = (t[None, :, i:i + 1] for i in range(4))
    assert q.stride(1) == 1 << 22
    check_all(q, k, v, do, True)
    # and a batch stride that does the same
    x = big.view(-1).as_strided((2, 100, 1, D), (1 << 31, D, D, 1))
    x.copy_(draw(2, 2, 100, 1, D))
    check_all(x, x, x, x, False)


def test_autograd_gives_the_same_gradients():
    say("[attention] autograd")
    q, k, v = (draw(i, 2, 90, h, 64).requires_grad_() for i, h in ((1, 4), (2, 2), (3, 2)))
    do = draw(4, 2, 90, 4, 64, std=1e-2)
    o = qn.attention(q, k, v)
    o.backward(do)
    o2, lse = qn.attention_fwd(q.detach(), k.detach(), v.detach())
    grads = qn.attention_bwd(q.detach(), k.detach(), v.detach(), o2, lse, do)
    assert torch.equal(o, o2)
    for a, b in zip((q.grad, k.grad, v.grad), grads):
        assert torch.equal(a, b)
    # a gradient with strides of 0, as sum().backward() hands down
    q.grad = None
    qn.attention(q, k, v).sum().backward()
    ones = torch.ones_like(o2)
    assert torch.equal(q.grad, qn.attention_bwd(q.detach(), k.detach(), v.detach(), o2, lse, ones)[0])


def test_gradients_against_differences_of_the_forward():
    """The directional derivative of sum(O dO), by central differences of the
    fp64 forward, against the kernels' gradients.  The kernels' error in the
    inner product is a sum of independent roundings: at most 4 times the root of
    the direction-weighted variances (a probability below 1e-4), plus the
    difference's own 1e-6."""
    say("[attention] differences")
    q, k, v, do = draw(1, 1, 130, 2, 64), draw(2, 1, 130, 1, 64), draw(3, 1, 130, 1, 64), \
        draw(4, 1, 130, 2, 64)
    o, lse = qn.attention_fwd(q, k, v)
    grads = qn.attention_bwd(q, k, v, o, lse, do)
    torch.cuda.synchronize()
    x = [flat(t, False) for t in (q, k, v)]
    g = flat(do, False)
    seqs = oracle.sequences(130, 130)
    r = oracle.run(*x, seqs, 1 / 8, True, g)
    rng = np.random.default_rng(0)
    for i, name in enumerate(("dq", "dk", "dv")):
        d = rng.standard_normal(x[i].shape)
        h = 1e-4

        def loss(sign):
            y = list(x)
            y[i] = x[i] + sign * h * d
            return float((oracle.run(*y, seqs, 1 / 8, True).o * g).sum())

        diff = (loss(1) - loss(-1)) / (2 * h)
        got = float((flat(grads[i], False) * d).sum())
        sd = float(np.sqrt((r.budget[name][1] * d * d).sum()))
        say(f"    {name}: {got:.6f} against {diff:.6f}, sd {sd:.6f}")
        assert abs(got - diff) <= 4 * sd + 1e-4 * (1 + abs(diff))


def test_more_workgroups_than_one_launch_takes():
    """2^24 + 48 tiles, whose threads are more than one grid dimension takes
    (2^32): equal sequences far apart give equal results, and the oracle's."""
    say("[attention] 2^24 + 48 tiles")
    n, batch, H, D = 4099, (1 << 20) + 3, 16, 8
    q, do = draw(1, n, 1, H, D, std=1.5), draw(2, n, 1, H, D, std=1e-2)
    k, v = draw(3, n, 2, H, D), draw(4, n, 2, H, D)
    one = check_all(q, k, v, do, True)
    q, k, v, do = (t.repeat(batch // n + 1, 1, 1, 1)[:batch] for t in (q, k, v, do))
    o, lse = qn.attention_fwd(q, k, v)
    many = (o, lse, *qn.attention_bwd(q, k, v, o, lse, do))
    torch.cuda.synchronize()
    for name, a, b in zip(("o", "lse", "dq", "dk", "dv"), many, one):
        for at in range(0, batch, n):
            m = min(n, batch - at)
            assert torch.equal(a[at:at + m], b[:m]), f"{name}: sequence {at} and on"


# sequences, queries of a few / keys of many rows, heads, key/value heads, dim, causal.
# 64 and more sequences are found in another way than fewer, and so are 128 and more.
MANY = [(63, False, 4, 2, 64, True), (64, False, 4, 2, 64, True), (65, False, 2, 1, 128, True),
        (127, False, 1, 1, 64, True), (128, False, 1, 1, 64, True), (127, True, 2, 2, 64, True),
        (130, False, 2, 2, 64, False), (129, False, 1, 1, 80, True), (64, True, 1, 1, 128, False),
        (131, True, 2, 1, 64, True), (700, False, 1, 1, 8, True)]


@pytest.mark.parametrize("case", MANY, ids=lambda c: "-".join(map(str, c)))
def test_packed_with_many_sequences_of_every_length(case):
    """Empty sequences, single rows, whole tiles, one row more, several tiles,
    with other lengths on the side of the keys and a tail of several tiles."""
    n, few, H, Hk, D, causal = case
    say(f"[attention] {n} sequences {case}")
    rng = np.random.default_rng(n)
    some = [0, 1, 2, 31, 64, 127, 128, 129, 300, 700]
    lk = rng.choice(some, n, p=[0.15, 0.15, 0.15, 0.15, 0.1, 0.07, 0.07, 0.07, 0.05, 0.04])
    lk = 4 * lk if few else lk
    lq = rng.integers(0, 5, n) if few else rng.permutation(lk)
    lq[-1], lk[-1] = (3, 700) if few else (257, 300)   # the last one is not a trivial one
    cq, ck = (torch.tensor(np.cumsum([0, *x]), dtype=torch.int32, device="cuda") for x in (lq, lk))
    tail = 300
    q, do = draw(1, sum(lq) + tail, H, D, std=1.5), draw(2, sum(lq) + tail, H, D, std=1e-2)
    k, v = draw(3, sum(lk) + tail, Hk, D), draw(4, sum(lk) + tail, Hk, D)
    for t in (q, do, k, v):
        t[-tail:] = float("nan")
    if few:
        c = qn.train_ops._AttnCall(q, k, v, causal, None, cq, ck).c
        assert qn.lib().qlora_attention_fwd_workspace_size(c) > 0   # walks are shared here
    o, lse, dq, dk, dv = check_all(q, k, v, do, causal, cu=cq, cu_k=ck)
    assert torch.isneginf(lse[:, -tail:]).all()
    for t in (o, dq, dk, dv):
        assert not t[-tail:].any()


def guarded(rows, heads, dim, value, guard=float("nan"), ends=300):
    """(rows of `value`, the buffer they lie in: `ends` rows of `guard` before
    and after them)."""
    buf = torch.full((rows + 2 * ends, heads, dim), guard, dtype=torch.bfloat16, device="cuda")
    buf[ends:-ends] = value
    return buf[ends:-ends], buf


WRONG = {"past the end": [0, 400, 300], "negative": [-5, 100, 300], "descending": [0, 200, 100],
         "not from zero": [250, 20, 299], "extreme": [0, 1 << 30, -(1 << 30)],
         "limits": [-(1 << 31), (1 << 31) - 1],
         "saw": [0, 300] * 40, "many extremes": [0, (1 << 31) - 1, -(1 << 31)] * 50,
         "many descending": list(range(299, 0, -2)), "many past the end": list(range(0, 100000, 500))}


@pytest.mark.parametrize("heads,kv_heads,rows", [(2, 1, 300), (1, 1, 5000)])
@pytest.mark.parametrize("bad", WRONG, ids=lambda s: s.replace(" ", "-"))
def test_wrong_offsets_touch_nothing_outside_the_tensors(bad, heads, kv_heads, rows):
    """Rows around the inputs are NaN and never reach an output; rows around
    the outputs keep what they held.  (The workspace starts as zeros: rows that
    no sequence covers are joined from what it holds.)"""
    say(f"[attention] guard rows, {bad}, {rows} rows")
    D = 64
    ins = [guarded(rows, h, D, draw(i, rows, h, D, std=0.1))[0]
           for i, h in enumerate((heads, kv_heads, kv_heads, heads, heads))]
    q, k, v, o, do = ins
    outs = [guarded(rows, h, D, 5.0, 7.0) for h in (heads, heads, kv_heads, kv_heads)]
    cu = torch.tensor(WRONG[bad], dtype=torch.int32, device="cuda")
    good = torch.tensor(np.linspace(0, rows, len(cu)).astype(int), dtype=torch.int32, device="cuda")
    lse = torch.zeros(heads, rows, device="cuda")
    for cq, ck in ((cu, cu), (cu, good), (good, cu)):
        c = qn.train_ops._AttnCall(q, k, v, True, None, cq, ck).c
        ws = torch.zeros(max(qn.lib().qlora_attention_fwd_workspace_size(c),
                             qn.lib().qlora_attention_bwd_workspace_size(c)),
                         dtype=torch.uint8, device="cuda")
        qn.attention_fwd(q, k, v, cu_seqlens=cq, cu_seqlens_k=ck, out=outs[0][0], ws=ws)
        ws.zero_()
        qn.attention_bwd(q, k, v, o, lse, do, cu_seqlens=cq, cu_seqlens_k=ck, ws=ws,
                         out=tuple(t for t, _ in outs[1:]))
        torch.cuda.synchronize()
        for t, buf in outs:
            assert not torch.isnan(t).any()
            assert bool((buf[:300] == 7.0).all()) and bool((buf[-300:] == 7.0).all())


def test_the_search_for_a_sequence_does_not_grow_with_their_number():
    """2^16 packed sequences of one token against the same as a dense batch:
    as many workgroups with the same work and the search, a few dependent
    loads each (measured: 1.4 times the dense call's time; 83 times with a walk
    over all offsets in each workgroup)."""
    say("[attention] 2^16 sequences")
    n, H, D = 1 << 16, 2, 64
    q, k, v, do = (draw(i, n, H, D) for i in range(4))
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")

    def run(ts, cu):
        o, lse = qn.attention_fwd(*ts[:3], cu_seqlens=cu)
        return (o, lse, *qn.attention_bwd(*ts[:3], o, lse, ts[3], cu_seqlens=cu))

    def best(ts, cu):
        run(ts, cu)
        times = []
        for _ in range(3):
            a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
            a.record()
            out = run(ts, cu)
            b.record()
            b.synchronize()
            times.append(a.elapsed_time(b))
        return min(times), out
    dense, ref = best([t[:, None] for t in (q, k, v, do)], None)
    packed, got = best([q, k, v, do], cu)
    say(f"    dense {dense:.2f} ms, packed {packed:.2f} ms")
    assert torch.equal(got[1], ref[1][:, :, 0].T)
    for a, b in zip((got[0], *got[2:]), (ref[0], *ref[2:])):
        assert torch.equal(a, b[:, 0])
    assert packed < 8 * dense


def test_outputs_over_inputs():
    """Over an input that is read again, over each other and with rows on top
    of each other they are refused; where each row is read before it is
    written they give the same bits."""
    say("[attention] outputs over inputs")
    for S, H, Hk in ((200, 4, 4), (1500, 2, 2)):   # whole and shared walks
        q, k, v, do = (draw(i, 1, S, h, 64) for i, h in ((1, H), (2, Hk), (3, Hk), (4, H)))
        o, lse = qn.attention_fwd(q, k, v)
        grads = qn.attention_bwd(q, k, v, o, lse, do)
        for bad in (k, v):
            with pytest.raises(qn.QloraError, match="invalid"):
                qn.attention_fwd(q, k, v, out=bad)
        new = [torch.empty_like(t) for t in (q, k, v)]
        for at, bad in ((0, q), (0, do), (0, k), (0, v), (1, q), (1, do), (1, o), (1, v), (2, k),
                        (2, q), (1, new[2]), (1, new[0]), (2, new[0])):
            out = list(new)
            out[at] = bad
            with pytest.raises(qn.QloraError, match="invalid"):
                qn.attention_bwd(q, k, v, o, lse, do, out=tuple(out))
        for at in range(3):
            flat = torch.empty_like(new[at][:, :1]).expand_as(new[at])
            out = list(new)
            out[at] = flat
            with pytest.raises(qn.QloraError, match="invalid"):
                qn.attention_bwd(q, k, v, o, lse, do, out=tuple(out))
        with pytest.raises(qn.QloraError, match="invalid"):
            qn.attention_fwd(q, k, v, out=new[0][:, :, :1].expand_as(q))
        buf = q.clone()
        o2, lse2 = qn.attention_fwd(buf, k, v, out=buf)
        assert o2 is buf and torch.equal(buf, o) and torch.equal(lse2, lse)
        o2, k2, v2 = o.clone(), k.clone(), v.clone()
        for a, b in zip(qn.attention_bwd(q, k2, v2, o2, lse, do, out=(o2, k2, v2)), grads):
            assert torch.equal(a, b)


@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -60, 2.0 ** 60, 2.0 ** 100], ids=str)
def test_extreme_scales(scale):
    """Tiny: every visible key counts alike.  Huge, with queries as small: the
    scores are those of ordinary inputs."""
    say(f"[attention] scale {scale}")
    q, do = draw(1, 1, 150, 2, 64, std=0.2), draw(2, 1, 150, 2, 64, std=1e-2)
    k, v = draw(3, 1, 150, 2, 64), draw(4, 1, 150, 2, 64)
    if scale > 1:
        q = q * (1 / scale)
    check_all(q, k, v, do, True, scale=scale)
