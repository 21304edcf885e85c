"""Rows of many adapters over one NF4 weight, against fp64 products with the
weight's bf16 values.

Tolerance per output, with u = 2^-8 (half a bf16 step): Y is rounded once
(u |Y|).  Up to 16 rows the weight enters as level times constant, levels
rounded to bf16 (u) instead of the product (u): 2 u of sum |x w| at most, and
independent from weight to weight, so 8 deviations of u sqrt(sum (x w)^2).  Other rows round
s U once (u of sum |s u b| at most, independent over the rank likewise).  Which
of the two a batch meets is the kernels' choice: both are counted.
Sums are fp32: 2^-24 per addition, K + r of them at most, of sum |x w| + ...;
both are far below the budget: 2^-16 of the sum of magnitudes is added.
"""

import numpy as np
import pytest
import torch

import quantized_base_lora_nf4_amd as qn
from gpu_util import say

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U = 2.0 ** -8


def make(N, K, n, r, code="nf4", blocksize=64, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = torch.randn(N, K, generator=g, device="cuda") * K ** -0.5
    levels = None
    if code == "user4":
        levels = np.linspace(-1, 1, 16)
    w = qn.nf4_quantize(W, code=code, blocksize=blocksize, levels=levels)
    A = (torch.randn(n, r, K, generator=g, device="cuda") * K ** -0.5).to(BF)
    B = (torch.randn(n, N, r, generator=g, device="cuda") * 0.5).to(BF)
    s = torch.rand(n, generator=g, device="cuda") * 4 - 1
    return w, A, B, s


def rows(M, K, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(M, K, generator=g, device="cuda").to(BF)


def check(name, Y, w, X, A, B, s, index):
    W = qn.nf4_dequantize(w).double()
    x = X.double()
    ref = x @ W.T
    size = x.abs() @ W.abs().T
    var = (x * x) @ (W * W).T * U * U
    idx = index.cpu()
    for a in set(idx.tolist()):
        if not 0 <= a < len(A):
            continue
        m = (idx == a).nonzero().flatten().cuda()
        u = x[m] @ A[a].double().T * float(s[a])
        b = B[a].double()
        ref[m] += u @ b.T
        size[m] += u.abs() @ b.abs().T
        var[m] += (u * u) @ (b * b).T * U * U
    tol = U * ref.abs() * (1 + U) + 8 * var.sqrt() + 2.0 ** -16 * size
    err = (Y.double() - ref).abs()
    say(f"    {name}: {float((err / tol).max()):.3f} of the bound, {float(err.norm() / ref.norm()):.2e} of the norm")
    assert (err <= tol).all(), name
    # what bf16 roundings leave of the whole: three at most, rms u / sqrt(3) each
    assert float(err.norm() / ref.norm()) <= U


def spread(M, n, how, seed=0):
    g = torch.Generator().manual_seed(seed)
    if how == "each":
        i = torch.arange(M) % n
    elif how == "runs":
        i = torch.sort(torch.randint(0, n, (M,), generator=g)).values
    elif how == "random":
        i = torch.randint(-1, n, (M,), generator=g)
    elif how == "one":
        i = torch.full((M,), n - 1)
    else:
        i = torch.full((M,), -1)
    return i.to(torch.int32).cuda()


@pytest.mark.parametrize("how", ["each", "runs", "random", "one", "none"])
@pytest.mark.parametrize("M", [1, 2, 7, 16, 17, 32, 33, 64, 65, 129, 300, 4097, 8300])
def test_rows_and_orders(M, how):
    say(f"[multi] {M} rows, {how}")
    w, A, B, s = make(264, 320, 9, 16)
    X, index = rows(M, 320), spread(M, 9, how)
    check("Y", qn.qlora_linear_multi_fwd(w, X, A, B, s, index), w, X, A, B, s, index)


@pytest.mark.parametrize("M", [3, 40, 4100])
@pytest.mark.parametrize("r", [1, 4, 8, 9, 16, 24, 33, 64, 100, 128, 256])
def test_ranks(M, r):
    say(f"[multi] {M} rows, rank {r}")
    w, A, B, s = make(136, 256, 5, r)
    X, index = rows(M, 256), spread(M, 5, "random")
    check("Y", qn.qlora_linear_multi_fwd(w, X, A, B, s, index), w, X, A, B, s, index)


@pytest.mark.parametrize("M", [1, 5, 16, 50, 700])
@pytest.mark.parametrize("N,K", [(8, 64), (16, 64), (1024, 64), (8, 2048), (520, 1088), (2048, 512), (28672, 512)])
def test_sizes(M, N, K):
    say(f"[multi] {M} rows, {N} x {K}")
    w, A, B, s = make(N, K, 3, 8)
    X, index = rows(M, K), spread(M, 3, "random")
    check("Y", qn.qlora_linear_multi_fwd(w, X, A, B, s, index), w, X, A, B, s, index)


@pytest.mark.parametrize("M", [5, 40, 100, 4100])
@pytest.mark.parametrize("r", [3, 9, 13, 23, 47, 95])
def test_rows_end_inside_a_piece(M, r):
    """Ranks that are no multiple of 8: what follows a row of B, in the same
    adapter or in the next, reaches no output of the row."""
    w, A, B, s = make(136, 128, 3, r)
    X, index = rows(M, 128), torch.zeros(M, dtype=torch.int32, device="cuda")
    bad = B.clone()
    bad[0, 1::2] = float("nan")
    bad[1:] = float("inf")
    Y, Z = (qn.qlora_linear_multi_fwd(w, X, A, b, s, index) for b in (B, bad))
    check(f"rank {r}", Y, w, X, A, B, s, index)
    assert torch.equal(Y[:, ::2], Z[:, ::2]) and Z[:, 1::2].isnan().all()


@pytest.mark.parametrize("M", [20, 70])
@pytest.mark.parametrize("r,K", [(8, 64), (33, 576), (64, 1024), (100, 192), (128, 448)])
@pytest.mark.parametrize("code", ["nf4", "nf3", "nf2"])
def test_wide_weights(M, r, K, code):
    """So many weight rows that workgroups take 64 of them, the last ones fewer."""
    say(f"[multi] {M} rows, 16392 x {K}, rank {r}, {code}")
    w, A, B, s = make(16392, K, 5, r, code)
    X, index = rows(M, K), spread(M, 5, "random")
    check("Y", qn.qlora_linear_multi_fwd(w, X, A, B, s, index), w, X, A, B, s, index)


@pytest.mark.parametrize("M", [4, 30, 100, 4100])
@pytest.mark.parametrize("code,blocksize", [("nf4", 128), ("nf4", 256), ("fp4", 64), ("nf3", 64), ("nf2", 128), ("user4", 64)])
def test_code_types(M, code, blocksize):
    say(f"[multi] {code}, blocks of {blocksize}")
    w, A, B, s = make(144, 512, 4, 16, code, blocksize)
    X, index = rows(M, 512), spread(M, 4, "random")
    Y = qn.qlora_linear_multi_fwd(w, X, A, B, s, index)
    check("Y", Y, w, X, A, B, s, index)


@pytest.mark.parametrize("M", [16, 64, 300, 4100])
def test_many_adapters(M):
    """More adapters than rows, and as many adapters as rows."""
    for n in (5000, M):
        w, A, B, s = make(72, 128, n, 16)
        X = rows(M, 128)
        index = torch.randperm(n, generator=torch.Generator().manual_seed(3))[:M].to(torch.int32).cuda()
        check(f"{n}", qn.qlora_linear_multi_fwd(w, X, A, B, s, index), w, X, A, B, s, index)


def test_wide_rows_are_taken_as_they_come():
    """Rows so wide that a window of them is past 32-bit offsets: no order."""
    K = 1 << 18
    w, A, B, s = make(8, K, 3, 8)
    X, index = rows(5000, K), spread(5000, 3, "random")
    Y = qn.qlora_linear_multi_fwd(w, X, A, B, s, index)
    some = torch.randperm(5000, generator=torch.Generator().manual_seed(1))[:200].cuda()
    check("200 rows", Y[some], w, X[some].contiguous(), A, B, s, index[some])


def test_large_few_token_rows():
    """K whose tables leave LDS: 16 rows take the tile path."""
    w, A, B, s = make(64, 64 * 520, 3, 256)
    X, index = rows(16, 64 * 520), spread(16, 3, "random")
    check("Y", qn.qlora_linear_multi_fwd(w, X, A, B, s, index), w, X, A, B, s, index)


@pytest.mark.parametrize("M", [1, 16, 17, 4100])
def test_one_adapter_is_the_layer(M):
    """All rows of one adapter: the layer's own forward within the roundings of
    U (it rounds U and s U, this s U or nothing)."""
    w, A, B, s = make(520, 512, 4, 16)
    X = rows(M, 512)
    Y = qn.qlora_linear_multi_fwd(w, X, A, B, s, spread(M, 4, "one"))
    Z = qn.qlora_linear_fwd(w, X, A[3].contiguous(), B[3].contiguous(), float(s[3]))
    assert float((Y.double() - Z.double()).norm() / Z.double().norm()) <= U
    none = qn.qlora_linear_multi_fwd(w, X, A, B, s, spread(M, 4, "none"))
    base = qn.qlora_linear_fwd(w, X, torch.zeros_like(A[0]), torch.zeros_like(B[0]), 1.0)
    # without an adapter both are X W^T: the same tiles for many rows, else the
    # weight enters as level times constant, with levels rounded in other places
    if M <= 17:
        assert float((none.double() - base.double()).norm() / base.double().norm()) <= U
    else:
        assert torch.equal(none, base)


@pytest.mark.parametrize("M", [5, 16, 20, 70, 4100])
def test_rows_do_not_see_other_adapters(M):
    """NaN and infinities in other rows and other adapters, in adapter 0 and in
    unused ones, change nothing."""
    w, A, B, s = make(136, 256, 6, 16)
    X = rows(M, 256)
    index = (torch.arange(M) % 3 * 2 - 1).to(torch.int32).cuda()     # -1, 1, 3
    Y = qn.qlora_linear_multi_fwd(w, X, A, B, s, index)
    for a in (0, 2, 4, 5):
        A[a], B[a], s[a] = float("nan"), float("inf"), float("nan")
    assert torch.equal(qn.qlora_linear_multi_fwd(w, X, A, B, s, index), Y)
    A[3], B[3] = float("inf"), float("nan")
    Z = qn.qlora_linear_multi_fwd(w, X, A, B, s, index)
    hit = index == 3
    assert torch.equal(Z[~hit], Y[~hit]) and Z[hit].isnan().all()
    X2 = X.clone()
    X2[0] = float("nan")
    Z = qn.qlora_linear_multi_fwd(w, X2, A, B, s, index)
    ok = ~hit
    ok[0] = False
    assert torch.equal(Z[ok], Y[ok]) and Z[0].isnan().all()


def test_wrong_indices_are_no_adapter():
    w, A, B, s = make(64, 128, 3, 8)
    for M in (9, 40, 4500):
        X = rows(M, 128)
        index = torch.tensor([0, 3, -1, 2 ** 31 - 1, -2 ** 31, 1, 2, 1000, -7] * 500, dtype=torch.int32)[:M].cuda()
        Y = qn.qlora_linear_multi_fwd(w, X, A, B, s, index)
        check("Y", Y, w, X, A, B, s, index)


@pytest.mark.parametrize("M", [6, 20, 200, 4100])
def test_order_of_rows(M):
    """A row's result does not depend on where it stands or on its neighbours."""
    w, A, B, s = make(136, 256, 6, 24)
    X, index = rows(M, 256), spread(M, 6, "random")
    Y = qn.qlora_linear_multi_fwd(w, X, A, B, s, index)
    # (windows of 4096 rows are put in order one by one: across them, sums stay
    # in their places too)
    p = torch.randperm(M, generator=torch.Generator().manual_seed(1)).cuda()
    assert torch.equal(qn.qlora_linear_multi_fwd(w, X[p].contiguous(), A, B, s, index[p].contiguous()), Y[p])
    assert torch.equal(qn.qlora_linear_multi_fwd(w, X, A, B, s, index), Y)


def test_pool_past_32_bits():
    """Adapters that start more than 2^32 bytes into the pool."""
    say("[multi] a pool of over 2^32 bytes")
    n, N, K, r = 2100, 8192, 8192, 128
    w, _, _, _ = make(N, K, 1, 8)
    A = torch.zeros(n, r, K, dtype=BF, device="cuda")
    B = torch.zeros(n, N, r, dtype=BF, device="cuda")
    s = torch.ones(n, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(0)
    for a in (0, n - 1):
        A[a] = (torch.randn(r, K, generator=g, device="cuda") * K ** -0.5).to(BF)
        B[a] = torch.randn(N, r, generator=g, device="cuda").to(BF)
    for M in (5, 60, 700):
        X = rows(M, K)
        index = torch.where(torch.arange(M) % 2 == 0, n - 1, 0).to(torch.int32).cuda()
        check(f"{M}", qn.qlora_linear_multi_fwd(w, X, A, B, s, index), w, X, A, B, s, index)


@pytest.mark.parametrize("M", [8, 90, 4100])
def test_captured_with_new_adapters(M):
    w, A, B, s = make(136, 256, 6, 16)
    X, index = rows(M, 256), spread(M, 6, "random")
    qn.qlora_linear_multi_fwd(w, X, A, B, s, index)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        Y = qn.qlora_linear_multi_fwd(w, X, A, B, s, index)
    for i in range(4):
        X.copy_(rows(M, 256, seed=10 + i))
        index.copy_(spread(M, 6, ("random", "none", "one", "runs")[i], seed=i))
        A[i] *= 2
        Z = qn.qlora_linear_multi_fwd(w, X, A, B, s, index)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(Y, Z)


def test_other_stream_workspace_and_output():
    w, A, B, s = make(136, 256, 6, 16)
    for M in (8, 90, 4100):
        X, index = rows(M, 256), spread(M, 6, "random")
        Y = qn.qlora_linear_multi_fwd(w, X, A, B, s, index)
        torch.cuda.synchronize()
        st = torch.cuda.Stream()
        out = torch.full((M + 2, 136), 5.0, dtype=BF, device="cuda")
        need = qn.multi_workspace_size(M, 136, 256, 16)
        ws = torch.full((need + 256,), 77, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        Z = qn.qlora_linear_multi_fwd(w, X, A, B, s, index, Y=out[1:M + 1], ws=ws[:need], stream=st)
        st.synchronize()
        assert torch.equal(Y, Z) and (out[0] == 5).all() and (out[-1] == 5).all()
        assert (ws[need:] == 77).all()


def test_module():
    """Adapters of different rank and scale in slots, against their layers."""
    g = torch.Generator(device="cuda").manual_seed(0)
    W = torch.randn(264, 256, generator=g, device="cuda") * 0.06
    layers = [qn.QLoRALinear(W, r, 2.0 * r + 1) for r in (4, 16, 12)]
    for l in layers:
        with torch.no_grad():
            l.B.copy_(torch.randn(l.B.shape, generator=g, device="cuda") * 0.3)
    many = qn.QLoRAMultiLinear(layers[0], slots=5, r=16)
    assert many.nf4 is layers[0].nf4 and not list(many.parameters())
    for i, l in enumerate(layers):
        many.load(i + 1, l)
    X = rows(4 * 30, 256).view(4, 30, 256)
    index = torch.tensor([1, 2, 3, -1], dtype=torch.int32, device="cuda")[:, None].expand(4, 30)
    Y = many(X, index)
    assert Y.shape == (4, 30, 264)
    with torch.no_grad():
        for i, l in enumerate(layers):
            Z = l(X[i])
            assert float((Y[i].double() - Z.double()).norm() / Z.double().norm()) <= U
    many.load(1, layers[2])   # a slot is taken again, by a smaller rank
    many.load(3, layers[0])
    assert torch.equal(many(X[2], index[2]), many(X[2], torch.full((30,), 3, dtype=torch.int32, device="cuda")))
    Z = layers[0](X[2])
    assert float((many(X[2], index[2]).double() - Z.double()).norm() / Z.double().norm()) <= U
    with pytest.raises(ValueError, match="slot"):
        many.load(5, layers[0])
    with pytest.raises(ValueError, match="do not fit"):
        many.put(0, torch.zeros(17, 256), torch.zeros(264, 17), 1.0)
    with pytest.raises(ValueError, match="do not fit"):
        many.put(0, torch.zeros(8, 256), torch.zeros(264, 4), 1.0)


@pytest.mark.parametrize("change,error,match", [
    (dict(X=lambda t: t[0]), ValueError, "X must be 2-D"),
    (dict(A=lambda t: t[0]), ValueError, "A must be 3-D"),
    (dict(B=lambda t: t[:2]), ValueError, "B has shape"),
    (dict(B=lambda t: t[:, :64]), ValueError, "B has shape"),
    (dict(A=lambda t: t.float()), TypeError, "A has dtype"),
    (dict(s=lambda t: t[:2]), ValueError, "s has shape"),
    (dict(s=lambda t: t.double()), TypeError, "s has dtype"),
    (dict(index=lambda t: t[:4]), ValueError, "index has shape"),
    (dict(index=lambda t: t.long()), TypeError, "index has dtype"),
    (dict(index=lambda t: t.cpu()), ValueError, "index is on cpu"),
    (dict(X=lambda t: t.cpu()), ValueError, "X is on cpu"),
    (dict(X=lambda t: torch.cat([t, t], 1)[:, :128]), ValueError, "contiguous"),
    (dict(X=lambda t: t[:0], index=lambda t: t[:0]), qn.QloraError, "invalid"),
    (dict(A=lambda t: t[:0], B=lambda t: t[:0], s=lambda t: t[:0]), qn.QloraError, "invalid"),
])
def test_refusals(change, error, match):
    w, A, B, s = make(72, 128, 3, 8)
    a = dict(X=rows(5, 128), A=A, B=B, s=s, index=spread(5, 3, "each"))
    for k, f in change.items():
        a[k] = f(a[k])
    with pytest.raises(error, match=match):
        qn.qlora_linear_multi_fwd(w, a["X"], a["A"], a["B"], a["s"], a["index"])


def test_refused_rank():
    w, A, B, s = make(72, 128, 1, 264)
    with pytest.raises(qn.QloraError, match="invalid"):
        qn.qlora_linear_multi_fwd(w, rows(5, 128), A, B, s, spread(5, 1, "each"))
