"""Layer norm and root-mean-square norm on the GPU against the fp64 oracle.

Tolerances: sums of a row are at most 64 terms in a thread and 11 levels of a
tree, so a row's mean is within 80 * 2^-24 of mean |x|, and with the handful
of further fp32 operations z = (x - mean) rstd is within
Ez = 200 * 2^-24 (|x| + mean |x|) rstd; the outputs follow from that, their own
fp32 terms (400 * 2^-24 of the terms' magnitudes; sums over rows 2^-24 (400 +
rows / 64)), and one rounding of at most 2^-8 where an output is bf16.
"""

import numpy as np
import pytest
import torch

import quantized_base_lora_nf4_amd as qn
from oracle import norms
from gpu_util import say

pytestmark = pytest.mark.gpu

E = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: E}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    qn.lib()


def draw(seed, *shape, std=1.0, mean=0.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype).cuda()


def host(t):
    return t.detach().double().cpu().numpy()


def within(name, got, ref, tol):
    got = host(got)
    assert got.shape == ref.shape
    assert np.all(np.isfinite(got)), f"{name}: non-finite output"
    worst = float((np.abs(got - ref) / (tol + 1e-37)).max(initial=0.0))
    say(f"    {name}: {worst:.3f} of its bound")
    assert worst <= 1.0, f"{name}: {worst:.3g} times its bound"


def check(x, w, b, dy, eps, rms):
    y, mean, rstd = qn.norm_fwd(x, w, b, eps=eps, rms=rms)
    dx, dw, db = qn.norm_bwd(dy, x, w, mean, rstd, rms=rms, need_db=True)
    torch.cuda.synchronize()
    assert y.dtype == x.dtype and dx.dtype == x.dtype and dw.dtype == w.dtype == db.dtype
    X, W, D = host(x), host(w), host(dy)
    B = None if b is None else host(b)
    ry, rmean, rrstd = norms.norm_forward(X, W, B, eps, rms)
    rdx, rdw, rdb = norms.norm_backward(D, X, W, eps, rms)
    ax = np.abs(X).mean(1, keepdims=True)
    rs = rrstd[:, None]
    ez = 200 * E * (np.abs(X) + ax) * rs
    if not rms:
        within("mean", mean, rmean, 80 * E * ax[:, 0])
    else:
        assert mean is None
    # relative: (x - mean)^2 moves by 2 |x - mean| times the mean's error at most
    c = np.abs(X - rmean[:, None])
    within("rstd", rstd, rrstd,
           rrstd * (100 * E + (80 * E * ax * 2 * c).mean(1) * rrstd ** 2))
    ux, uw = U[x.dtype], U[w.dtype]
    within("y", y, ry, ez * np.abs(W) + 4 * E * (0 if B is None else np.abs(B)) + ux * np.abs(ry))
    z, g = (X - rmean[:, None]) * rs, D * W
    gz = np.abs(g * z).mean(1, keepdims=True)
    t = 400 * E * rs * (np.abs(g) + np.abs(z) * gz + np.abs(g).mean(1, keepdims=True))
    t = t + rs * (ez * gz + np.abs(z) * (np.abs(g) * ez).mean(1, keepdims=True))
    within("dx", dx, rdx, t + ux * np.abs(rdx))
    n = E * (400 + len(X) / 64)
    within("dw", dw, rdw, (np.abs(D) * ez).sum(0) + n * np.abs(D * z).sum(0) + uw * np.abs(rdw))
    within("db", db, rdb, n * np.abs(D).sum(0) + uw * np.abs(rdb))


SIZES = [(1, 1), (3, 2), (1, 7), (5, 8), (2, 33), (64, 64), (7, 100), (3, 255), (4, 512), (6, 513),
         (1, 1000), (2, 1027), (9, 2048), (3, 4097), (2, 5120), (1, 8192), (2049, 130),
         (2050, 1023), (2100, 2100), (700, 4096), (5000, 24), (2, 16384), (1100, 520)]


@pytest.mark.parametrize("xt,wt", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                   (torch.bfloat16, torch.float32),
                                   (torch.float32, torch.bfloat16)], ids=str)
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("rows,width", SIZES)
def test_norm(rows, width, rms, xt, wt):
    say(f"[norm] {rows}x{width} rms={rms} {xt} {wt}")
    x = draw(1, rows, width, std=2.0, mean=0.25, dtype=xt)
    w, b = draw(2, width, std=0.2, mean=1.0, dtype=wt), draw(3, width, dtype=wt)
    check(x, w, b if rows % 2 else None, draw(4, rows, width, std=1e-2, dtype=xt), 1e-5, rms)


@pytest.mark.parametrize("xt,width", [(torch.bfloat16, 65536), (torch.bfloat16, 65535),
                                      (torch.float32, 32768), (torch.bfloat16, 40000),
                                      (torch.float32, 20001)])
def test_the_widest_rows(xt, width):
    say(f"[norm] widest {width} {xt}")
    check(draw(1, 3, width, dtype=xt), draw(2, width), draw(3, width), draw(4, 3, width, dtype=xt),
          1e-5, False)


def test_rows_far_from_zero_and_constant_rows():
    say("[norm] offset, constant")
    x = draw(1, 8, 1000, mean=300.0)
    x[3] = 5.0
    x[4] = 0.0
    check(x, draw(2, 1000), draw(3, 1000), draw(4, 8, 1000), 1e-5, False)
    check(x, draw(2, 1000), None, draw(4, 8, 1000), 1e-5, True)


def test_views_at_odd_addresses():
    """Rows of a slice: element-aligned pointers."""
    say("[norm] odd addresses")
    for dt in (torch.bfloat16, torch.float32):
        x, dy = draw(1, 12, 129, dtype=dt)[1:], draw(2, 12, 129, dtype=dt)[1:]
        w, b = draw(3, 132, dtype=dt)[3:], draw(4, 130, dtype=dt)[1:]
        assert x.data_ptr() % 16 and w.data_ptr() % 16
        check(x, w, b, dy, 1e-5, False)


def test_more_than_2_to_31_elements():
    """The last rows of a matrix of 2.3e9 elements, with the first ones' stale
    neighbours far away, are those of the same rows alone."""
    say("[norm] 64-bit offsets")
    rows, width = 70000, 32768
    x = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    dy = torch.zeros_like(x)
    x[-3:], dy[-3:] = draw(1, 3, width, dtype=x.dtype), draw(2, 3, width, dtype=x.dtype)
    w = draw(3, width)
    y, mean, rstd = qn.norm_fwd(x, w)
    dx, dw, db = qn.norm_bwd(dy, x, w, mean, rstd)
    y3, mean3, rstd3 = qn.norm_fwd(x[-3:], w)
    dx3, dw3, db3 = qn.norm_bwd(dy[-3:], x[-3:], w, mean3, rstd3)
    torch.cuda.synchronize()
    # other launch shapes for few and many rows: the sums' order differs, so
    # fp32 statistics agree to 80 * 2^-24 and bf16 results to one rounding
    assert torch.allclose(rstd[-3:], rstd3, rtol=1e-5) and torch.allclose(mean[-3:], mean3, atol=1e-5)
    assert not y[:100].any() and not dx[:100].any()
    for a, b in ((y[-3:], y3), (dx[-3:], dx3)):
        assert torch.allclose(a.float(), b.float(), rtol=2.0 ** -7, atol=1e-5)
    # rows of zeros add nothing to the parameters' gradients
    for a, b in ((dw, dw3), (db, db3)):
        assert torch.allclose(a, b, rtol=1e-4, atol=1e-4)


def test_no_rows():
    say("[norm] no rows")
    x = torch.zeros(0, 40, device="cuda")
    w, b = draw(1, 40), draw(2, 40)
    y, mean, rstd = qn.norm_fwd(x, w, b)
    dx, dw, db = qn.norm_bwd(x, x, w, mean, rstd)
    torch.cuda.synchronize()
    assert y.shape == x.shape and mean.shape == rstd.shape == (0,) and dx.shape == x.shape
    assert not dw.any() and not db.any()


def test_a_nan_stays_in_its_row():
    say("[norm] NaN")
    x = draw(1, 6, 200)
    x[2, 5] = float("nan")
    w, b, dy = draw(2, 200), draw(3, 200), draw(4, 6, 200)
    y, mean, rstd = qn.norm_fwd(x, w, b)
    dx, _, _ = qn.norm_bwd(dy, x, w, mean, rstd)
    torch.cuda.synchronize()
    keep = [0, 1, 3, 4, 5]
    assert torch.isnan(y[2]).all() and torch.isfinite(y[keep]).all()
    assert torch.isnan(dx[2]).all() and torch.isfinite(dx[keep]).all()


def test_parts_alone_and_the_same_bits_on_every_run():
    say("[norm] parts")
    x, w, b, dy = draw(1, 300, 500), draw(2, 500), draw(3, 500), draw(4, 300, 500)
    _, mean, rstd = qn.norm_fwd(x, w, b)
    full = qn.norm_bwd(dy, x, w, mean, rstd)
    for need in ((True, False, False), (False, True, False), (False, False, True),
                 (False, False, False), (True, True, True)):
        part = qn.norm_bwd(dy, x, w, mean, rstd, need_dx=need[0], need_dw=need[1], need_db=need[2])
        for n, p, f in zip(need, part, full):
            assert (p is None) if not n else torch.equal(p, f)


@pytest.mark.parametrize("rms", [False, True])
def test_modules_and_autograd(rms):
    say("[norm] modules")
    m = (qn.RMSNorm if rms else qn.LayerNorm)(96, dtype=torch.bfloat16)
    with torch.no_grad():
        m.weight.copy_(draw(1, 96))
        if not rms:
            m.bias.copy_(draw(2, 96))
    x = draw(3, 4, 5, 96, dtype=torch.bfloat16).requires_grad_()
    dy = draw(4, 4, 5, 96, dtype=torch.bfloat16)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        y = m(x)
        y.backward(dy)
    st.synchronize()
    bias = None if rms else m.bias.detach()
    y2, mean, rstd = qn.norm_fwd(x.detach(), m.weight.detach(), bias, m.eps, rms)
    dx, dw, db = qn.norm_bwd(dy, x.detach(), m.weight.detach(), mean, rstd, rms)
    assert torch.equal(y, y2) and torch.equal(x.grad, dx) and torch.equal(m.weight.grad, dw)
    if not rms:
        assert torch.equal(m.bias.grad, db)


@pytest.mark.parametrize("rms", [False, True])
def test_gradients_against_differences_of_the_forward(rms):
    """Central differences (h = 1e-4) of the fp64 forward; fp32 gradients, so
    what remains is the differences' own h^2 and fp32 rounding: 1e-5."""
    say("[norm] differences")
    x, w, dy = draw(1, 7, 60), draw(2, 60), draw(3, 7, 60)
    _, mean, rstd = qn.norm_fwd(x, w, None, rms=rms)
    dx, dw, _ = qn.norm_bwd(dy, x, w, mean, rstd, rms=rms)
    X, W, D = host(x), host(w), host(dy)
    rng = np.random.default_rng(0)
    for got, at, f in (
            (dx, X, lambda t: (norms.norm_forward(t, W, None, 1e-5, rms)[0] * D).sum()),
            (dw, W, lambda t: (norms.norm_forward(X, t, None, 1e-5, rms)[0] * D).sum())):
        d = rng.standard_normal(at.shape)
        diff = (f(at + 1e-4 * d) - f(at - 1e-4 * d)) / 2e-4
        assert abs((host(got) * d).sum() - diff) <= 1e-5 * (1 + (np.abs(host(got) * d)).sum())


# Rows whose forward launch would have more threads than one grid dimension takes (2^32: four rows
# per 256 threads), and rows just past one launch's workgroups in the other shapes.
@pytest.mark.parametrize("rows,width,dtype", [((1 << 26) + 5, 8, torch.bfloat16),
                                              ((1 << 20) + 3, 2056, torch.bfloat16),
                                              ((1 << 20) + 3, 1032, torch.float32)], ids=str)
@pytest.mark.parametrize("rms", [False, True])
def test_more_rows_than_one_launch_takes(rows, width, dtype, rms):
    """Equal rows far apart give equal results, and those of the oracle."""
    say(f"[norm] {rows} rows of {width} rms={rms}")
    n = 2053
    few = draw(1, n, width, std=2.0, mean=0.25, dtype=dtype)
    w, b = draw(2, width, std=0.2, mean=1.0), draw(3, width)
    x = few.repeat((rows + n - 1) // n, 1)[:rows]
    y, mean, rstd = qn.norm_fwd(x, w, b, rms=rms)
    y1, mean1, rstd1 = qn.norm_fwd(few, w, b, rms=rms)   # 2053 rows: the same shape of launch
    check(few, w, b, few, 1e-5, rms)
    torch.cuda.synchronize()
    for at in range(0, rows, n * 500):
        k = min(n, rows - at)
        assert torch.equal(y[at:at + k], y1[:k]) and torch.equal(rstd[at:at + k], rstd1[:k])
    at = (rows - 1) // n * n
    for a, b1 in ((y, y1), (rstd, rstd1), *(() if rms else ((mean, mean1),))):
        assert torch.equal(a[at:], b1[:rows - at])
        edge = (1 << 20) // n * n   # where a launch of one row per workgroup ends
        assert torch.equal(a[edge:edge + n], b1[:min(n, rows - edge)])


def test_frozen_parameters_take_no_workspace():
    """dx alone: nothing but dx is allocated (the partial sums of dw and db
    would take 16 MB here)."""
    say("[norm] dx alone")
    x, w = draw(1, 2048, 8192, dtype=torch.bfloat16), draw(2, 8192)
    _, mean, rstd = qn.norm_fwd(x, w)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    dx, dw, db = qn.norm_bwd(x, x, w, mean, rstd, need_dw=False, need_db=False)
    torch.cuda.synchronize()
    assert dw is None and db is None
    assert torch.cuda.max_memory_allocated() - before <= dx.numel() * 2 + (1 << 20)
    assert torch.equal(dx, qn.norm_bwd(x, x, w, mean, rstd)[0])
