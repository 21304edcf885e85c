"""The global gradient norm and clipping on the GPU against the fp64 oracle.

Tolerances: squares add up in fp64 and the norm is rounded once, 2^-23 of it;
a scaled gradient has the factor's rounding and its own: 2^-22 in fp32 and
2^-8 in bf16.
"""

import numpy as np
import pytest
import torch

import quantized_base_lora_nf4_amd as qn
from oracle import norms
from gpu_util import say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    qn.lib()


def draw(seed, *shape, std=1.0, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std).to(dtype).cuda()


def host(t):
    return t.detach().double().cpu().numpy()


def check_scaled(got, ref, dtype):
    tol = 2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -22
    assert np.all(np.abs(host(got) - ref) <= tol * np.abs(ref) + 1e-40)


def check(grads, max_norm):
    """Norm alone, into new tensors, and in place."""
    ref_norm, ref = norms.clip([host(g) for g in grads], max_norm)
    before = [g.clone() for g in grads]
    n = qn.grad_norm(grads)
    assert n.shape == (1,) and n.dtype == torch.float32
    assert abs(float(n) - ref_norm) <= 2.0 ** -23 * ref_norm
    out = [torch.full_like(g, 9.0) for g in grads]
    assert torch.equal(qn.clip_grad_norm(grads, max_norm, out=out), n)
    for o, r, g, b in zip(out, ref, grads, before):
        check_scaled(o, r, o.dtype)
        assert torch.equal(g, b)
    assert torch.equal(qn.clip_grad_norm(grads, max_norm), n)
    for o, g in zip(out, grads):
        assert torch.equal(o, g)
    if len({g.dtype for g in grads}) == 1:
        flat = torch.full((sum(g.numel() for g in grads) + 2,), 9.0, dtype=grads[0].dtype,
                          device="cuda")
        qn.clip_grad_norm(before, max_norm, out=flat[1:-1])
        assert torch.equal(flat[1:-1], torch.cat([g.flatten() for g in grads]))
        assert flat[0] == 9.0 and flat[-1] == 9.0


SHAPES = [
    [(1,)], [(7,)], [(8,), (16,)], [(3, 5), (1, 1), (1023,), (64, 33)],
    [(16384,)], [(16383,), (16385,)], [(70000, 3)], [(8, 1024), (1024, 8), (2730, 8)],
    [(5,)] * 239, [(5,)] * 240, [(17,)] * 241, [(3, 3)] * 700, [(40000,)] * 170,
    [(0,), (4,), (0, 3), (2,)],
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32, None], ids=["bf16", "fp32", "both"])
@pytest.mark.parametrize("shapes", SHAPES, ids=lambda s: f"{len(s)}x{'x'.join(map(str, s[0]))}")
@pytest.mark.parametrize("max_norm", [0.5, 1e9])
def test_clip(shapes, dtype, max_norm):
    say(f"[clip] {len(shapes)} {shapes[:4]} {dtype} {max_norm}")
    grads = [draw(i, *s, std=0.1 + i % 3,
                  dtype=dtype or (torch.bfloat16, torch.float32)[(i // 2) % 2])
             for i, s in enumerate(shapes)]
    check(grads, max_norm)


def test_gradients_at_odd_addresses():
    say("[clip] odd addresses")
    for dt in (torch.bfloat16, torch.float32):
        flat = draw(1, 60001, dtype=dt)
        cuts = [1, 8, 20, 33333, 33336, 60000]
        check([flat[a:b] for a, b in zip(cuts, cuts[1:])], 1.0)


def test_more_than_2_to_31_elements():
    say("[clip] 64-bit offsets")
    n = (1 << 31) + 20001
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    tail = draw(1, 30000, dtype=torch.bfloat16)
    g[-30000:] = tail
    small = draw(2, 5)
    ref_norm, ref = norms.clip([host(tail), host(small)], 1.0)
    norm = qn.clip_grad_norm([g, small], 1.0)
    assert abs(float(norm) - ref_norm) <= 2.0 ** -23 * ref_norm
    check_scaled(g[-30000:], ref[0], g.dtype)
    check_scaled(small, ref[1], small.dtype)
    assert not g[:100000].any() and not g[-40000:-30000].any()


@pytest.mark.parametrize("std", [1e30, 1e18, 1e-25, 1e-38])
def test_sizes_whose_squares_leave_fp32(std):
    say(f"[clip] std {std}")
    check([draw(1, 5000, std=std), draw(2, 77, std=std)], 1.0)


def test_zero_gradients_and_a_limit_of_zero():
    say("[clip] zeros")
    g = [torch.zeros(100, device="cuda"), torch.zeros(3, device="cuda")]
    check(g, 1.0)
    g = [draw(1, 100)]
    qn.clip_grad_norm(g, 0.0)
    assert not g[0].any()
    check([draw(1, 100)], float("inf"))


@pytest.mark.parametrize("bad", ["nan", "inf"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_non_finite_gradients(bad, dtype):
    """A NaN anywhere scales everything by NaN, an infinity by 0."""
    say(f"[clip] {bad}")
    g = [draw(1, 300, dtype=dtype), draw(2, 5, dtype=dtype)]
    g[1][3] = float(bad)
    n = qn.clip_grad_norm(g, 1.0)
    if bad == "nan":
        assert torch.isnan(n).all() and torch.isnan(g[0]).all() and torch.isnan(g[1]).all()
    else:
        assert torch.isinf(n).all() and not g[0].any()
        assert torch.isnan(g[1][3]) and not g[1][:3].any()


def test_a_single_tensor_nones_and_another_stream():
    say("[clip] stream")
    a, b = draw(1, 1000, std=2.0), draw(2, 50)
    ref_norm, ref = norms.clip([host(a), host(b)], 1.0)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    n = qn.clip_grad_norm([None, a, None, b], 1.0, stream=st)
    st.synchronize()
    assert abs(float(n) - ref_norm) <= 2.0 ** -23 * ref_norm
    check_scaled(a, ref[0], a.dtype)
    check_scaled(b, ref[1], b.dtype)
    c = draw(3, 10)
    assert abs(float(qn.grad_norm(c)) - np.linalg.norm(host(c))) < 1e-6


def test_replays_in_a_graph():
    """No table is kept in device memory: a captured call replays on new values
    in the same gradients, every time."""
    say("[clip] graph")
    g = [draw(i, 3000 + i) for i in range(300)]
    ws = torch.empty(qn.lib().qlora_clip_workspace_size(300), dtype=torch.uint8, device="cuda")
    qn.clip_grad_norm(g, 1.0, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        n = qn.clip_grad_norm(g, 1.0, ws=ws)
    for k in range(4):
        for i, t in enumerate(g):
            t.copy_(draw(100 * k + i, 3000 + i))
        copy = [t.clone() for t in g]
        expect = qn.clip_grad_norm(copy, 1.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(n, expect)
        assert all(torch.equal(a, b) for a, b in zip(g, copy))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_no_limit_leaves_infinite_gradients_alone(dtype):
    """max_norm = inf: the same bits in place and elsewhere, though the norm is
    infinite; a NaN norm still scales by NaN."""
    say("[clip] no limit")
    inf = float("inf")
    g = [draw(1, 300, dtype=dtype), draw(2, 5, dtype=dtype)]
    g[1][3] = -inf
    before = [t.clone() for t in g]
    out = [torch.zeros_like(t) for t in g]
    for o in (out, None):
        n = qn.clip_grad_norm(g, inf, out=o)
        assert torch.isinf(n).all()
        for a, b in zip(g if o is None else o, before):
            assert torch.equal(a, b)
    ref_norm, ref = norms.clip([host(t) for t in before], inf)
    assert ref_norm == inf and all(np.array_equal(host(a), b) for a, b in zip(g, ref))
    g[0][7] = float("nan")
    n = qn.clip_grad_norm(g, inf)
    assert torch.isnan(n).all() and all(torch.isnan(t).all() for t in g)
