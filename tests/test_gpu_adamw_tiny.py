"""The AdamW step where second moments are below the smallest normal number of
32 bits and eps adds nothing to their root.

Tolerance: m and v are the fp32 numbers of the states, exact here; the update
lr m^ / (sqrt(v^) + eps) then takes a root and a reciprocal (one unit in the
last place each, 2^-23), and four products, a sum and three rounded constants
(2^-24 each): 12 roundings of 2^-24, counted as 16."""

import numpy as np
import pytest
import torch

import quantized_base_lora_nf4_amd as qn
from oracle import adamw as oracle

pytestmark = pytest.mark.gpu

B1, B2, LR = 0.9, 0.999, 1e-2


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("eps", [0.0, 1e-25, 1e-20, 1e-8])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("t", [1, 1000])
def test_subnormal_second_moments(dtype, eps, bits, t):
    rng = np.random.default_rng(0)
    n = 1000
    # v from normal numbers down to a few units of the smallest subnormal one
    size = 10.0 ** rng.uniform(-21.0, -15.0, n)
    size[::256] = 1e-12   # 8 bits: a large one in every block, so that it keeps its scale
    g = torch.from_numpy(np.float32(size * rng.choice([-1, 1], n))).to(dtype)
    g64 = g.double().numpy()
    p = torch.zeros(n, device="cuda")
    state = qn.adamw_init([p], bits)
    qn.adamw_step([p], [g.cuda()], state, t, LR, betas=(B1, B2), eps=eps, weight_decay=0.0)
    m, v = oracle.states32(np.float32(g64), np.zeros(n, np.float32), np.zeros(n, np.float32), B1, B2)
    assert (v > 0).all() and (v < 2.0 ** -126).sum() > n // 2
    way = m.astype(np.float64) / (1 - B1 ** t) / (np.sqrt(v.astype(np.float64) / (1 - B2 ** t)) + eps)
    err = np.abs(p.cpu().numpy().astype(np.float64) + LR * way)
    assert float((err / (16 * 2.0 ** -24 * LR * np.abs(way))).max()) <= 1.0
    if bits == 32:
        assert np.array_equal(state.m[:n].cpu().numpy(), m) and np.array_equal(state.v[:n].cpu().numpy(), v)
    else:
        cm, cv, ms, vs = oracle.pack(m, v)
        assert np.array_equal(state.v.cpu().numpy(), cv) and np.array_equal(state.v_scale.cpu().numpy(), vs)
        assert np.array_equal(state.m.cpu().numpy(), cm) and np.array_equal(state.m_scale.cpu().numpy(), ms)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("ptype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("gtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("copied", [False, True])
def test_ordinary_gradients_with_no_eps(bits, ptype, gtype, copied):
    """The kernels for a small eps over ordinary values and several tensors: the
    update as above, the parameter rounded once to its type (half a step of
    2^-8 or 2^-24), its copy once to bf16."""
    gen = torch.Generator(device="cuda").manual_seed(0)
    sizes = (1, 255, 5000, 256 * 40)
    p = [(torch.randn(n, generator=gen, device="cuda")).to(ptype) for n in sizes]
    g = [(torch.randn(n, generator=gen, device="cuda") * 1e-3).to(gtype) for n in sizes]
    old = [t.double() for t in p]
    copies = [torch.empty_like(t, dtype=torch.bfloat16) for t in p] if copied else None
    qn.adamw_step(p, g, qn.adamw_init(p, bits), 3, LR, betas=(B1, B2), eps=0.0, weight_decay=0.1, copies=copies)
    half = 2.0 ** -24 if ptype == torch.float32 else 2.0 ** -8
    for i, (t, d, before) in enumerate(zip(p, g, old)):
        want, _, _ = oracle.step64(before.cpu(), d.double().cpu(), np.zeros(len(d)), np.zeros(len(d)), 3, LR, B1, B2, 0.0, 0.1)
        way = np.abs(want - before.cpu().numpy() * (1 - LR * 0.1))
        # (keep is rounded to fp32, and the product with it: 2 2^-24 of p)
        tol = 16 * 2.0 ** -24 * way + 2 * 2.0 ** -24 * np.abs(before.cpu().numpy())
        err = np.abs(t.double().cpu().numpy() - want)
        assert float((err - tol - half * (np.abs(want) + tol)).max()) <= 0.0
        if copied:
            err = np.abs(copies[i].double().cpu().numpy() - want)
            assert float((err - tol - 2.0 ** -8 * (np.abs(want) + tol)).max()) <= 0.0
