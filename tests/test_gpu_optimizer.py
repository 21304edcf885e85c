"""The optimizer and its step where parameters differ in their history, and
what an update tells torch."""

import pytest
import torch

import quantized_base_lora_nf4_amd as qn
from gpu_util import say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
SHAPES = ((8, 300), (77,), (513,))


def _params(dtype=F32, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.nn.Parameter((0.1 * torch.randn(*s, generator=g, device="cuda")).to(dtype)) for s in SHAPES]


def _have(step):
    """The parameters with a gradient: one in every step, one from the 20th on,
    one in every third step."""
    return [True, step >= 20, step % 3 == 2]


def test_gradients_that_begin_late():
    """Against torch's optimizer in 64 bits.  Per step and element an update of
    lr |m^ / sqrt(v^)|, at most 4 lr for these gradients, is off by up to 16
    roundings (states, root, reciprocal, products) and the parameter, below 1,
    is rounded once: 30 (2^-24 + 64 lr 2^-24) in 30 steps."""
    steps, lr = 30, 1e-2
    a = _params()
    b = [torch.nn.Parameter(p.detach().double()) for p in a]
    x, y = qn.AdamW(a, lr=lr, weight_decay=0.1), torch.optim.AdamW(b, lr=lr, weight_decay=0.1)
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(steps):
        for p, q, has in zip(a, b, _have(i)):
            p.grad = torch.randn(p.shape, generator=g, device="cuda") if has else None
            q.grad = p.grad.double() if has else None
        x.step()
        y.step()
    bound = steps * 2.0 ** -24 * (1 + 64 * lr)
    for n, p, q in zip(SHAPES, a, b):
        err = float((p.detach().double() - q.detach()).abs().max())
        say(f"    {n}: {err:.2e}, bound {bound:.2e}")
        assert err <= bound


@pytest.mark.parametrize("bits,dtype,masters", [(32, F32, False), (8, F32, False), (8, BF, False), (8, BF, True)])
def test_a_group_is_its_parameters(bits, dtype, masters):
    """The same bits as with an optimizer for each parameter."""
    kw = dict(lr=1e-2, weight_decay=0.1, bits=bits, masters=masters)
    a, b = _params(dtype), _params(dtype)
    x, ys = qn.AdamW(a, **kw), [qn.AdamW([q], **kw) for q in b]
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(24):
        for p, q, has in zip(a, b, _have(i)):
            p.grad = torch.randn(p.shape, generator=g, device="cuda").to(dtype) if has else None
            q.grad = p.grad
        x.step()
        for y in ys:
            y.step()
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_counts_of_a_step():
    """adamw_step with a count for each tensor: the step with that count."""
    g = torch.Generator(device="cuda").manual_seed(2)
    p = [torch.randn(n, generator=g, device="cuda") for n in (300, 0, 77, 5000)]
    d = [torch.randn_like(t) for t in p]
    counts = [7, 1, 1000000, 7]
    each = []
    for t, e, c in zip(p, d, counts):
        t = t.clone()
        if t.numel():
            qn.adamw_step([t], [e], qn.adamw_init([t]), c, 1e-2)
        each.append(t)
    for left in ((), (2,), (0, 3)):
        q = [t.clone() for t in p]
        qn.adamw_step(q, [None if i in left else e for i, e in enumerate(d)], qn.adamw_init(q), counts, 1e-2)
        for i, (t, e) in enumerate(zip(q, each)):
            assert torch.equal(t, p[i] if i in left else e)
    for bad, match in (([1, 2], "2 steps for 4"), ([1, 1, 0, 1], "from 1"), ([1, 1, 1.5, 1], "whole numbers")):
        q = [t.clone() for t in p]
        with pytest.raises(ValueError, match=match):
            qn.adamw_step(q, d, qn.adamw_init(q), bad, 1e-2)
        assert all(torch.equal(s, t) for s, t in zip(p, q))
    # what has no gradient is not looked at
    q = [t.clone() for t in p]
    qn.adamw_step(q, [d[0], None, None, None], qn.adamw_init(q), [7, 0, -3, 0], 1e-2)
    assert torch.equal(q[0], each[0]) and torch.equal(q[2], p[2])
