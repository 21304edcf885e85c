"""Rotation in place, against the rotation into new tensors, whose values
test_gpu_rope.py checks: the same bits in every layout, and what is not turned
stays as it is."""

import pytest
import torch

import quantized_base_lora_nf4_amd as qn
from gpu_util import say

pytestmark = pytest.mark.gpu


def randn(*shape, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 64), (64, 32), (128, 126), (80, 20), (136, 34), (72, 70), (8, 2)])
@pytest.mark.parametrize("cu", [None, [0, 60], [0, 5], [0, 0, 3, 3, 40, 41, 41], [0, 20, 57], [0, 0], [7, 30]])
def test_in_place(dim, rot, interleaved, cu):
    say(f"[rope] in place, heads of {dim}, {rot} turned, interleaved {interleaved}, offsets {cu}")
    f, scale = qn.rope_frequencies(rot, scaling="parts" if rot > 8 else None, factor=4.0)
    rows = 60
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda")
    none = torch.ones(rows, dtype=torch.bool, device="cuda")   # rows of no sequence
    none[0 if cu is None else cu[0]:rows if cu is None else cu[-1]] = False
    for call in (qn.rope_fwd, qn.rope_bwd):
        qkv = randn(rows, 6 + 3 + 3, dim)                      # views of one tensor, rows apart
        q, k, v = qkv.split([6, 3, 3], 1)
        before = qkv.clone()
        how = dict(cu_seqlens=c, interleaved=interleaved, scale=scale)
        a, b = call(q, k, f, **how)
        assert torch.equal(qkv, before)
        x, y = call(q, k, f, out=(q, k), **how)
        assert x is q and y is k
        assert torch.equal(q, a) and torch.equal(k, b) and torch.equal(v, before[:, 9:])
        assert torch.equal(qkv[none], before[none])
        assert torch.equal(qkv[..., rot:], before[..., rot:])
        turned = qkv[~none][:, :9, :rot] != before[~none][:, :9, :rot]
        # (of rows at positions above 0 something changes: this is a rotation)
        assert cu is not None and cu[-1] - cu[0] < 2 or turned.any()
        # q alone, k as it was
        q2, k2 = before.split([6, 3, 3], 1)[:2]
        kept = k2.clone()
        call(q2, None, f, out=(q2, None), **how)
        assert torch.equal(q2, a) and torch.equal(k2, kept)


def test_in_place_dense_with_positions():
    f, _ = qn.rope_frequencies(48)
    q, k = randn(3, 9, 4, 64), randn(3, 9, 2, 64, seed=1)
    pos = torch.randint(0, 1 << 20, (3, 9), generator=torch.Generator().manual_seed(0)).cuda()
    for interleaved in (False, True):
        a, b = qn.rope_fwd(q, k, f, positions=pos, interleaved=interleaved)
        x, y = q.clone(), k.clone()
        qn.rope_fwd(x, y, f, positions=pos, interleaved=interleaved, out=(x, y))
        assert torch.equal(x, a) and torch.equal(y, b)
        assert torch.equal(x[..., 48:], q[..., 48:]) and torch.equal(y[..., 48:], k[..., 48:])
        assert not torch.equal(x, q)
