"""The oracles of rotary positions and of the AdamW step, against closed forms,
torch's AdamW and brute force; rope_frequencies against its definitions."""

import math

import numpy as np
import pytest
import torch

import quantized_base_lora_nf4_amd as qn
from oracle import adamw, rope

RNG = np.random.default_rng(0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_norms_and_depends_on_the_distance_alone(interleaved):
    f = 10000.0 ** -(np.arange(8) / 8)
    q, k = RNG.standard_normal((2, 1, 1, 24))
    a = rope.rotate(q, [5], f, interleaved)
    assert np.allclose(np.linalg.norm(a), np.linalg.norm(q))
    assert np.array_equal(a[..., 16:], q[..., 16:])

    def score(i, j):
        return float((rope.rotate(q, [i], f, interleaved) * rope.rotate(k, [j], f, interleaved)).sum())
    assert score(12, 7) == pytest.approx(score(105, 100), rel=1e-12)
    back = rope.rotate(a, [5], f, interleaved, inverse=True)
    assert np.allclose(back, q, rtol=0, atol=1e-14)


def test_rotation_of_known_pairs():
    x = np.array([[[1.0, 2.0, 3.0, 4.0]]])
    quarter = [math.pi / 2, math.pi]
    assert np.allclose(rope.rotate(x, [1], quarter), [[[-3.0, -2.0, 1.0, -4.0]]])
    assert np.allclose(rope.rotate(x, [1], quarter, interleaved=True), [[[-2.0, 1.0, -3.0, -4.0]]])
    assert np.allclose(rope.rotate(x, [2], quarter, scale=2.0), [[[-2.0, 4.0, -6.0, 8.0]]])


def test_packed_positions():
    assert rope.packed_positions(7, [0, 2, 2, 5]) == [0, 1, 0, 1, 2, None, None]


def test_rope_gradient_against_differences():
    f = np.array([1.0, 0.3, 0.01])
    x, w = RNG.standard_normal((2, 2, 1, 8))
    pos = [3, 11]
    grad = rope.rotate(w, pos, f, scale=1.2, inverse=True)
    grad[..., 6:] = w[..., 6:]
    for i in np.ndindex(x.shape):
        h = 1e-6
        d = np.zeros_like(x)
        d[i] = h
        slope = ((rope.rotate(x + d, pos, f, scale=1.2) - rope.rotate(x - d, pos, f, scale=1.2)) * w).sum()
        assert slope / (2 * h) == pytest.approx(grad[i], abs=1e-8)


def test_frequencies():
    f, s = qn.rope_frequencies(64, device="cpu")
    assert f.dtype == torch.float64 and s == 1.0
    assert np.allclose(f, 10000.0 ** -(np.arange(32) / 32), rtol=1e-15)
    g, s = qn.rope_frequencies(64, scaling="linear", factor=4.0, device="cpu")
    assert torch.equal(g, f / 4) and s == 1.0
    g, s = qn.rope_frequencies(64, scaling="base", factor=4.0, device="cpu")
    assert g[0] == f[0] and float(g[-1]) == pytest.approx(float(f[-1]) / 4, rel=1e-12)
    for how in ("parts", "bands"):
        g, s = qn.rope_frequencies(64, scaling=how, factor=4.0, length=2048, low=1.0, high=16.0, device="cpu")
        turns = 2048 * f / (2 * math.pi)
        assert torch.equal(g[turns >= 16], f[turns >= 16])
        slow = turns <= 1
        assert slow.any() and torch.equal(g[slow], f[slow] / 4)
        assert ((g <= f) & (g >= f / 4)).all()
        assert s == (0.1 * math.log(4.0) + 1.0 if how == "parts" else 1.0)


@pytest.mark.parametrize("kw,match", [
    (dict(dim=7), "even"), (dict(dim=0), "even"), (dict(dim=8, scaling="other"), "scaling"),
    (dict(dim=8, factor=0.5), "factor"), (dict(dim=8, base=0.0), "base"),
    (dict(dim=2, scaling="base"), "4 elements"), (dict(dim=8, scaling="bands", low=4.0, high=4.0), "high"),
])
def test_frequencies_refuse(kw, match):
    with pytest.raises(ValueError, match=match):
        qn.rope_frequencies(device="cpu", **kw)


def test_step_against_torch():
    p0, m, v = RNG.standard_normal(50), np.zeros(50), np.zeros(50)
    t = torch.nn.Parameter(torch.from_numpy(p0.copy()))
    opt = torch.optim.AdamW([t], lr=1e-2, betas=(0.8, 0.95), eps=1e-6, weight_decay=0.1)
    p = p0
    for i in range(1, 6):
        g = RNG.standard_normal(50)
        t.grad = torch.from_numpy(g.copy())
        opt.step()
        p, m, v = adamw.step64(p, g, m, v, i, 1e-2, 0.8, 0.95, 1e-6, 0.1)
        assert np.allclose(p, t.detach().numpy(), rtol=1e-12, atol=1e-14)


def test_clip_factor():
    assert adamw.clip_factor(2.0, 1.0) == 1.0 / (2.0 + 1e-6)
    assert adamw.clip_factor(0.5, 1.0) == 1.0
    assert adamw.clip_factor(np.inf, 1.0) == 0.0
    assert adamw.clip_factor(np.inf, np.inf) == 1.0
    assert math.isnan(adamw.clip_factor(np.nan, 1.0))


def test_codes_are_the_nearest_in_the_companded_domain():
    m = (RNG.standard_normal(700) * 10.0 ** RNG.uniform(-4, 0, 700)).astype(np.float32)
    v = (m * m).astype(np.float32)
    cm, cv, ms, vs = adamw.pack(m, v)
    assert len(cm) == len(cv) == 768 and len(ms) == 3
    for i in range(700):
        b = i // 256
        s, w = float(ms[b]), float(vs[b])
        assert s == np.abs(m[256 * b:256 * (b + 1)]).max()
        root = math.sqrt(abs(float(m[i])) / s) * 127
        assert abs(abs(int(cm[i])) - root) <= 0.5 + 1e-4 and (cm[i] == 0 or (cm[i] > 0) == (m[i] > 0))
        root = (float(v[i]) / w) ** 0.25 * 255
        assert abs(int(cv[i]) - root) <= 0.5 + 1e-4 or (cv[i] == 1 and root < 0.5)
    assert not cm[700:].any() and not cv[700:].any()
    # the largest come back as they are but for the rounding of the constant
    um, uv = adamw.unpack(cm, cv, ms, vs)
    for b in range(3):
        assert np.abs(um[256 * b:256 * (b + 1)]).max() == pytest.approx(ms[b], rel=2.0 ** -22)
        assert uv[256 * b:256 * (b + 1)].max() == pytest.approx(vs[b], rel=2.0 ** -22)


def test_codes_of_codes_are_the_codes():
    cm = RNG.integers(-127, 128, 512).astype(np.int8)
    cv = RNG.integers(0, 256, 512).astype(np.uint8)
    cm[[0, 256]], cv[[1, 257]] = 127, 255
    ms, vs = np.array([0.3, 1e-20], np.float32), np.array([2e-9, 5.0], np.float32)
    m, v = adamw.unpack(cm, cv, ms, vs)
    a, b, c, d = adamw.pack(m, v)
    assert np.array_equal(a, cm) and np.array_equal(b, cv)


def test_codes_of_special_blocks():
    x = np.zeros(1024, np.float32)
    x[3] = 2.0 ** -97          # below the smallest scale
    x[256 + 3], x[256 + 4] = np.inf, 1.0
    x[512 + 3], x[512 + 4] = np.nan, 1.0
    x[768 + 3], x[768 + 4] = 1.0, 1e-30   # not 0: v's code is 1
    cm, cv, ms, vs = adamw.pack(x, x)
    assert ms[0] == vs[0] == 0 and not cm[:256].any() and not cv[:256].any()
    assert np.isnan(ms[1:3]).all() and np.isnan(vs[1:3]).all() and not cm[256:768].any()
    assert cm[771] == 127 and cm[772] == 0 and cv[771] == 255 and cv[772] == 1
    m, v = adamw.unpack(cm, cv, ms, vs)
    assert np.isnan(m[256:768]).all() and np.isnan(v[256:768]).all() and v[772] > 0


def test_new_states():
    ps = [torch.zeros(n) for n in (1, 256, 0, 257)]
    s = qn.adamw_init(ps, 8)
    assert s.bits == 8 and s.m.numel() == 1024 and s.m_scale.numel() == 4 and s.nbytes() == 2048 + 32
    s = qn.adamw_init(ps)
    assert s.bits == 32 and s.v.numel() == 1024 and s.m_scale is None and s.nbytes() == 8192
    with pytest.raises(ValueError, match="bits"):
        qn.adamw_init(ps, 16)
    with pytest.raises(ValueError, match="no parameters"):
        qn.adamw_init([])
