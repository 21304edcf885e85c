"""CPU pins of the oracle's attention, norms and clipping: the gradients
against central differences of the forward pass in fp64, and the forwards
against closed forms."""

import numpy as np
import pytest

from oracle import attention, norms

# Central differences with step h leave an error of h^2 / 6 times the third
# derivative (of order 1 to 10 here) plus rounding 1e-16 / h: at h = 1e-5,
# about 1e-9 and 1e-11 for derivatives of order 1.
H, TOL = 1e-5, 1e-7


def _difference(f, x, d):
    return (f(x + H * d) - f(x - H * d)) / (2 * H)


@pytest.mark.parametrize("lq,lk,heads,kv,causal", [
    (1, 1, 1, 1, True), (5, 5, 2, 2, True), (4, 9, 4, 2, True), (9, 4, 2, 1, True),
    (7, 3, 3, 3, False)])
def test_attention_gradients_are_the_differences(lq, lk, heads, kv, causal):
    rng = np.random.default_rng(lq * 100 + lk)
    q, k, v = (rng.standard_normal((n, h, 8)) for n, h in ((lq, heads), (lk, kv), (lk, kv)))
    do = rng.standard_normal((lq, heads, 8))
    seqs = attention.sequences(lq, lk)
    r = attention.run(q, k, v, seqs, 0.4, causal, do)

    def loss(q, k, v):
        return float((attention.run(q, k, v, seqs, 0.4, causal).o * do).sum())

    for x, g, f in ((q, r.dq, lambda t: loss(t, k, v)), (k, r.dk, lambda t: loss(q, t, v)),
                    (v, r.dv, lambda t: loss(q, k, t))):
        d = rng.standard_normal(x.shape)
        assert abs(_difference(f, x, d) - (g * d).sum()) < TOL * (1 + abs((g * d).sum()))


def test_attention_of_one_key_is_its_value_and_of_none_is_zero():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 1, 4)), rng.standard_normal((1, 1, 4)), \
        rng.standard_normal((1, 1, 4))
    r = attention.run(q, k, v, attention.sequences(3, 1), 0.5, True, np.ones((3, 1, 4)))
    assert np.array_equal(r.o[:2], np.zeros((2, 1, 4))) and np.allclose(r.o[2], v[0])
    assert np.all(np.isneginf(r.lse[0, :2])) and np.isclose(r.lse[0, 2], 0.5 * (q[2, 0] @ k[0, 0]))
    # one key: the probability is 1 whatever the score.  dP and its mean are the same four
    # products summed in two orders, so what is left is their rounding (4 * 2^-53 of terms of order 1)
    assert np.abs(r.dq).max() < 1e-14 and np.abs(r.dk).max() < 1e-14


def test_attention_with_equal_scores_is_the_mean():
    v = np.arange(12.0).reshape(6, 1, 2)
    z = np.zeros((6, 1, 2))
    r = attention.run(z, z, v, attention.sequences(6, 6), 1.0, True)
    for i in range(6):
        assert np.allclose(r.o[i, 0], v[: i + 1, 0].mean(0))
        assert np.isclose(r.lse[0, i], np.log(i + 1))


def test_packed_sequences_do_not_see_each_other():
    rng = np.random.default_rng(2)
    q, k, v, do = (rng.standard_normal((7, 1, 4)) for _ in range(4))
    cu = [0, 3, 3, 7]
    r = attention.run(q, k, v, attention.sequences(7, 7, cu, cu), 0.5, False, do)
    for a, b in ((0, 3), (3, 7)):
        one = attention.run(q[a:b], k[a:b], v[a:b], attention.sequences(b - a, b - a), 0.5, False,
                            do[a:b])
        assert np.allclose(r.o[a:b], one.o) and np.allclose(r.dk[a:b], one.dk)


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("rows,width", [(1, 2), (3, 7), (5, 32)])
def test_norm_gradients_are_the_differences(rows, width, rms):
    rng = np.random.default_rng(width)
    x, dy = rng.standard_normal((rows, width)) + 0.5, rng.standard_normal((rows, width))
    w, b = rng.standard_normal(width), rng.standard_normal(width)
    dx, dw, db = norms.norm_backward(dy, x, w, 1e-2, rms)

    def loss(x, w, b):
        return float((norms.norm_forward(x, w, b, 1e-2, rms)[0] * dy).sum())

    for t, g, f in ((x, dx, lambda t: loss(t, w, b)), (w, dw, lambda t: loss(x, t, b)),
                    (b, db, lambda t: loss(x, w, t))):
        d = rng.standard_normal(t.shape)
        assert abs(_difference(f, t, d) - (g * d).sum()) < TOL * (1 + abs((g * d).sum()))


def test_norm_of_a_row_has_mean_zero_and_variance_one():
    x = np.random.default_rng(3).standard_normal((4, 100)) * 5 + 3
    y, mean, rstd = norms.norm_forward(x, np.ones(100), None, 0.0, False)
    assert np.allclose(y.mean(1), 0) and np.allclose(y.var(1), 1)
    assert np.allclose(mean, x.mean(1)) and np.allclose(rstd, 1 / x.std(1))
    y, _, _ = norms.norm_forward(x, np.ones(100), None, 0.0, True)
    assert np.allclose((y * y).mean(1), 1)


def test_clip_leaves_small_gradients_and_bounds_large_ones():
    g = [np.array([3.0, 0.0]), np.array([[4.0]])]
    norm, out = norms.clip(g, 10.0)
    assert norm == 5.0 and np.array_equal(out[0], g[0])
    norm, out = norms.clip(g, 1.0)
    assert np.isclose(np.sqrt(sum((o ** 2).sum() for o in out)), 1.0, atol=1e-6)
