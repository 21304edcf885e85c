"""One AdamW step in fp64, and the 8-bit form of its states: the codes by their
definition, in fp32 operations that are each rounded once (numpy's), so that
they can be compared bit for bit."""

import numpy as np

BLOCK = 256
F = np.float32


def step64(p, grad, m, v, t, lr, b1, b2, eps, decay, factor=1.0):
    """(p, m, v) after the step, all fp64."""
    p, g, m, v = (np.asarray(x, np.float64) for x in (p, grad, m, v))
    g = g * factor
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    way = m / (1 - b1 ** t) / (np.sqrt(v / (1 - b2 ** t)) + eps)
    return p * (1 - lr * decay) - lr * way, m, v


def clip_factor(norm, max_norm) -> float:
    with np.errstate(invalid="ignore"):
        f = np.float64(max_norm) / (np.float64(norm) + 1e-6)
    return 1.0 if f >= 1.0 or max_norm == norm == np.inf else float(f)


def states32(grad, m, v, b1, b2, factor=1.0):
    """m and v after the step as fp32 operations rounded one by one."""
    g = np.asarray(grad, F) * F(factor)
    return (np.asarray(m, F) * F(b1) + g * F(1 - b1),
            np.asarray(v, F) * F(b2) + g * g * F(1 - b2))


def _blocks(x):
    n = -(-len(x) // BLOCK) * BLOCK
    return np.concatenate([x, np.zeros(n - len(x), x.dtype)]).reshape(-1, BLOCK)


def _scale(top):
    return np.where(~np.isfinite(top), F(np.nan), np.where(top < F(2.0 ** -96), F(0), top)).astype(F)


def pack(m, v):
    """(m codes int8, v codes uint8, m scales, v scales) of one tensor's fp32
    states, padded to whole blocks."""
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        m, v = _blocks(np.asarray(m, F)), _blocks(np.asarray(v, F))
        # (numpy's max passes NaN on)
        ms, vs = _scale(np.abs(m).max(1)), _scale(v.max(1))
        edges = (np.arange(1, 256) - 0.5) ** 2
        out = []
        for x, s, top, e in ((np.abs(m), ms, 127.0 ** 2, edges[:127]), (v, vs, 255.0 ** 4, (edges ** 2))):
            y = x * (F(top) / s)[:, None]
            c = np.searchsorted(e.astype(F), y.ravel(), side="right").reshape(y.shape)
            out.append(np.where(s[:, None] > 0, c, 0))
    cm, cv = out
    cv = np.where((vs[:, None] > 0) & (v > 0), np.maximum(cv, 1), cv)
    return (np.where(m < 0, -cm, cm).astype(np.int8).ravel(), cv.astype(np.uint8).ravel(), ms, vs)


def unpack(cm, cv, ms, vs):
    """The fp32 values that codes and scales stand for."""
    c, d = np.asarray(cm).astype(F).reshape(-1, BLOCK), np.asarray(cv).astype(F).reshape(-1, BLOCK)
    with np.errstate(invalid="ignore"):
        m = c * np.abs(c) * F(1 / 16129) * np.asarray(ms, F)[:, None]
        v = d * d
        v = v * v * F(1 / 255 ** 4) * np.asarray(vs, F)[:, None]
    return m.ravel(), v.ravel()
