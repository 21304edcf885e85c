"""Layer norm and root-mean-square norm with their gradients, and the clipping
of gradients by their global norm, in fp64."""

import numpy as np


def norm_forward(x, weight, bias, eps: float, rms: bool):
    """(y, mean, rstd) over the rows of x [rows, width]; mean is 0 if rms."""
    x = np.asarray(x, np.float64)
    mean = np.zeros(len(x)) if rms else x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None] * np.asarray(weight, np.float64)
    return (y if bias is None else y + np.asarray(bias, np.float64)), mean, rstd


def norm_backward(dy, x, weight, eps: float, rms: bool):
    """(dx, dweight, dbias), from the definition (the statistics are those of
    x, not given)."""
    dy, weight = np.asarray(dy, np.float64), np.asarray(weight, np.float64)
    x = np.asarray(x, np.float64)
    _, mean, rstd = norm_forward(x, weight, None, eps, rms)
    z = (x - mean[:, None]) * rstd[:, None]
    g = dy * weight
    dx = g - z * (g * z).mean(1, keepdims=True)
    if not rms:
        dx = dx - g.mean(1, keepdims=True)
    return dx * rstd[:, None], (dy * z).sum(0), dy.sum(0)


def clip(grads, max_norm: float):
    """(norm, scaled gradients) of a list of arrays."""
    norm = np.sqrt(sum(float((np.asarray(g, np.float64) ** 2).sum()) for g in grads))
    # without a limit nothing is scaled, whatever size the norm has
    factor = 1.0 if max_norm == norm == np.inf else max_norm / (norm + 1e-6)
    factor = 1.0 if factor >= 1.0 else factor
    return norm, [np.asarray(g, np.float64) * factor for g in grads]
