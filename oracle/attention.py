"""Attention and its gradients in fp64, one sequence and one head at a time,
and the error that bf16 roundings of the probabilities, of dS and of the
outputs may leave.

A "sequence" is a pair of row ranges; `sequences` lists them for a dense or a
packed batch, so that one function serves both.
"""

from dataclasses import dataclass
from typing import List, Optional, Tuple

import numpy as np

U = 2.0 ** -8   # largest relative error of rounding to bf16 (8 significant bits)


def sequences(q_rows: int, k_rows: int, cu_q=None, cu_k=None,
              batch: int = 1) -> List[Tuple[slice, slice]]:
    """(query rows, key rows) of each sequence in tensors flattened over the
    batch."""
    if cu_q is None:
        return [(slice(b * q_rows, (b + 1) * q_rows), slice(b * k_rows, (b + 1) * k_rows))
                for b in range(batch)]
    return [(slice(cu_q[s], cu_q[s + 1]), slice(cu_k[s], cu_k[s + 1]))
            for s in range(len(cu_q) - 1)]


def visible(lq: int, lk: int, causal: bool) -> np.ndarray:
    if not causal:
        return np.ones((lq, lk), bool)
    return np.arange(lk)[None, :] <= np.arange(lq)[:, None] + (lk - lq)


def probabilities(q, k, scale: float, causal: bool):
    """P [lq, lk] and lse [lq] of one head; rows that see nothing: 0, -inf."""
    s = scale * (q @ k.T)
    s = np.where(visible(len(q), len(k), causal), s, -np.inf)
    top = np.max(s, axis=1, initial=-np.inf)
    e = np.exp(s - np.where(np.isfinite(top), top, 0.0)[:, None])
    total = e.sum(1)
    with np.errstate(divide="ignore"):
        lse = np.where(total > 0, top + np.log(total), -np.inf)
    return e / np.where(total > 0, total, 1.0)[:, None], lse


@dataclass
class Result:
    o: np.ndarray
    lse: np.ndarray                      # [heads, rows]
    dq: Optional[np.ndarray] = None
    dk: Optional[np.ndarray] = None
    dv: Optional[np.ndarray] = None
    # name -> (largest error per element, variance per element)
    budget: Optional[dict] = None


def run(q, k, v, seqs, scale: float, causal: bool, do=None) -> Result:
    """q, do [Tq, H, D], k, v [Tk, Hkv, D] (fp64).  Outputs where no sequence
    has rows: o = 0, lse = -inf, gradients 0.

    The budget counts, for operands rounded to bf16 with a relative error of
    at most U and a variance of U^2 / 3 each, independent of one another:
      o   P and o itself
      dv  P and dv itself
      dq  dS, dq itself, and the row sums of dO O from an o with o's error
      dk  likewise."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    H, share = q.shape[1], q.shape[1] // k.shape[1]
    r = Result(np.zeros_like(q), np.full((H, q.shape[0]), -np.inf))
    lim = {n: np.zeros_like(x) for n, x in (("o", q), ("dq", q), ("dk", k), ("dv", v))}
    var = {n: np.zeros_like(x) for n, x in lim.items()}
    if do is not None:
        do = np.asarray(do, np.float64)
        r.dq, r.dk, r.dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for a, b in seqs:
        for h in range(H):
            g = h // share
            Q, K, V = q[a, h], k[b, g], v[b, g]
            P, lse = probabilities(Q, K, scale, causal)
            O = P @ V
            r.o[a, h], r.lse[h, a] = O, lse
            PV = P @ np.abs(V)
            o_var = U * U / 3 * (P * P @ (V * V) + O * O)
            lim["o"][a, h] = U * (PV + np.abs(O))
            var["o"][a, h] = o_var
            if do is None:
                continue
            G = do[a, h]
            dP = G @ V.T
            dS = P * (dP - (G * O).sum(1, keepdims=True))
            r.dv[b, g] += P.T @ G
            r.dk[b, g] += scale * dS.T @ Q
            r.dq[a, h] = scale * dS @ K
            d_lim = (np.abs(G) * lim["o"][a, h]).sum(1, keepdims=True)
            d_var = (G * G * o_var).sum(1, keepdims=True)
            lim["dv"][b, g] += U * P.T @ np.abs(G)
            var["dv"][b, g] += U * U / 3 * (P * P).T @ (G * G)
            e = U * np.abs(dS) + P * d_lim
            lim["dq"][a, h] = scale * e @ np.abs(K)
            lim["dk"][b, g] += scale * e.T @ np.abs(Q)
            # the error of a row's sum is common to the row: it moves dq along P K,
            # and dk's columns independently from row to row
            var["dq"][a, h] = scale ** 2 * (U * U / 3 * (dS * dS) @ (K * K) + d_var * (P @ K) ** 2)
            var["dk"][b, g] += scale ** 2 * (U * U / 3 * (dS * dS).T @ (Q * Q)
                                             + (P * P * d_var).T @ (Q * Q))
    if do is not None:
        for n, x in (("dq", r.dq), ("dk", r.dk), ("dv", r.dv)):
            lim[n] += U * np.abs(x)
            var[n] += U * U / 3 * x * x
    r.budget = {n: (lim[n], var[n]) for n in lim}
    return r
