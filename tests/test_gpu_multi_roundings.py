"""Rows of many adapters: the roundings that each kernel makes, and no others.

Up to 16 rows (the weight stream) and from 17 rows on while the rows' kernel is
taken, a weight is its level, rounded to bf16 after a factor that brings the
levels nearer to bf16 values, times an fp32 constant; U stays in fp32.  Elsewhere
(the tiles) it is the bf16 weight that nf4_dequantize gives, and s U is rounded
to bf16 once.

Tolerance: against fp64 products with the weight that the path has, an output is
rounded once (2^-8 of it), and sums, constants and U are fp32: K + r + 16
roundings of 2^-24 of the sum of magnitudes.  The tiles' rounding of s U (2^-8 of
each at most, independent over the rank) adds 8 deviations of
2^-8 sqrt(sum (s u b)^2)."""

import numpy as np
import pytest
import torch

import quantized_base_lora_nf4_amd as qn
from gpu_util import say

pytestmark = pytest.mark.gpu

BF = torch.bfloat16
U = 2.0 ** -8
FACTOR = {"nf4": 1.43701171875, "nf3": 1.781005859375, "nf2": 1.15625, "fp4": 1.0078125, "user4": 1.0}
STREAM, ROWS, TILES = "stream", "rows", "tiles"


def path_of(M, N, K, r):
    """Which kernels a call takes, from its workspace: 32 slices of U for the
    stream, X in another order for the rows' kernel, an order of rows (4 bytes
    each) for the tiles, beside partial sums of U."""
    ws = qn.multi_workspace_size(M, N, K, r)

    def up(n):
        return -(-n // 256) * 256
    if M <= 16 and ws == up(32 * M * r * 4):
        return STREAM
    part = [up(s * M * -(-r // 8) * 8 * 4) for s in range(1, 9)]
    rows, tiles = (any(ws == p + up(n) for p in part) for n in (-(-M // 16) * 16 * K * 2, M * 4))
    assert rows != tiles
    return ROWS if rows else TILES


def weights(w, code, levels):
    """(the rounded levels times their constants, the bf16 weight) in fp64."""
    W = qn.nf4_dequantize(w).double()
    const = w.q8.double() * w.step.double().repeat_interleave(256)[:w.q8.numel()]
    const = const.view(w.N, -1).repeat_interleave(w.blocksize, 1)
    L = torch.tensor(levels, dtype=torch.float64, device="cuda")
    # (bf16 values are within 2^-8 of level times constant: the nearest is it)
    ratio = torch.where(const > 0, W / const, 0.0)
    at = torch.cat([(part.unsqueeze(-1) - L).abs().argmin(-1) for part in ratio.split(64)])
    # fp32 product, then bf16, as the table is made
    rounded = (L.float() * FACTOR[code]).to(BF).double() / FACTOR[code]
    return torch.where(const > 0, rounded[at] * const, 0.0), W


@pytest.mark.parametrize("code,blocksize", [("nf4", 64), ("nf4", 128), ("fp4", 64), ("nf3", 64), ("nf2", 64), ("user4", 64)])
@pytest.mark.parametrize("path,M,N,K,r", [
    (STREAM, 1, 136, 512, 16), (STREAM, 7, 264, 640, 9), (STREAM, 16, 1024, 256, 64), (ROWS, 16, 64, 64 * 520, 256), (TILES, 16, 64, 64 * 1200, 8),
    (ROWS, 17, 136, 512, 16), (ROWS, 40, 264, 256, 33), (ROWS, 129, 1032, 512, 64), (ROWS, 64, 16392, 256, 24),
    (TILES, 4100, 136, 256, 16), (TILES, 4200, 264, 512, 75)])
def test_roundings(path, M, N, K, r, code, blocksize):
    say(f"[multi] {path}: {M} rows, {N} x {K}, rank {r}, {code}, blocks of {blocksize}")
    assert path_of(M, N, K, r) == path
    g = torch.Generator(device="cuda").manual_seed(0)
    levels = list(np.linspace(-1, 1, 16)) if code == "user4" else qn.code_table(code)[0]
    w = qn.nf4_quantize(torch.randn(N, K, generator=g, device="cuda") * K ** -0.5, code=code, blocksize=blocksize,
                        levels=np.array(levels) if code == "user4" else None)
    if code == "user4":
        levels = [float(np.float32(v)) for v in levels]
    n = 4
    A = (torch.randn(n, r, K, generator=g, device="cuda") * K ** -0.5).to(BF)
    B = (torch.randn(n, N, r, generator=g, device="cuda") * 0.5).to(BF)
    s = torch.rand(n, generator=g, device="cuda") * 4 - 1
    X = torch.randn(M, K, generator=g, device="cuda").to(BF)
    index = (torch.arange(M) % (n + 1) - 1).to(torch.int32).cuda()     # -1: the base alone
    Y = qn.qlora_linear_multi_fwd(w, X, A, B, s, index).double()
    fine, W = weights(w, code, levels)
    x = X.double()
    here = W if path == TILES else fine
    ref, size, var = x @ here.T, x.abs() @ here.abs().T, torch.zeros(M, N, dtype=torch.float64, device="cuda")
    for a in range(n):
        m = (index == a).nonzero().flatten()
        u = x[m] @ A[a].double().T * float(s[a])
        ref[m] += u @ B[a].double().T
        size[m] += (x[m].abs() @ A[a].double().abs().T * abs(float(s[a]))) @ B[a].double().abs().T
        var[m] += (u * u) @ B[a].double().square().T
    tol = U * ref.abs() * (1 + U) + (K + r + 16) * 2.0 ** -24 * size
    if path == TILES:
        tol += 8 * U * var.sqrt()
    err = (Y - ref).abs()
    say(f"    {float((err / tol).max()):.3f} of the bound, {float(err.norm() / ref.norm()):.2e} of the norm")
    assert float((err - tol).max()) <= 0.0
    base = index < 0
    if base.any() and path != TILES and code != "user4":
        # the bf16 weight's rounding is not made as well: against products with
        # it these rows are off by more than their own rounding
        other = ((Y - x @ W.T)[base]).norm() / ref[base].norm()
        assert float(other) > float(err[base].norm() / ref[base].norm())
