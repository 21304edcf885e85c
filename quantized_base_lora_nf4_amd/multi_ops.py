"""Thin torch binding of the layer for rows of many adapters.  As in
:mod:`quantized_base_lora_nf4_amd.train_ops`: argument checks and marshalling
only, every call enqueues on ``torch.cuda.current_stream()`` of the weight's
device unless a stream is passed."""

import ctypes
from typing import Optional

import torch

from ._lib import check, lib, tensors, written
from .ops import NF4Weight, QLoRALinear, _check_weight
from .train_ops import _SIXTEEN, _bytes, _on, _same, _scratch


def multi_workspace_size(M: int, N: int, K: int, r: int) -> int:
    return int(lib().qlora_multi_workspace_size(M, N, K, r))


def qlora_linear_multi_fwd(w: NF4Weight, X: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                           s: torch.Tensor, index: torch.Tensor, Y: Optional[torch.Tensor] = None,
                           ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Rows of many adapters over one frozen weight:
    Y_i = X_i W^T + s_a (X_i A_a^T) B_a^T with a = index[i], and X_i W^T where
    index[i] is not one of 0 .. n - 1.

    X [M, K] (M at least 1), A [n, r, K], B [n, N, r] bf16 (adapters of smaller
    rank padded with zeros), s [n] float32, index [M] int32, all on the weight's
    GPU.  Rows may come in any order; Y overlaps nothing that is read.  M, N, K
    and r choose the kernel, and with it where bf16 is rounded to (see the C
    header): a row's last bits depend on how many rows come with it."""
    dev = _check_weight(w)
    if dev.type != "cuda":
        raise ValueError(f"codes is on {dev}, expected a GPU")
    for name, t, nd in (("X", X, 2), ("A", A, 3), ("B", B, 3)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch tensor")
        if t.dim() != nd:
            raise ValueError(f"{name} must be {nd}-D")
    M, N, K = len(X), w.N, w.K
    n, r, _ = A.shape
    # (the weight's types are checked above, its layout with its struct below)
    for name, t in (("q8", w.q8), ("step", w.step)):
        if t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if not tensors().fits(dev.index, "sssfi", (X, A, B, s, index),
                          ((M, K), (n, r, K), (n, N, r), (n,), (M,))):
        _same("X", X, (M, K), _SIXTEEN, dev)
        _same("A", A, (n, r, K), _SIXTEEN, dev)
        _same("B", B, (n, N, r), _SIXTEEN, dev)
        _same("s", s, (n,), (torch.float32,), dev)
        _same("index", index, (M,), (torch.int32,), dev)
    if Y is not None:
        _same("Y", Y, (M, N), _SIXTEEN, dev)
    given = Y
    st, ctx = _on(dev, stream)
    with ctx:
        if Y is None:
            Y = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
        L = lib()
        ws = _scratch(L.qlora_multi_workspace_size(M, N, K, r), dev, ws)
        rc = L.qlora_linear_multi_fwd(ctypes.byref(w.struct()), X.data_ptr(), M, A.data_ptr(),
                                      B.data_ptr(), s.data_ptr(), n, r, index.data_ptr(), Y.data_ptr(),
                                      ws.data_ptr(), _bytes(ws), st)
    check(rc, "qlora_linear_multi_fwd")
    if given is not None:
        written(given)
    return Y


class QLoRAMultiLinear(torch.nn.Module):
    """A frozen NF4 weight with `slots` places for LoRA pairs of rank up to r,
    for rows that each use one of them (serving what QLoRALinear trained; no
    gradients).  The weight is a QLoRALinear's (shared, not copied) or an
    NF4Weight."""

    def __init__(self, base, slots: int, r: int):
        super().__init__()
        self.nf4 = base.nf4 if isinstance(base, QLoRALinear) else base
        dev = self.nf4.codes.device
        self.register_buffer("A", torch.zeros(slots, r, self.nf4.K, dtype=torch.bfloat16, device=dev))
        self.register_buffer("B", torch.zeros(slots, self.nf4.N, r, dtype=torch.bfloat16, device=dev))
        self.register_buffer("scales", torch.zeros(slots, dtype=torch.float32, device=dev))

    @torch.no_grad()
    def put(self, slot: int, A: torch.Tensor, B: torch.Tensor, s: float) -> None:
        """Copy an adapter (A [k, K], B [N, k], k <= r) with its scale into a slot."""
        slots, r, K = self.A.shape
        if not 0 <= slot < slots:
            raise ValueError(f"slot {slot} is not one of {slots}")
        k = A.shape[0]
        if k > r or A.shape != (k, K) or B.shape != (self.nf4.N, k):
            raise ValueError(f"A {tuple(A.shape)} and B {tuple(B.shape)} do not fit rank {r} beside a "
                             f"{self.nf4.N} x {K} weight")
        self.A[slot].zero_()[:k] = A
        self.B[slot].zero_()[:, :k] = B
        self.scales[slot] = s

    def load(self, slot: int, layer: QLoRALinear) -> None:
        """Copy the adapter of a QLoRALinear into a slot."""
        self.put(slot, layer.A, layer.B, layer.s)

    @torch.no_grad()
    def forward(self, X, index):
        """X [..., K] bf16 of one row or more, index int32 of X's leading shape:
        the slot of each row, -1 for none."""
        shp = X.shape
        Y = qlora_linear_multi_fwd(self.nf4, X.reshape(-1, shp[-1]).contiguous(), self.A, self.B,
                                   self.scales, index.reshape(-1).contiguous())
        return Y.reshape(*shp[:-1], Y.shape[-1])
