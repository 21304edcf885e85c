"""Thin torch binding of the AdamW step over many tensors, and an optimizer
around it.  As in :mod:`quantized_base_lora_nf4_amd.train_ops`: argument checks
and marshalling only, every call enqueues on ``torch.cuda.current_stream()`` of
the tensors' device unless a stream is passed."""

import array
import math
from dataclasses import dataclass
from typing import Optional

import torch

from ._lib import QLORA_ADAMW_BLOCK, QLORA_TYPE_BF16, check, lib, tensors, written
from ._lib import AdamW as _Args
from .train_ops import _describe, _device_of, _grad_arrays, _on, _ptr_of, _same, grad_norm


@dataclass
class AdamWState:
    """The states of a list of tensors, one after the other, each from a
    multiple of 256 elements on (new states are zeros).  32 bits: m and v are
    float32.  8 bits: m int8, v uint8, with one float32 scale each per block of
    256 elements of a tensor."""
    m: torch.Tensor
    v: torch.Tensor
    m_scale: Optional[torch.Tensor] = None
    v_scale: Optional[torch.Tensor] = None

    @property
    def bits(self) -> int:
        return 8 if self.m.dtype == torch.int8 else 32

    def nbytes(self) -> int:
        return sum(t.numel() * t.element_size()
                   for t in (self.m, self.v, self.m_scale, self.v_scale) if t is not None)


def _spans(sizes):
    """Elements that each tensor takes in the states."""
    return [-(-n // QLORA_ADAMW_BLOCK) * QLORA_ADAMW_BLOCK for n in sizes]


def adamw_init(params, bits: int = 32, device=None) -> AdamWState:
    """New states (zeros) for a list of tensors, on their device unless one is
    given."""
    if bits not in (8, 32):
        raise ValueError(f"bits must be 8 or 32, got {bits}")
    params = list(params)
    if device is None:
        if not params:
            raise ValueError("there are no parameters")
        device = params[0].device
    n = sum(_spans(p.numel() for p in params))
    if bits == 32:
        return AdamWState(*(torch.zeros(n, dtype=torch.float32, device=device) for _ in range(2)))
    return AdamWState(torch.zeros(n, dtype=torch.int8, device=device),
                      torch.zeros(n, dtype=torch.uint8, device=device),
                      *(torch.zeros(n // QLORA_ADAMW_BLOCK, dtype=torch.float32, device=device)
                        for _ in range(2)))


def _check_state(state: AdamWState, device) -> int:
    """Blocks that the states hold."""
    if not isinstance(state, AdamWState):
        raise TypeError("state must be an AdamWState")
    m, v, ms, vs = state.m, state.v, state.m_scale, state.v_scale
    if isinstance(m, torch.Tensor):
        n = m.numel()
        blocks = n // QLORA_ADAMW_BLOCK
        if n % QLORA_ADAMW_BLOCK == 0 and (
                tensors().fits(device.index, "cbff", (m, v, ms, vs), ((n,), (n,), (blocks,), (blocks,)))
                if ms is not None else
                vs is None and tensors().fits(device.index, "ff", (m, v), ((n,), (n,)))):
            return blocks
    # what is wrong with it
    if not isinstance(m, torch.Tensor) or m.dim() != 1 or m.numel() % QLORA_ADAMW_BLOCK:
        raise ValueError(f"state.m must be a 1-D tensor of a multiple of {QLORA_ADAMW_BLOCK} elements")
    eight = m.dtype == torch.int8
    _same("state.m", m, m.shape, (torch.int8 if eight else torch.float32,), device)
    _same("state.v", v, m.shape, (torch.uint8 if eight else torch.float32,), device)
    blocks = m.numel() // QLORA_ADAMW_BLOCK
    if eight:
        _same("state.m_scale", ms, (blocks,), (torch.float32,), device)
        _same("state.v_scale", vs, (blocks,), (torch.float32,), device)
    elif ms is not None or vs is not None:
        raise ValueError("32-bit states have no scales")
    return blocks


def _scalar(name, x, dtype, device):
    """(host value, device address) of a number or a one-element tensor."""
    if not isinstance(x, torch.Tensor):
        return x, None
    if x.numel() != 1 or x.dtype != dtype or x.device != device:
        raise ValueError(f"{name} must be a number or a one-element {dtype} tensor on {device}")
    return 0, x.data_ptr()


def _passes(steps, grads, gptrs):
    """(step, addresses of the gradients that take part in it) of each number in
    `steps`, one per tensor.  All are checked before the first pass."""
    if len(steps) != len(grads):
        raise ValueError(f"{len(steps)} steps for {len(grads)} parameters")
    counts = {s for s, g in zip(steps, grads) if g is not None}
    if not all(isinstance(s, int) for s in counts):
        raise ValueError("steps must be whole numbers")
    if min(counts) < 1:
        raise ValueError(f"steps count from 1, one is {min(counts)}")
    if len(counts) == 1:
        return ((counts.pop(), gptrs),)
    return [(c, array.array("Q", [p if s == c else 0 for p, s in zip(gptrs, steps)]))
            for c in sorted(counts)]


def adamw_step(params, grads, state: AdamWState, step, lr, betas=(0.9, 0.999), eps: float = 1e-8,
               weight_decay: float = 0.01, norm: Optional[torch.Tensor] = None,
               max_norm: Optional[float] = None, copies=None, stream=None) -> None:
    """One AdamW step of all tensors in place:

        g = grad min(1, max_norm / (norm + 1e-6))      (norm given, else grad)
        m = b1 m + (1 - b1) g,  v = b2 v + (1 - b2) g^2
        p = p (1 - lr weight_decay) - lr m / (1 - b1^step) / (sqrt(v / (1 - b2^step)) + eps)

    params: contiguous bfloat16 or float32 tensors, each given once; grads: as
    many tensors of the same sizes, of either type (None: that tensor and its
    states are left alone); state: from adamw_init, updated.  step: the number
    of updates that the tensors have had, this one included; a list of as many
    numbers where they differ (tensors that had no gradient in some steps; one
    pass for each number).  norm: the one-element float32 device tensor of
    grad_norm, with max_norm (the gradients themselves stay as they are).
    copies: bfloat16 tensors (or None) that take the updated parameters,
    rounded: for parameters kept in float32 beside a bfloat16 copy.

    step and lr may be one-element device tensors (int64, float32), read when
    the kernels run: so a captured step can be replayed with new values."""
    params, grads = list(params), list(grads)
    n = len(params)
    if not n:
        raise ValueError("there are no parameters")
    if len(grads) != n:
        raise ValueError(f"{len(grads)} gradients for {n} parameters")
    dev, ptrs, sizes, types = _grad_arrays("params", params)
    if not tensors().distinct(_ptr_of(ptrs), n):
        given = [p.data_ptr() for p in params if p.numel()]
        if len(set(given)) != len(given):
            raise ValueError("a parameter is given twice")
    got = _describe(grads)
    if got is None:  # some are None, or not what they should be
        there = [g for g in grads if g is not None]
        if not there:
            return
        got = _grad_arrays("grads", there)
    gdev, gptrs, gsizes, gtypes = got
    if gdev != dev:
        raise ValueError(f"grads are on {gdev}, expected {dev}")
    some = None
    if len(gptrs) != n:
        at = [i for i, g in enumerate(grads) if g is not None]
        if [sizes[i] for i in at] != gsizes.tolist():
            raise ValueError("a gradient has another size than its parameter")
        some, gptrs = gptrs, array.array("Q", bytes(8 * n))
        stypes, gtypes = gtypes, array.array("i", bytes(4 * n))
        for i, p, t in zip(at, some, stypes):
            gptrs[i], gtypes[i] = p, t
    elif gsizes != sizes:
        raise ValueError("a gradient has another size than its parameter")
    blocks = _check_state(state, dev)
    cptrs = None
    if copies is not None:
        copies = list(copies)
        if len(copies) != n:
            raise ValueError(f"{len(copies)} copies for {n} parameters")
        got = _describe(copies)
        if (got is not None and got[0] == dev and got[3].count(QLORA_TYPE_BF16) == n and
                tensors().same_shapes(copies, params)):
            cptrs = got[1]
        else:
            for p, c in zip(params, copies):
                if c is not None:
                    _same("copy", c, p.shape, (torch.bfloat16,), dev)
            cptrs = array.array("Q", [0 if c is None else c.data_ptr() for c in copies])
    if (norm is None) != (max_norm is None):
        raise ValueError("norm and max_norm go together")
    if norm is not None:
        if not isinstance(norm, torch.Tensor):
            raise TypeError("norm must be a torch tensor")
        if norm.numel() != 1 or norm.dtype != torch.float32 or norm.device != dev:
            raise ValueError(f"norm must be a one-element float32 tensor on {dev}")
        if not max_norm >= 0.0:
            raise ValueError(f"max_norm must be at least 0, got {max_norm}")
    passes = _passes(step, grads, gptrs) if isinstance(step, (list, tuple)) else ((step, gptrs),)
    lr, lr_dev = _scalar("lr", lr, torch.float32, dev)
    L = lib()
    if L.qlora_adamw_blocks(n, _ptr_of(sizes)) > blocks:
        raise ValueError(f"state has {blocks} blocks, too few for these parameters")
    st, ctx = _on(dev, stream)
    eight = state.bits == 8
    with ctx:
        for step, gptrs in passes:
            step, step_dev = _scalar("step", step, torch.int64, dev)
            check(L.qlora_adamw_step(_Args(
                n, _ptr_of(ptrs), _ptr_of(gptrs), None if cptrs is None else _ptr_of(cptrs),
                _ptr_of(sizes), _ptr_of(types), _ptr_of(gtypes), state.m.data_ptr(),
                state.v.data_ptr(), state.m_scale.data_ptr() if eight else None,
                state.v_scale.data_ptr() if eight else None, blocks, int(step), float(lr),
                float(betas[0]), float(betas[1]), float(weight_decay), lr_dev, step_dev,
                None if norm is None else norm.data_ptr(), float(eps),
                0.0 if max_norm is None else float(max_norm), 8 if eight else 32), st),
                "qlora_adamw_step")
    for given in (params, copies):
        if given is not None:
            tensors().written(given if some is None else
                              [t for t, g in zip(given, grads) if g is not None])
    written(state.m, state.v, state.m_scale, state.v_scale)


def adamw_values(state: AdamWState, stream=None):
    """(m, v) in float32, laid out as the states: 32-bit states themselves, and
    new tensors of the values that 8-bit ones stand for."""
    dev = _device_of("state.m", state.m)
    blocks = _check_state(state, dev)
    if state.bits == 32:
        return state.m, state.v
    st, ctx = _on(dev, stream)
    with ctx:
        m, v = (torch.empty(state.m.numel(), dtype=torch.float32, device=dev) for _ in range(2))
        check(lib().qlora_adamw_values(state.m.data_ptr(), state.v.data_ptr(),
                                       state.m_scale.data_ptr(), state.v_scale.data_ptr(), blocks,
                                       m.data_ptr(), v.data_ptr(), st), "qlora_adamw_values")
    return m, v


class AdamW(torch.optim.Optimizer):
    """AdamW with states in 32 or 8 bits, one kernel pass per parameter group
    (and per number of updates, which each parameter counts for itself: one
    without a gradient is left alone), for parameters on one GPU.

    max_norm: the gradients of all groups are clipped by their global norm
    within the step (step() leaves them as they are; the norm before clipping
    is in `last_norm`).  masters: bfloat16 parameters are updated through
    float32 masters kept here, and take their rounded values; after parameters
    were changed in another way (a checkpoint loaded), call take_masters()."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 0.01, bits: int = 32, max_norm: Optional[float] = None,
                 masters: bool = False):
        if bits not in (8, 32):
            raise ValueError(f"bits must be 8 or 32, got {bits}")
        if max_norm is not None and not max_norm >= 0.0:
            raise ValueError(f"max_norm must be at least 0, got {max_norm}")
        for name, x in (("lr", lr), ("eps", eps), ("weight_decay", weight_decay)):
            if not (x >= 0.0 and math.isfinite(x)):
                raise ValueError(f"{name} must be at least 0 and finite, got {x}")
        if not all(0.0 <= b < 1.0 for b in betas):
            raise ValueError(f"betas must be at least 0 and below 1, got {betas}")
        self.bits, self.max_norm, self.use_masters = bits, max_norm, masters
        self.last_norm = None
        self._kept = []   # per group: its parameters' states, masters and numbers of updates
        super().__init__(params, dict(lr=lr, betas=tuple(betas), eps=eps, weight_decay=weight_decay))

    def add_param_group(self, group) -> None:
        super().add_param_group(group)
        ps = self.param_groups[-1]["params"]
        try:
            masters = [p.detach().float() if p.dtype == torch.bfloat16 else None for p in ps] \
                if self.use_masters else None
            # (a group without parameters has empty states)
            state = adamw_init(ps, self.bits, ps[0].device if ps else "cpu")
        except BaseException:   # no memory
            self.param_groups.pop()
            raise
        self._kept.append({"state": state, "masters": masters, "step": [0] * len(ps)})

    @torch.no_grad()
    def take_masters(self) -> None:
        """Set the masters to the parameters' present values."""
        for group, kept in zip(self.param_groups, self._kept):
            for p, m in zip(group["params"], kept["masters"] or ()):
                if m is not None:
                    m.copy_(p)

    def __getstate__(self):   # of copies and pickles
        own = {n: getattr(self, n) for n in ("bits", "max_norm", "use_masters", "last_norm", "_kept")}
        return {**super().__getstate__(), **own}

    def __setstate__(self, state):
        super().__setstate__(state)
        for k, g in zip(self._kept, self.param_groups):   # (one number per group before)
            if isinstance(k["step"], int):
                k["step"] = [k["step"]] * len(g["params"])

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        norm = None
        given = [[p.grad for p in g["params"]] for g in self.param_groups]
        if self.max_norm is not None:
            there = [g for grads in given for g in grads if g is not None]
            if there:
                norm = self.last_norm = grad_norm(there)
        for group, kept, grads in zip(self.param_groups, self._kept, given):
            ps = group["params"]
            have, counts = [g is not None for g in grads], kept["step"]
            if not any(have):
                continue
            if all(have) and counts.count(counts[0]) == len(counts):
                step = counts[0] + 1
                counts = [step] * len(counts)
            else:
                counts = [s + h for s, h in zip(counts, have)]
                told = {s for s, h in zip(counts, have) if h}
                step = counts if len(told) > 1 else told.pop()
            data, copies = [p.detach() for p in ps], None
            if kept["masters"] is not None:
                copies = [None if m is None else p for p, m in zip(data, kept["masters"])]
                data = [p if m is None else m for p, m in zip(data, kept["masters"])]
            adamw_step(data, grads, kept["state"], step, group["lr"], group["betas"],
                       group["eps"], group["weight_decay"], norm,
                       None if norm is None else self.max_norm, copies)
            kept["step"] = counts   # (a call that refuses has updated nothing)
        return loss

    def state_dict(self):
        """The groups' settings, and each group's states, masters and numbers of
        updates (tensors that later steps update: clone them to keep them), with
        the shapes of its parameters."""
        kept = []
        for k, g in zip(self._kept, self.param_groups):
            s = k["state"]
            kept.append({"m": s.m, "v": s.v, "m_scale": s.m_scale, "v_scale": s.v_scale,
                         "masters": k["masters"], "step": list(k["step"]),
                         "shapes": [tuple(p.shape) for p in g["params"]]})
        groups = [{n: v for n, v in g.items() if n != "params"} for g in self.param_groups]
        return {"bits": self.bits, "groups": groups, "kept": kept}

    @torch.no_grad()
    def load_state_dict(self, d) -> None:
        """States of the same parameters in the same order and groups."""
        if (d["bits"] != self.bits or len(d["kept"]) != len(self._kept) or
                len(d["groups"]) != len(self.param_groups)):
            raise ValueError("the states are of other bits or groups")
        pairs, steps = [], []
        for k, g, new in zip(self._kept, self.param_groups, d["kept"]):
            s = k["state"]
            # (states of 256-element blocks alone do not tell whose they are)
            shapes = [tuple(p.shape) for p in g["params"]]
            if [tuple(x) for x in new.get("shapes", shapes)] != shapes:
                raise ValueError("the states are of other parameters")
            here = [s.m, s.v, s.m_scale, s.v_scale, *(k["masters"] or [])]
            there = [new["m"], new["v"], new["m_scale"], new["v_scale"], *(new["masters"] or [])]
            if len(here) != len(there) or any(
                    (a is None) != (b is None) or
                    (a is not None and (a.shape != b.shape or a.dtype != b.dtype))
                    for a, b in zip(here, there)):
                raise ValueError("the states are of other parameters")
            pairs += [(a, b) for a, b in zip(here, there) if a is not None]
            # (one number for the whole group: as it was counted before)
            count, n = new["step"], len(k["step"])
            steps.append([int(count)] * n if isinstance(count, int) else list(map(int, count)))
            if len(steps[-1]) != n:
                raise ValueError("the states are of other parameters")
        for a, b in pairs:
            a.copy_(b)
        for k, g, step, settings in zip(self._kept, self.param_groups, steps, d["groups"]):
            k["step"] = step
            g.update(settings)
