"""Thin torch binding of the operators around the layer: attention, layer and
root-mean-square norms, and the clipping of gradients by their global norm.

As in :mod:`quantized_base_lora_nf4_amd.ops`: argument checks and marshalling
only, every call enqueues on ``torch.cuda.current_stream()`` of the tensors'
device unless a stream is passed, buffers allocated here are allocated on
that stream, and all arithmetic happens in the HIP kernels.
"""

import array
import contextlib
import itertools
import math
import operator
from typing import Optional

import torch
from torch.autograd.function import once_differentiable

from ._lib import QLORA_TYPE_BF16, QLORA_TYPE_FP32, Attention, check, lib
from .ops import _stream_obj

_SIXTEEN = (torch.bfloat16, torch.int16, torch.uint16)
_TYPES = {torch.bfloat16: QLORA_TYPE_BF16, torch.float32: QLORA_TYPE_FP32}
_HERE = contextlib.nullcontext()


def _on(device: torch.device, stream):
    """(stream handle, context to allocate and launch in) for tensors on
    `device`: the given stream, or the device's current one."""
    if stream is None:
        i = device.index
        return (torch._C._cuda_getCurrentRawStream(i),
                _HERE if i == torch.cuda.current_device() else torch.cuda.device(device))
    st = _stream_obj(stream)
    return st.cuda_stream, torch.cuda.stream(st)


def _device_of(name: str, t: torch.Tensor) -> torch.device:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} is on {t.device}, expected a GPU")
    return t.device


def _same(name: str, t, shape, dtypes, device) -> None:
    """Shape, dtype, device and layout of one contiguous tensor."""
    if (isinstance(t, torch.Tensor) and t.shape == shape and t.dtype in dtypes and
            t.device == device and t.is_contiguous()):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {' or '.join(map(str, dtypes))}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _bytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _floats(shape, device) -> torch.Tensor:
    """An uninitialized float32 tensor (sizes given one by one: torch takes
    twice as long over a tuple)."""
    if shape:
        return torch.empty(*shape, dtype=torch.float32, device=device)
    return torch.empty((), dtype=torch.float32, device=device)


def _scratch(nbytes: int, device, ws: Optional[torch.Tensor]) -> torch.Tensor:
    if ws is not None:
        if ws.device != device or not ws.is_contiguous():
            raise ValueError("ws must be a contiguous tensor on the operands' GPU")
        if _bytes(ws) >= nbytes:
            return ws
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------

def _heads(name, t, shape, device, packed) -> tuple:
    """(address, batch, row and head stride), as qlora_heads_t, of one
    [batch, row, head, dim] (packed: [row, head, dim]) tensor of any strides
    that the kernels take."""
    if isinstance(t, torch.Tensor) and t.shape == shape and t.device == device:
        st = t.stride()
        if t.dtype in _SIXTEEN and st[-1] == 1 and not (st[-2] | st[-3] | st[0]) & 7:
            return (t.data_ptr(), 0 if packed else st[0], st[-3], st[-2])
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype not in _SIXTEEN:
        raise TypeError(f"{name} must be bf16 (or its 16-bit view), got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.numel() == 0:
        return (0, 0, 0, 0)
    # the stride of a dimension of size 1 says nothing
    st = [0 if n == 1 else s for n, s in zip(shape, t.stride()[:-1])]
    if (t.stride()[-1] != 1 and shape[-1] != 1) or any(s % 8 for s in st):
        raise ValueError(f"{name} needs contiguous head vectors and strides of a multiple of 8, "
                         f"has {t.stride()}")
    return (t.data_ptr(), 0 if packed else st[0], st[-2], st[-1])


class _AttnCall:
    """Checked arguments of an attention call."""

    def __init__(self, q, k, v, causal, scale, cu_seqlens, cu_seqlens_k):
        self.dev = dev = _device_of("q", q)
        self.packed = packed = cu_seqlens is not None
        if not packed and cu_seqlens_k is not None:
            raise ValueError("cu_seqlens_k needs cu_seqlens")
        nd = 3 if packed else 4
        for name, t in (("q", q), ("k", k)):
            if not isinstance(t, torch.Tensor) or t.dim() != nd:
                raise ValueError(f"{name} must have {nd} dimensions "
                                 f"({'[row, head, dim]' if packed else '[batch, row, head, dim]'})")
        self.q_shape = qs = q.shape
        ks = k.shape
        h, d = qs[-2], qs[-1]
        hk = ks[-2]
        if h < 1 or hk < 1 or h % hk:
            raise ValueError(f"{h} query heads cannot share {hk} key/value heads")
        cq = ck = None
        if packed:
            self.k_shape = (ks[0], hk, d)
            if cu_seqlens_k is None:
                cu_seqlens_k = cu_seqlens
                if ks[0] != qs[0]:
                    raise ValueError("q and k have different rows: cu_seqlens_k is needed")
            for name, c in (("cu_seqlens", cu_seqlens), ("cu_seqlens_k", cu_seqlens_k)):
                if not isinstance(c, torch.Tensor) or c.dim() != 1 or c.numel() < 1:
                    raise ValueError(f"{name} must be a 1-D tensor of offsets")
                _same(name, c, cu_seqlens.shape, (torch.int32,), dev)
            cq, ck = cu_seqlens.data_ptr(), cu_seqlens_k.data_ptr()
            n = cu_seqlens.numel() - 1
            self.lse_shape = (h, qs[0])
        else:
            n = qs[0]
            self.k_shape = (n, ks[1], hk, d)
            self.lse_shape = (n, h, qs[1])
        if scale is None:
            scale = 1.0 / math.sqrt(d) if d else 1.0
        self.c = Attention(n, qs[-3], ks[-3], cq, ck, h, hk, d, int(causal), float(scale))
        self.q_rhd = (qs[-3], h, d)
        # the tensors' descriptions, one after the other
        self.words = [*_heads("q", q, qs, dev, packed), *_heads("k", k, self.k_shape, dev, packed),
                      *_heads("v", v, self.k_shape, dev, packed)]

    def add(self, name, t, keys: bool) -> None:
        """One more tensor of the queries' or keys' shape."""
        self.words += _heads(name, t, self.k_shape if keys else self.q_shape, self.dev, self.packed)

    def new(self, like, keys: bool) -> torch.Tensor:
        """A new tensor of the queries' or keys' shape, added."""
        t = torch.empty_like(like, dtype=torch.bfloat16, memory_format=torch.contiguous_format)
        rows, h, d = self.k_shape[-3:] if keys else self.q_rhd
        self.words += (t.data_ptr(), 0 if self.packed else rows * h * d, h * d, d)
        return t

    def views(self):
        """The addresses of the tensors' descriptions, in the order added."""
        self.array = array.array("q", self.words)
        base = self.array.buffer_info()[0]
        return range(base, base + 8 * len(self.words), 32)


def attention_fwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, causal: bool = True,
                  scale: Optional[float] = None, cu_seqlens: Optional[torch.Tensor] = None,
                  cu_seqlens_k: Optional[torch.Tensor] = None,
                  out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                  stream=None):
    """softmax(scale q k^T) v per head, and the rows' log-sum-exp (fp32).

    Dense: q [B, Sq, H, D], k and v [B, Sk, Hkv, D]; returns out like q and
    lse [B, H, Sq].  Packed: q [T, H, D], k and v [Tk, Hkv, D] with the
    sequences' offsets as an int32 device tensor `cu_seqlens` (and
    `cu_seqlens_k` if the keys have their own); lse [H, T].  bf16; H a
    multiple of Hkv; D a multiple of 8 up to 128; views with strides of a
    multiple of 8 are taken as they are.  Causal: the last query of a sequence
    sees its last key.  A query that sees no key gets 0 and an lse of -inf.
    scale defaults to 1 / sqrt(D) (2^-100 to 2^100).  `out` takes the output: rows that lie apart,
    overlapping no input, or q itself."""
    c = _AttnCall(q, k, v, causal, scale, cu_seqlens, cu_seqlens_k)
    st, ctx = _on(c.dev, stream)
    with ctx:
        if out is None:
            out = c.new(q, False)
        else:
            c.add("out", out, False)
        lse = _floats(c.lse_shape, c.dev)
        L = lib()
        need = L.qlora_attention_fwd_workspace_size(c.c)
        ws = _scratch(need, c.dev, ws) if need else None
        check(L.qlora_attention_fwd(c.c, *c.views(), lse.data_ptr(),
                                    None if ws is None else ws.data_ptr(), _bytes(ws), st),
              "qlora_attention_fwd")
    return out, lse


def attention_bwd(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor,
                  lse: torch.Tensor, do: torch.Tensor, causal: bool = True,
                  scale: Optional[float] = None, cu_seqlens: Optional[torch.Tensor] = None,
                  cu_seqlens_k: Optional[torch.Tensor] = None, out: Optional[tuple] = None,
                  ws: Optional[torch.Tensor] = None, stream=None):
    """(dq, dk, dv) for the output gradient `do`, with o and lse as
    attention_fwd returned them; the other arguments as there.  `out`: the
    three tensors to write, of rows that lie apart; they overlap neither each
    other nor an input, but dq may be o itself, dk k and dv v."""
    c = _AttnCall(q, k, v, causal, scale, cu_seqlens, cu_seqlens_k)
    _same("lse", lse, c.lse_shape, (torch.float32,), c.dev)
    c.add("o", o, False)
    c.add("do", do, False)
    st, ctx = _on(c.dev, stream)
    with ctx:
        if out is None:
            dq, dk, dv = c.new(q, False), c.new(k, True), c.new(k, True)
        else:
            dq, dk, dv = out
            c.add("dq", dq, False)
            c.add("dk", dk, True)
            c.add("dv", dv, True)
        L = lib()
        ws = _scratch(L.qlora_attention_bwd_workspace_size(c.c), c.dev, ws)
        w = c.views()
        check(L.qlora_attention_bwd(c.c, *w[:4], lse.data_ptr(), *w[4:], ws.data_ptr(),
                                    _bytes(ws), st), "qlora_attention_bwd")
    return dq, dk, dv


def _takeable(t: torch.Tensor) -> torch.Tensor:
    """t, or a copy if its strides are not ones the kernels take."""
    st = t.stride()
    ok = st[-1] == 1 and all(s % 8 == 0 for s in st[:-1]) and t.data_ptr() % 16 == 0
    return t if ok else t.clone(memory_format=torch.contiguous_format)


class _AttentionFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal, scale, cu_seqlens, cu_seqlens_k):
        o, lse = attention_fwd(q, k, v, causal, scale, cu_seqlens, cu_seqlens_k)
        ctx.save_for_backward(q, k, v, o, lse, cu_seqlens, cu_seqlens_k)
        ctx.how = causal, scale
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        q, k, v, o, lse, cu_seqlens, cu_seqlens_k = ctx.saved_tensors
        grads = attention_bwd(q, k, v, o, lse, _takeable(do), *ctx.how, cu_seqlens, cu_seqlens_k)
        return (*grads, None, None, None, None)


def attention(q, k, v, causal: bool = True, scale: Optional[float] = None, cu_seqlens=None,
              cu_seqlens_k=None) -> torch.Tensor:
    """attention_fwd with gradients for q, k and v (torch autograd); returns
    the output only."""
    return _AttentionFunction.apply(q, k, v, causal, scale, cu_seqlens, cu_seqlens_k)


# ---------------------------------------------------------------------------
# Norms
# ---------------------------------------------------------------------------

def _check_norm(x, weight):
    """(device, rows, width) of the rows of x, with the weight checked."""
    dev = _device_of("x", x)
    shape = x.shape
    if not shape:
        raise ValueError("x must have at least 1 dimension")
    if x.dtype not in _TYPES:
        raise TypeError(f"x must be bfloat16 or float32, got {x.dtype}")
    if not x.is_contiguous():
        raise ValueError("x must be contiguous")
    width = shape[-1]
    _same("weight", weight, (width,), _TYPES, dev)
    return dev, x.numel() // width if width else 0, width


def norm_fwd(x: torch.Tensor, weight: torch.Tensor, bias: Optional[torch.Tensor] = None,
             eps: float = 1e-5, rms: bool = False, out: Optional[torch.Tensor] = None,
             stream=None):
    """Layer norm (or, with `rms`, root-mean-square norm) over the last
    dimension of x: y = (x - mean) rstd weight + bias.

    x and y are bfloat16 or float32, weight and bias either (of one type);
    mean and rstd are float32, one per row, and mean is None with `rms`.
    Returns (y, mean, rstd)."""
    dev, rows, width = _check_norm(x, weight)
    if bias is not None:
        _same("bias", bias, weight.shape, (weight.dtype,), dev)
    if out is not None:
        _same("out", out, x.shape, (x.dtype,), dev)
    st, ctx = _on(dev, stream)
    with ctx:
        if out is None:
            out = torch.empty_like(x)
        lead = x.shape[:-1]
        mean = None if rms else _floats(lead, dev)
        rstd = _floats(lead, dev)
        check(lib().qlora_norm_fwd(x.data_ptr(), rows, width, _TYPES[x.dtype], weight.data_ptr(),
                                   None if bias is None else bias.data_ptr(),
                                   _TYPES[weight.dtype], float(eps), int(rms), out.data_ptr(),
                                   None if rms else mean.data_ptr(), rstd.data_ptr(), st),
              "qlora_norm_fwd")
    return out, mean, rstd


def norm_bwd(dy: torch.Tensor, x: torch.Tensor, weight: torch.Tensor,
             mean: Optional[torch.Tensor], rstd: torch.Tensor, rms: bool = False,
             need_dx: bool = True, need_dw: bool = True, need_db: Optional[bool] = None,
             ws: Optional[torch.Tensor] = None, stream=None):
    """(dx, dweight, dbias) of norm_fwd for the output gradient dy, from its
    mean and rstd.  dbias is computed without `rms` unless need_db says
    otherwise; what is not computed is None."""
    dev, rows, width = _check_norm(x, weight)
    lead = x.shape[:-1]
    _same("dy", dy, x.shape, (x.dtype,), dev)
    _same("rstd", rstd, lead, (torch.float32,), dev)
    if not rms:
        if mean is None:
            raise ValueError("mean is needed without rms")
        _same("mean", mean, lead, (torch.float32,), dev)
    if need_db is None:
        need_db = not rms
    st, ctx = _on(dev, stream)
    with ctx:
        dx = torch.empty_like(x) if need_dx else None
        dw = torch.empty_like(weight) if need_dw else None
        db = torch.empty_like(weight) if need_db else None
        L = lib()
        if need_dw or need_db:
            need = int(L.qlora_norm_bwd_workspace_size(rows, width, _TYPES[x.dtype]))
            ws = _scratch(need, dev, ws)
        else:
            ws = None   # not used
        check(L.qlora_norm_bwd(dy.data_ptr(), x.data_ptr(), rows, width, _TYPES[x.dtype],
                               weight.data_ptr(), _TYPES[weight.dtype], int(rms),
                               None if rms else mean.data_ptr(), rstd.data_ptr(),
                               *(None if t is None else t.data_ptr() for t in (dx, dw, db)),
                               None if ws is None else ws.data_ptr(), _bytes(ws), st),
              "qlora_norm_bwd")
    return dx, dw, db


class _NormFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, rms):
        x = x.contiguous()
        y, mean, rstd = norm_fwd(x, weight, bias, eps, rms)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.rms = rms
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        need = ctx.needs_input_grad
        grads = norm_bwd(dy.contiguous(), x, weight, mean, rstd, ctx.rms, need_dx=need[0],
                         need_dw=need[1], need_db=need[2])
        return (*grads, None, None)


def norm(x, weight, bias=None, eps: float = 1e-5, rms: bool = False) -> torch.Tensor:
    """norm_fwd with gradients for x, weight and bias (torch autograd);
    returns y only."""
    return _NormFunction.apply(x, weight, bias, eps, rms)


class LayerNorm(torch.nn.Module):
    """Layer norm over the last dimension, with weight and bias."""

    def __init__(self, width: int, eps: float = 1e-5, device="cuda", dtype=torch.float32):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(width, device=device, dtype=dtype))
        self.bias = torch.nn.Parameter(torch.zeros(width, device=device, dtype=dtype))

    def forward(self, x):
        return norm(x, self.weight, self.bias, self.eps)


class RMSNorm(torch.nn.Module):
    """Root-mean-square norm over the last dimension, with a weight."""

    def __init__(self, width: int, eps: float = 1e-5, device="cuda", dtype=torch.float32):
        super().__init__()
        self.eps = eps
        self.weight = torch.nn.Parameter(torch.ones(width, device=device, dtype=dtype))

    def forward(self, x):
        return norm(x, self.weight, None, self.eps, rms=True)


# ---------------------------------------------------------------------------
# Gradient norm and clipping
# ---------------------------------------------------------------------------

_dtype_of = operator.attrgetter("dtype")


def _grad_arrays(name: str, grads):
    """(device, addresses, sizes, types) of a list of gradients."""
    if not isinstance(grads[0], torch.Tensor):
        raise TypeError(f"{name} must all be torch tensors")
    dev = _device_of(f"{name}[0]", grads[0])
    try:
        devices = set(map(torch.Tensor.get_device, grads))
    except TypeError:
        raise TypeError(f"{name} must all be torch tensors") from None
    if devices != {dev.index}:
        other = max(devices - {dev.index})
        raise ValueError(f"{name} are on {dev} and {f'cuda:{other}' if other >= 0 else 'cpu'}, "
                         "expected one GPU")
    dtypes = set(map(_dtype_of, grads))
    for dt in dtypes:
        if dt not in _TYPES:
            raise TypeError(f"{name} must be bfloat16 or float32, one is {dt}")
    if not all(map(torch.Tensor.is_contiguous, grads)):
        raise ValueError(f"{name} must be contiguous")
    types = ([_TYPES[dtypes.pop()]] * len(grads) if len(dtypes) == 1 else
             [_TYPES[t.dtype] for t in grads])
    return (dev, array.array("Q", map(torch.Tensor.data_ptr, grads)),
            array.array("q", map(torch.Tensor.numel, grads)), array.array("i", types))


def _ptr_of(a: "array.array") -> int:
    return a.buffer_info()[0]


def _clip_call(grads, max_norm, out, ws, stream):
    grads = [grads] if isinstance(grads, torch.Tensor) else [g for g in grads if g is not None]
    if max_norm is not None and not max_norm >= 0.0:
        raise ValueError(f"max_norm must be at least 0, got {max_norm}")
    if not grads:
        raise ValueError("there are no gradients")
    dev, ptrs, sizes, types = _grad_arrays("gradients", grads)
    n, outs = len(grads), None
    if isinstance(out, torch.Tensor):
        dt = grads[0].dtype
        if out.dtype != dt or types.count(types[0]) != n:
            raise TypeError("a flat out takes gradients of its own dtype only")
        _same("out", out, (sum(sizes),), (dt,), dev)
        step = out.element_size()
        outs = array.array("Q", itertools.accumulate(map(step.__mul__, sizes),
                                                     initial=out.data_ptr()))
    elif out is not None:
        out = list(out)
        if len(out) != n:
            raise ValueError(f"out has {len(out)} tensors for {n} gradients")
        for g, o in zip(grads, out):
            _same("out", o, g.shape, (g.dtype,), dev)
        outs = array.array("Q", [o.data_ptr() for o in out])
    st, ctx = _on(dev, stream)
    with ctx:
        norm_out = torch.empty(1, dtype=torch.float32, device=dev)
        L = lib()
        ws = _scratch(int(L.qlora_clip_workspace_size(n)), dev, ws)
        if max_norm is None:
            check(L.qlora_grad_norm(n, _ptr_of(ptrs), _ptr_of(sizes), _ptr_of(types),
                                    norm_out.data_ptr(), ws.data_ptr(), _bytes(ws), st),
                  "qlora_grad_norm")
        else:
            check(L.qlora_clip_grad_norm(n, _ptr_of(ptrs), _ptr_of(sizes), _ptr_of(types),
                                         max_norm, None if outs is None else _ptr_of(outs),
                                         norm_out.data_ptr(), ws.data_ptr(), _bytes(ws), st),
                  "qlora_clip_grad_norm")
    return norm_out


def grad_norm(grads, ws: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The 2-norm of all gradients together (a one-element float32 device
    tensor, written on the stream).  grads: contiguous bfloat16 or float32
    tensors, in any mixture; None entries are left out."""
    return _clip_call(grads, None, None, ws, stream)


def clip_grad_norm(grads, max_norm: float, out=None, ws: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Scale the gradients by min(1, max_norm / (norm + 1e-6)) and return
    their norm before that (a one-element float32 device tensor).  A max_norm
    of infinity leaves them as they are, unless the norm is NaN.

    Each gradient is given once.  out: None scales in place; a list of tensors (one per gradient that is
    not None, same shape and dtype) takes the scaled gradients instead, and
    so does one flat tensor of their dtype, one gradient after the other."""
    return _clip_call(grads, float(max_norm), out, ws, stream)
