"""Refusals of the operators around the layer, on the CPU: the torch binding
rejects wrong shapes, types, devices and layouts, and the C ABI rejects bad
sizes, strides, alignments and workspaces, before anything is launched."""

import ctypes
import math
import re
import subprocess

import pytest
import torch

import quantized_base_lora_nf4_amd as qn
from quantized_base_lora_nf4_amd import _lib
from quantized_base_lora_nf4_amd._lib import Attention, Heads

INVALID, UNSUPPORTED, WORKSPACE = (_lib.QLORA_ERR_INVALID, _lib.QLORA_ERR_UNSUPPORTED,
                                   _lib.QLORA_ERR_WORKSPACE)


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


# ---- binding ----

def test_attention_rejects_host_tensors():
    with pytest.raises(ValueError, match="q is on cpu"):
        qn.attention_fwd(_bf(1, 4, 2, 64), _bf(1, 4, 2, 64), _bf(1, 4, 2, 64))
    with pytest.raises(TypeError, match="q must be a torch tensor"):
        qn.attention_fwd(None, _bf(1, 4, 2, 64), _bf(1, 4, 2, 64))


def test_norms_reject_host_tensors():
    with pytest.raises(ValueError, match="x is on cpu"):
        qn.norm_fwd(_bf(3, 8), _bf(8))
    with pytest.raises(ValueError, match="x is on cpu"):
        qn.norm_bwd(_bf(3, 8), _bf(3, 8), _bf(8), torch.zeros(3), torch.zeros(3))


def test_clip_rejects_what_is_not_a_list_of_device_gradients():
    with pytest.raises(ValueError, match="is on cpu"):
        qn.clip_grad_norm([_bf(4)], 1.0)
    with pytest.raises(ValueError, match="no gradients"):
        qn.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError, match="no gradients"):
        qn.grad_norm([None])
    with pytest.raises(TypeError, match="torch tensors"):
        qn.clip_grad_norm([1.0], 1.0)
    for bad in (-1.0, float("nan")):
        with pytest.raises(ValueError, match="max_norm"):
            qn.clip_grad_norm([_bf(4)], bad)


@pytest.mark.gpu
def test_binding_checks_on_device_tensors():
    def bf(*s):
        return _bf(*s).cuda()
    q, k = bf(2, 6, 4, 64), bf(2, 5, 2, 64)
    with pytest.raises(ValueError, match="v has shape"):
        qn.attention_fwd(q, k, bf(2, 5, 1, 64))
    with pytest.raises(ValueError, match="k has shape"):
        qn.attention_fwd(q, bf(1, 5, 2, 64), bf(1, 5, 2, 64))
    with pytest.raises(ValueError, match="k has shape"):
        qn.attention_fwd(q, bf(2, 5, 2, 32), bf(2, 5, 2, 32))
    with pytest.raises(ValueError, match="cannot share"):
        qn.attention_fwd(q, bf(2, 5, 3, 64), bf(2, 5, 3, 64))
    with pytest.raises(ValueError, match="dimensions"):
        qn.attention_fwd(q[0], k, k)
    with pytest.raises(TypeError, match="k must be bf16"):
        qn.attention_fwd(q, k.float(), k)
    with pytest.raises(ValueError, match="strides"):
        qn.attention_fwd(q.transpose(2, 3).contiguous().transpose(2, 3), k, k)
    with pytest.raises(ValueError, match="strides"):
        qn.attention_fwd(bf(2, 6, 4, 68)[..., :64], k, k)
    with pytest.raises(ValueError, match="out has shape"):
        qn.attention_fwd(q, k, k, out=k)
    with pytest.raises(ValueError, match="needs cu_seqlens"):
        qn.attention_fwd(q, k, k, cu_seqlens_k=torch.zeros(2, dtype=torch.int32, device="cuda"))
    cu = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="different rows"):
        qn.attention_fwd(q[0], k[0], k[0], cu_seqlens=cu)
    with pytest.raises(TypeError, match="cu_seqlens has dtype"):
        qn.attention_fwd(q[0], q[0], q[0], cu_seqlens=cu.long())
    with pytest.raises(ValueError, match="cu_seqlens is on"):
        qn.attention_fwd(q[0], q[0], q[0], cu_seqlens=cu.cpu())
    with pytest.raises(ValueError, match="cu_seqlens_k has shape"):
        qn.attention_fwd(q[0], q[0], q[0], cu_seqlens=cu, cu_seqlens_k=cu[:1])
    o, lse = qn.attention_fwd(q, k, k)
    with pytest.raises(ValueError, match="lse has shape"):
        qn.attention_bwd(q, k, k, o, lse[:1], o)
    with pytest.raises(ValueError, match="do has shape"):
        qn.attention_bwd(q, k, k, o, lse, k)
    with pytest.raises(qn.QloraError, match="invalid"):
        qn.attention_fwd(q, k, k, scale=-1.0)
    with pytest.raises(qn.QloraError, match="unsupported"):
        qn.attention_fwd(bf(1, 4, 1, 136), bf(1, 4, 1, 136), bf(1, 4, 1, 136))
    flat = bf(6 * 4 * 64 + 8)
    with pytest.raises(qn.QloraError, match="invalid"):   # 2 bytes off
        qn.attention_fwd(flat[1:1 + 6 * 4 * 64].view(1, 6, 4, 64), k[:1], k[:1])

    x, w = bf(3, 40), bf(40)
    with pytest.raises(ValueError, match="weight has shape"):
        qn.norm_fwd(x, bf(41))
    with pytest.raises(TypeError, match="x must be bfloat16 or float32"):
        qn.norm_fwd(x.half(), w)
    with pytest.raises(TypeError, match="bias has dtype"):
        qn.norm_fwd(x, w, w.float())
    with pytest.raises(ValueError, match="contiguous"):
        qn.norm_fwd(x.t().contiguous().t(), w)
    with pytest.raises(qn.QloraError, match="invalid"):
        qn.norm_fwd(x, w, eps=-1.0)
    with pytest.raises(qn.QloraError, match="unsupported"):
        qn.norm_fwd(torch.zeros(1, 32769, device="cuda"), torch.zeros(32769, device="cuda"))
    _, mean, rstd = qn.norm_fwd(x, w)
    with pytest.raises(ValueError, match="mean"):
        qn.norm_bwd(x, x, w, None, rstd)
    with pytest.raises(ValueError, match="dy has shape"):
        qn.norm_bwd(x[:2], x, w, mean, rstd)

    with pytest.raises(TypeError, match="bfloat16 or float32"):
        qn.clip_grad_norm([x.half()], 1.0)
    with pytest.raises(ValueError, match="contiguous"):
        qn.clip_grad_norm([x.t()], 1.0)
    with pytest.raises(ValueError, match="expected one GPU"):
        qn.clip_grad_norm([x, _bf(3)], 1.0)
    with pytest.raises(ValueError, match="out has shape"):
        qn.clip_grad_norm([x], 1.0, out=bf(119))
    with pytest.raises(ValueError, match="out has 2"):
        qn.clip_grad_norm([x], 1.0, out=[x, x])
    with pytest.raises(TypeError, match="out has dtype"):
        qn.clip_grad_norm([x], 1.0, out=[x.float()])
    with pytest.raises(TypeError, match="flat out"):
        qn.clip_grad_norm([x, x.float()], 1.0, out=bf(240))


# ---- C ABI ----
# Addresses that are never followed: every call below fails its checks.
P = 1 << 20


def _attn(**kw):
    a = dict(n_seq=2, q_rows=10, k_rows=12, cu_seqlens_q=None, cu_seqlens_k=None, heads=4,
             kv_heads=2, head_dim=64, causal=1, scale=0.125)
    a.update(kw)
    return Attention(*a.values())


def _view(**kw):
    v = dict(data=P, batch_stride=640, row_stride=64, head_stride=8)
    v.update(kw)
    return ctypes.byref(Heads(*v.values()))


def _fwd(a, q=None, k=None, v=None, o=None, lse=P):
    vs = [x if x is not None else _view() for x in (q, k, v, o)]
    return _lib.lib().qlora_attention_fwd(a, *vs, lse, P, 1 << 30, None)


@pytest.mark.parametrize("bad", [
    dict(n_seq=-1), dict(q_rows=-1), dict(k_rows=-1), dict(q_rows=1 << 30), dict(k_rows=1 << 30),
    dict(heads=0), dict(kv_heads=0), dict(kv_heads=3), dict(head_dim=0), dict(scale=0.0),
    dict(scale=-1.0), dict(scale=math.inf), dict(scale=math.nan), dict(cu_seqlens_q=P),
    dict(cu_seqlens_k=P), dict(cu_seqlens_q=P + 2, cu_seqlens_k=P), dict(n_seq=1 << 30),
    dict(heads=1 << 30, q_rows=1000)], ids=str)
def test_attention_abi_rejects_bad_sizes(bad):
    assert _fwd(_attn(**bad)) == INVALID
    assert _lib.lib().qlora_attention_fwd_workspace_size(_attn(**bad)) == 0
    assert _lib.lib().qlora_attention_bwd_workspace_size(_attn(**bad)) == 0


@pytest.mark.parametrize("dim", [4, 63, 132, 136, 256])
def test_attention_abi_rejects_unsupported_dims(dim):
    assert _fwd(_attn(head_dim=dim)) == UNSUPPORTED


@pytest.mark.parametrize("bad", [
    dict(data=None), dict(data=P + 8), dict(row_stride=60), dict(row_stride=-64),
    dict(row_stride=(1 << 22) + 8), dict(head_stride=4), dict(head_stride=-8),
    dict(batch_stride=-8), dict(batch_stride=1)], ids=str)
def test_attention_abi_rejects_bad_views(bad):
    for name in "qkvo":
        assert _fwd(_attn(), **{name: _view(**bad)}) == INVALID
    L = _lib.lib()
    for i in range(8):
        vs = [_view() for _ in range(8)]
        vs[i] = _view(**bad)
        q, k, v, o, do, dq, dk, dv = vs
        assert L.qlora_attention_bwd(_attn(), q, k, v, o, P, do, dq, dk, dv, P, 1 << 20,
                                     None) == INVALID


def test_attention_abi_rejects_missing_statistics_and_small_workspaces():
    L = _lib.lib()
    assert _fwd(_attn(), lse=None) == INVALID and _fwd(_attn(), lse=P + 2) == INVALID
    vs = [_view() for _ in range(8)]
    need = L.qlora_attention_bwd_workspace_size(_attn())
    assert need >= 2 * 4 * 10 * 4

    def bwd(lse=P, ws=P, nbytes=need):
        return L.qlora_attention_bwd(_attn(), *vs[:4], lse, *vs[4:], ws, nbytes, None)
    assert bwd(lse=None) == INVALID and bwd(ws=None) == INVALID and bwd(ws=P + 4) == INVALID
    assert bwd(nbytes=need - 1) == WORKSPACE
    assert L.qlora_attention_fwd(None, *vs[:4], P, P, 0, None) == INVALID
    few = _attn(n_seq=1, q_rows=1, k_rows=1 << 16)   # one query, many keys: split
    need = L.qlora_attention_fwd_workspace_size(few)
    assert need > 0
    assert L.qlora_attention_fwd(few, *vs[:4], P, P, need - 1, None) == WORKSPACE
    assert L.qlora_attention_fwd(few, *vs[:4], P, None, need, None) == INVALID
    assert L.qlora_attention_fwd(few, *vs[:4], P, P + 8, need, None) == INVALID


def test_attention_abi_with_no_queries_does_nothing():
    assert _fwd(_attn(q_rows=0), q=_view(data=None), o=_view(data=None), lse=None) == 0
    assert _fwd(_attn(n_seq=0), *[_view(data=None)] * 4, lse=None) == 0


def test_norm_abi_refusals():
    L = _lib.lib()

    def fwd(x=P, rows=4, width=10, xt=0, w=P, b=P, wt=0, eps=1e-5, rms=0, y=P, mean=P, rstd=P):
        return L.qlora_norm_fwd(x, rows, width, xt, w, b, wt, eps, rms, y, mean, rstd, None)
    for bad in (dict(x=None), dict(rows=-1), dict(rows=1 << 30), dict(width=0), dict(w=None),
                dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf), dict(y=None),
                dict(mean=None), dict(rstd=None), dict(x=P + 1), dict(y=P + 1), dict(w=P + 1),
                dict(b=P + 1), dict(xt=1, x=P + 2), dict(wt=1, w=P + 2), dict(mean=P + 2),
                dict(rstd=P + 2)):
        assert fwd(**bad) == INVALID, bad
    for bad in (dict(xt=2), dict(wt=-1), dict(width=65537), dict(xt=1, width=32769)):
        assert fwd(**bad) == UNSUPPORTED, bad
    assert fwd(rows=0, x=None, y=None, mean=None, rstd=None) == 0

    need = L.qlora_norm_bwd_workspace_size(4, 10, 0)
    assert need >= 10 * 8
    assert L.qlora_norm_bwd_workspace_size(0, 10, 0) == 0
    assert L.qlora_norm_bwd_workspace_size(4, 0, 0) == L.qlora_norm_bwd_workspace_size(4, 8, 2) == 0

    def bwd(dy=P, x=P, rows=4, width=10, xt=0, w=P, wt=0, rms=0, mean=P, rstd=P, dx=P, dw=P, db=P,
            ws=P, nbytes=need):
        return L.qlora_norm_bwd(dy, x, rows, width, xt, w, wt, rms, mean, rstd, dx, dw, db, ws,
                                nbytes, None)
    for bad in (dict(dy=None), dict(x=None), dict(w=None), dict(mean=None), dict(rstd=None),
                dict(ws=None), dict(ws=P + 8), dict(dx=P + 1), dict(dw=P + 1), dict(db=P + 1),
                dict(dy=P + 1), dict(rows=-1), dict(width=0)):
        assert bwd(**bad) == INVALID, bad
    for bad in (dict(xt=3), dict(wt=3), dict(width=65537)):
        assert bwd(**bad) == UNSUPPORTED, bad
    assert bwd(nbytes=need - 1) == WORKSPACE


def test_clip_abi_refusals():
    L = _lib.lib()
    need = L.qlora_clip_workspace_size(2)
    assert need > 0 and L.qlora_clip_workspace_size(1000) > need
    assert L.qlora_clip_workspace_size(-1) == L.qlora_clip_workspace_size((1 << 20) + 1) == 0

    def arr(t, *v):
        return None if v == (None,) else ctypes.cast((t * len(v))(*v), ctypes.c_void_p)

    def clip(n=2, grads=(P, P), sizes=(4, 5), types=(0, 1), max_norm=1.0, out=(P, P), norm=P,
             ws=P, nbytes=need):
        keep = [arr(ctypes.c_void_p, *grads), arr(ctypes.c_int64, *sizes),
                arr(ctypes.c_int32, *types), arr(ctypes.c_void_p, *out)]
        return L.qlora_clip_grad_norm(n, *keep[:3], max_norm, keep[3], norm, ws, nbytes, None)
    for bad in (dict(n=-1), dict(n=(1 << 20) + 1), dict(grads=(None,)), dict(sizes=(None,)),
                dict(types=(None,)), dict(sizes=(4, -1)), dict(sizes=((1 << 44), 1)),
                dict(grads=(P, 0)), dict(grads=(P + 1, P)), dict(grads=(P, P + 2)),
                dict(out=(P, 0)), dict(out=(P, P + 2)), dict(max_norm=-0.5),
                dict(max_norm=math.nan), dict(norm=None), dict(norm=P + 2), dict(ws=None),
                dict(ws=P + 8)):
        assert clip(**bad) == INVALID, bad
    assert clip(types=(0, 2)) == UNSUPPORTED
    assert clip(nbytes=need - 1) == WORKSPACE


def test_attention_abi_rejects_outputs_that_overlap():
    """On the host: rows of an output that lie on top of each other, and
    outputs that start where a tensor does that is read after them."""
    L = _lib.lib()
    far = [P << i for i in range(1, 9)]
    dense = dict(batch_stride=4 * 12 * 64, row_stride=4 * 64, head_stride=64)

    def view(i, **kw):
        return _view(**{"data": far[i], **dense, **kw})

    def bwd(**kw):
        vs = [kw.get(n, view(i)) for i, n in enumerate(("q", "k", "v", "o", "do", "dq", "dk", "dv"))]
        return L.qlora_attention_bwd(_attn(), *vs[:4], P, *vs[4:], P, 1 << 30, None)
    for bad in (dict(batch_stride=0), dict(row_stride=0), dict(head_stride=0), dict(head_stride=56),
                dict(row_stride=192), dict(batch_stride=4 * 64), dict(row_stride=64)):
        assert _fwd(_attn(), view(0), view(1), view(2), view(3, **bad)) == INVALID, bad
        for i, n in ((5, "dq"), (6, "dk"), (7, "dv")):
            # 2 key/value heads of 64 fit a row stride of 192
            if n == "dq" or bad != dict(row_stride=192):
                assert bwd(**{n: view(i, **bad)}) == INVALID, (n, bad)
    for i in (1, 2):
        assert _fwd(_attn(), view(0), view(1), view(2), view(i)) == INVALID
    assert _fwd(_attn(), view(0), view(1), view(2), view(0, row_stride=2 * 4 * 64,
                                                         batch_stride=1 << 16)) == INVALID
    for n, over in (("dq", (0, 1, 2, 4, 6, 7)), ("dk", (0, 2, 3, 4, 5, 7)), ("dv", (0, 1, 3, 4, 5, 6))):
        for i in over:
            assert bwd(**{n: view(i)}) == INVALID, (n, i)
    for n, i in (("dq", 3), ("dk", 1), ("dv", 2)):   # the view that it may be, with other strides
        assert bwd(**{n: view(i, batch_stride=1 << 16)}) == INVALID


@pytest.mark.parametrize("scale", [1e-45, 1e-39, 2.0 ** -101, 2.0 ** 101, 3e38])
def test_attention_abi_rejects_scales_whose_inverse_leaves_fp32(scale):
    assert _fwd(_attn(scale=scale), lse=None) == INVALID
    assert _lib.lib().qlora_attention_bwd_workspace_size(_attn(scale=scale)) == 0


@pytest.mark.parametrize("scale", [2.0 ** -100, 1.0, 2.0 ** 100])
def test_attention_abi_takes_the_other_scales(scale):
    assert _lib.lib().qlora_attention_bwd_workspace_size(_attn(scale=scale)) > 0


def test_only_backward_norm_kernels_that_a_call_reaches_are_built():
    """(threads, threads per row, vectors per thread) of each row type: between
    1025 and 2048 vectors fp32 rows take 1024 threads with two each, bf16 rows 512
    with four, and neither has the other's kernel."""
    names = subprocess.run(["nm", qn.LIB_PATH], capture_output=True, text=True, check=True).stdout
    found = re.findall(r"stub__k_norm_bwdINS0_\d(F32T|BF16T)E\w*?Li(\d+)ELi(\d+)ELi(\d+)E", names)
    got = {(t, *map(int, n)) for t, *n in found}
    both = {(1024, 64, 1), (512, 64, 2), (1024, 256, 1), (1024, 512, 1), (1024, 1024, 1),
            (1024, 1024, 4), (1024, 1024, 8)}
    assert got == ({(t, *s) for t in ("F32T", "BF16T") for s in both} |
                   {("F32T", 1024, 1024, 2), ("BF16T", 512, 512, 4)})
