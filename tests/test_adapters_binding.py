"""Refusals of rotary positions, the AdamW step and the many-adapter layer, on
the CPU: the torch binding rejects host tensors, and the C ABI rejects bad
sizes, strides, alignments and workspaces, before anything is launched."""

import array
import ctypes

import pytest
import torch

import quantized_base_lora_nf4_amd as qn
from quantized_base_lora_nf4_amd import _lib
from quantized_base_lora_nf4_amd._lib import AdamW, Heads, Nf4Tensor, Rope

INVALID, UNSUPPORTED, WORKSPACE = (_lib.QLORA_ERR_INVALID, _lib.QLORA_ERR_UNSUPPORTED,
                                   _lib.QLORA_ERR_WORKSPACE)
# Addresses that are never followed: every call below fails its checks or has nothing to do.
P = 1 << 20


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


# ---- binding ----

def test_rope_rejects_host_tensors():
    f, _ = qn.rope_frequencies(64, device="cpu")
    with pytest.raises(ValueError, match="q is on cpu"):
        qn.rope_fwd(_bf(1, 4, 2, 64), _bf(1, 4, 2, 64), f)
    with pytest.raises(ValueError, match="dq is on cpu"):
        qn.rope_bwd(_bf(1, 4, 2, 64), None, f)
    with pytest.raises(TypeError, match="q must be a torch tensor"):
        qn.rope_fwd(None, None, f)


def test_adamw_rejects_host_tensors():
    p = [torch.zeros(300)]
    with pytest.raises(ValueError, match="is on cpu"):
        qn.adamw_step(p, p, qn.adamw_init(p), 1, 1e-3)
    with pytest.raises(ValueError, match="is on cpu"):
        qn.adamw_values(qn.adamw_init(p, 8))
    with pytest.raises(TypeError, match="torch tensors"):
        qn.adamw_step([1.0], [None], qn.adamw_init(p), 1, 1e-3)
    for kw, match in ((dict(bits=16), "bits"), (dict(lr=-1.0), "lr"), (dict(eps=float("nan")), "eps"),
                      (dict(betas=(1.0, 0.9)), "betas"), (dict(weight_decay=-1.0), "weight_decay"),
                      (dict(max_norm=-1.0), "max_norm")):
        with pytest.raises(ValueError, match=match):
            qn.AdamW([torch.nn.Parameter(torch.zeros(3))], **kw)


def test_multi_rejects_host_tensors():
    w = qn.alloc_nf4(64, 64, device="cpu")
    with pytest.raises(ValueError, match="is on cpu"):
        qn.qlora_linear_multi_fwd(w, _bf(3, 64), _bf(2, 8, 64), _bf(2, 64, 8), torch.zeros(2),
                                  torch.zeros(3, dtype=torch.int32))


# ---- C ABI: rotary positions ----

def _rope(view=None, **kw):
    a = dict(n_seq=2, rows=10, cu_seqlens=None, positions=None, position_batch_stride=0,
             position_row_stride=0, inv_freq=P, position_bytes=0, q_heads=4, k_heads=2, head_dim=64,
             rot=64, interleaved=0, inverse=0, scale=1.0)
    a.update(kw)
    v = {"q": dict(data=P), "k": dict(data=2 * P), "qo": dict(data=3 * P), "ko": dict(data=4 * P)}
    for n, d in (view or {}).items():
        v[n].update(d)
    views = []
    for n in ("q", "k", "qo", "ko"):
        h = a["q_heads"] if n[0] == "q" else a["k_heads"]
        d = dict(batch_stride=10 * h * 64, row_stride=h * 64, head_stride=64)
        d.update(v[n])
        views.append(Heads(d["data"], d["batch_stride"], d["row_stride"], d["head_stride"]))
    return _lib.lib().qlora_rope(Rope(*a.values()), *(ctypes.addressof(x) for x in views), None), views


@pytest.mark.parametrize("kw,status", [
    (dict(n_seq=-1), INVALID), (dict(rows=-1), INVALID), (dict(rows=1 << 30), INVALID),
    (dict(q_heads=0), INVALID), (dict(k_heads=-1), INVALID), (dict(rot=0), INVALID),
    (dict(rot=63), INVALID), (dict(rot=66), INVALID), (dict(head_dim=0), INVALID),
    (dict(head_dim=68), UNSUPPORTED), (dict(head_dim=1032), UNSUPPORTED),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(inv_freq=None), INVALID), (dict(inv_freq=P + 4), INVALID),
    (dict(cu_seqlens=P + 2), INVALID), (dict(positions=P, position_bytes=2), INVALID),
    (dict(positions=P + 4, position_bytes=8), INVALID),
    (dict(positions=P, position_bytes=4, position_row_stride=-1), INVALID),
    (dict(view=dict(q=dict(data=None))), INVALID), (dict(view=dict(k=dict(data=P + 2))), INVALID),
    (dict(view=dict(q=dict(row_stride=12))), INVALID), (dict(view=dict(k=dict(head_stride=-8))), INVALID),
    (dict(view=dict(qo=dict(row_stride=64))), INVALID), (dict(view=dict(ko=dict(batch_stride=0))), INVALID),
    (dict(view=dict(qo=dict(data=P, row_stride=512))), INVALID),   # q's address, another view
    (dict(view=dict(qo=dict(data=2 * P))), INVALID), (dict(view=dict(ko=dict(data=P))), INVALID),
    (dict(view=dict(ko=dict(data=3 * P))), INVALID),
])
def test_abi_rope(kw, status):
    assert _rope(**kw)[0] == status


def test_abi_rope_with_nothing_to_do():
    assert _rope(rows=0, inv_freq=None)[0] == _lib.QLORA_OK
    assert _rope(n_seq=0, view=dict(q=dict(data=None)))[0] == _lib.QLORA_OK


# ---- C ABI: AdamW ----

def _adamw(sizes=(300, 7), **kw):
    n = len(sizes)
    lists = dict(params=array.array("Q", [P * (i + 1) for i in range(n)]),
                 grads=array.array("Q", [P * (i + 9) for i in range(n)]), copies=None,
                 sizes=array.array("q", sizes), param_types=array.array("i", [1] * n),
                 grad_types=array.array("i", [0] * n))
    lists.update({k: kw.pop(k) for k in list(kw) if k in lists})
    a = dict(n=n, m=P, v=2 * P, m_scale=None, v_scale=None, state_blocks=3, step=1, lr=1e-3, beta1=0.9,
             beta2=0.999, weight_decay=0.0, lr_dev=None, step_dev=None, norm=None, eps=1e-8, max_norm=0.0,
             state_bits=32)
    a.update(kw)
    ptr = {k: v.buffer_info()[0] if isinstance(v, array.array) else v for k, v in lists.items()}
    s = AdamW(a["n"], ptr["params"], ptr["grads"], ptr["copies"], ptr["sizes"], ptr["param_types"],
              ptr["grad_types"], a["m"], a["v"], a["m_scale"], a["v_scale"], a["state_blocks"], a["step"],
              a["lr"], a["beta1"], a["beta2"], a["weight_decay"], a["lr_dev"], a["step_dev"], a["norm"],
              a["eps"], a["max_norm"], a["state_bits"])
    return _lib.lib().qlora_adamw_step(s, None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(n=(1 << 20) + 1), INVALID), (dict(sizes=(300, -1)), INVALID),
    (dict(sizes=(1 << 40, 7)), INVALID), (dict(state_bits=16), UNSUPPORTED),
    (dict(param_types=array.array("i", [1, 2])), UNSUPPORTED),
    (dict(grad_types=array.array("i", [5, 0])), UNSUPPORTED),
    (dict(params=None), INVALID), (dict(grads=None), INVALID), (dict(param_types=None), INVALID),
    (dict(params=array.array("Q", [0, P])), INVALID), (dict(params=array.array("Q", [P + 2, P])), INVALID),
    (dict(grads=array.array("Q", [P + 1, P])), INVALID), (dict(copies=array.array("Q", [P + 1, 0])), INVALID),
    (dict(m=None), INVALID), (dict(v=P + 8), INVALID), (dict(state_blocks=2), WORKSPACE),
    (dict(state_bits=8), INVALID), (dict(state_bits=8, m_scale=P, v_scale=P + 2), INVALID),
    (dict(step=0), INVALID), (dict(lr=-1e-3), INVALID), (dict(lr=float("nan")), INVALID),
    (dict(beta1=1.0), INVALID), (dict(beta2=-0.1), INVALID), (dict(beta2=float("nan")), INVALID),
    (dict(weight_decay=-1.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("inf")), INVALID),
    (dict(norm=P, max_norm=float("nan")), INVALID), (dict(norm=P, max_norm=-1.0), INVALID),
    (dict(norm=P + 2), INVALID), (dict(lr_dev=P + 2), INVALID), (dict(step_dev=P + 4), INVALID),
])
def test_abi_adamw(kw, status):
    assert _adamw(**kw) == status


def test_abi_adamw_with_nothing_to_do():
    assert _adamw(sizes=()) == _lib.QLORA_OK
    assert _adamw(sizes=(0, 0), m=None, v=None, state_blocks=0) == _lib.QLORA_OK
    assert _adamw(grads=array.array("Q", [0, 0])) == _lib.QLORA_OK


def test_abi_adamw_blocks():
    L = _lib.lib()
    sizes = array.array("q", [0, 1, 256, 257, 5000])
    assert L.qlora_adamw_blocks(5, sizes.buffer_info()[0]) == 0 + 1 + 1 + 2 + 20
    assert L.qlora_adamw_blocks(0, None) == 0
    assert L.qlora_adamw_blocks(1, None) == -1 and L.qlora_adamw_blocks(-1, None) == -1
    big = array.array("q", [1 << 38] * 2)
    assert L.qlora_adamw_blocks(1, big.buffer_info()[0]) == 1 << 30
    assert L.qlora_adamw_blocks(2, big.buffer_info()[0]) == -1


@pytest.mark.parametrize("args", [
    (None, P, P, P, 1, P, P), (P, P + 1, P, P, 1, P, P), (P, P, P + 2, P, 1, P, P),
    (P, P, P, None, 1, P, P), (P, P, P, P, 1, P + 4, P), (P, P, P, P, -1, P, P),
    (P, P, P, P, 1 << 31, P, P)])
def test_abi_adamw_values(args):
    assert _lib.lib().qlora_adamw_values(*args, None) == INVALID


# ---- C ABI: many adapters ----

def _multi(w=None, **kw):
    t = dict(codes=P, q8=P, step=P, N=64, K=128, blocksize=64, dq_blocksize=256, code_type=0, levels=None)
    t.update(w or {})
    a = dict(X=P, M=40, A=P, B=P, s=P, n=3, r=8, index=P, Y=2 * P, ws=P, ws_bytes=1 << 30)
    a.update(kw)
    return _lib.lib().qlora_linear_multi_fwd(ctypes.byref(Nf4Tensor(*t.values())), *a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(X=None), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(s=None), INVALID),
    (dict(index=None), INVALID), (dict(Y=None), INVALID), (dict(ws=None), INVALID),
    (dict(X=P + 2), INVALID), (dict(s=P + 2), INVALID), (dict(index=P + 1), INVALID), (dict(ws=P + 8), INVALID),
    (dict(M=0), INVALID), (dict(M=(1 << 26) + 1), INVALID), (dict(n=0), INVALID), (dict(r=0), INVALID),
    (dict(r=257), INVALID), (dict(ws_bytes=100), WORKSPACE), (dict(M=3, ws_bytes=100), WORKSPACE),
    (dict(M=5000, ws_bytes=100), WORKSPACE), (dict(w=dict(N=60)), INVALID), (dict(w=dict(K=96)), INVALID),
    (dict(w=dict(blocksize=32)), UNSUPPORTED), (dict(w=dict(code_type=9)), UNSUPPORTED),
    (dict(w=dict(code_type=4)), INVALID), (dict(Y=P), INVALID),
])
def test_abi_multi(kw, status):
    assert _multi(**kw) == status


def test_multi_workspace_sizes():
    f = qn.multi_workspace_size
    assert f(0, 64, 64, 8) == f(5, 60, 64, 8) == f(5, 64, 60, 8) == f(5, 64, 64, 0) == f(5, 64, 64, 257) == 0
    assert f((1 << 26) + 1, 64, 64, 8) == 0
    # U's partial sums of every row at least
    for M in (1, 16, 17, 300, 5000):
        for r in (1, 8, 100):
            assert f(M, 1024, 4096, r) >= 4 * M * r


# ---- the tile kernels' waits ----

def test_step_barriers_of_the_many_adapter_tiles():
    """The check of test_gemm_step_waits, on the instances for rows of many
    adapters: no step's barrier runs before its tile has landed."""
    import os
    import subprocess
    import tempfile

    import test_gemm_step_waits as waits
    if not os.path.exists(waits.HIPCC):
        pytest.skip("hipcc not available")
    src = os.path.join(os.path.dirname(waits.SRC), "qgemm_multi.hip")
    with tempfile.TemporaryDirectory() as d:
        out = os.path.join(d, "qgemm_multi.s")
        subprocess.run([waits.HIPCC, "--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang",
                        "-target-feature", "-Xclang", "-packed-fp32-ops",
                        "-I" + os.path.join(waits.ROOT, "include"), "--cuda-device-only", "-S", src,
                        "-o", out], check=True, capture_output=True)
        text = open(out).read()
    checked = 0
    for name, body in waits.kernels(text):
        for seg in waits.step_segments(body):
            assert waits.tile_covered(seg), f"{name}: a step barrier may run before the tile landed"
            checked += 1
    assert checked >= 4 * 14


def test_tensor_lists():
    """The compiled reader: ordinary lists only (its values are tested on the GPU)."""
    import array
    from quantized_base_lora_nf4_amd._lib import tensors
    T = tensors()
    x = [torch.zeros(3, 2), torch.zeros(3, 2)]
    room = array.array("Q", bytes(64))
    at = room.buffer_info()[0]
    for bad in (x, [3], [None], [], [x[0], "a"], [torch.zeros(2, device="meta")]):
        assert T.describe(bad, at, at, at, 0, 1) == -1
    assert not any(room)
    for args in (((1, 2), at, at, at, 0, 1), (x, at), (x, "a", at, at, 0, 1)):
        with pytest.raises(TypeError):
            T.describe(*args)
    for bad in ((0, "f", (x[0],), ((3, 2),)), (0, "f", (3,), ((3,),)), (0, "ff", (x[0],), ((3, 2),)), (0, "f", (x[0],), (None,))):
        assert not T.fits(*bad)
    assert T.fits(0, "", (), ())
    assert T.same_shapes(x, [torch.ones(3, 2, dtype=torch.int8)] * 2) and T.same_shapes([], [])
    for other in ([x[0]], [x[0], torch.zeros(2, 3)], [x[0], torch.zeros(6)], [x[0], None]):
        assert not T.same_shapes(x, other)
    for values, apart in (([], True), ([5], True), ([1, 2, 9], True), ([9, 1, 2], True), ([3, 3], False),
                          ([7, 1, 8, 1], False), ([2**64 - 1, 0, 2**63], True)):
        a = array.array("Q", values)
        assert T.distinct(a.buffer_info()[0], len(a)) is apart
