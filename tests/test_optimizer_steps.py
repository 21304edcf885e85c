"""The optimizer's own bookkeeping, on the CPU: what step() hands to adamw_step
and what it keeps when that refuses.  (The values are tested on the GPU.)"""

import pytest
import torch

import quantized_base_lora_nf4_amd as qn
from quantized_base_lora_nf4_amd import optim


def _opt(n=3, **kw):
    ps = [torch.nn.Parameter(torch.ones(300 + i)) for i in range(n)]
    return ps, qn.AdamW(ps, lr=1e-2, **kw)


def _counts(opt, i=0):
    """Steps that each of three parameters has made."""
    k = opt.state_dict()["kept"][i]["step"]
    return [k] * 3 if isinstance(k, int) else list(k)


def test_a_refused_step_is_not_counted(monkeypatch):
    """Host tensors are refused: nothing was updated, so nothing is counted."""
    ps, opt = _opt()
    for p in ps:
        p.grad = torch.ones_like(p)
    for _ in range(2):
        with pytest.raises(ValueError, match="is on cpu"):
            opt.step()
    assert _counts(opt) == [0, 0, 0]
    monkeypatch.setattr(optim, "adamw_step", lambda *a, **k: None)
    opt.step()
    assert _counts(opt) == [1, 1, 1]
