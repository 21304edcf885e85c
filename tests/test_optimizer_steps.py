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


def test_every_parameter_counts_its_own_steps(monkeypatch):
    """adamw_step is told the number of steps that each tensor with a gradient
    has made, this one included: one number where they agree."""
    told = []
    monkeypatch.setattr(optim, "adamw_step", lambda p, g, s, step, *a: told.append(
        (step, [x is not None for x in g])))
    ps, opt = _opt()

    def step(*have):
        for i, p in enumerate(ps):
            p.grad = torch.ones_like(p) if i in have else None
        opt.step()
    step(0, 1)
    step(0)
    step(0, 1, 2)
    step()                # no gradient at all: no call
    step(1, 2)
    assert told[0] == (1, [True, True, False])
    assert told[1] == (2, [True, False, False])
    assert told[2] == ([3, 2, 1], [True] * 3)
    assert told[3][1] == [False, True, True] and list(told[3][0])[1:] == [3, 2]
    assert len(told) == 4 and _counts(opt) == [3, 3, 2]


def test_counts_are_saved_and_loaded(monkeypatch):
    monkeypatch.setattr(optim, "adamw_step", lambda *a, **k: None)
    ps, opt = _opt()
    ps[1].grad = torch.ones_like(ps[1])
    opt.step()
    saved = opt.state_dict()
    opt.step()
    assert _counts(opt) == [0, 2, 0]
    _, other = _opt()
    other.load_state_dict(saved)
    assert _counts(other) == [0, 1, 0]
    # states saved with one count for the group: every parameter's
    saved["kept"][0]["step"] = 7
    other.load_state_dict(saved)
    assert _counts(other) == [7, 7, 7]
    saved["kept"][0]["step"] = [1, 2]
    with pytest.raises(ValueError, match="other parameters"):
        other.load_state_dict(saved)


def test_copies_keep_the_counts(monkeypatch):
    import copy
    monkeypatch.setattr(optim, "adamw_step", lambda *a, **k: None)
    ps, opt = _opt()
    ps[2].grad = torch.ones_like(ps[2])
    opt.step()
    other = copy.deepcopy(opt)
    opt.step()
    assert _counts(opt) == [0, 0, 2] and _counts(other) == [0, 0, 1]
    opt._kept[0]["step"] = 5   # a copy of the time when the group had one count
    assert _counts(copy.deepcopy(opt)) == [5, 5, 5]
