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


def test_states_of_other_parameters_are_refused():
    """The same number of blocks in all, other tensors: [300, 64] takes 2 + 1
    blocks, [64, 300] 1 + 2."""
    def opt(*sizes, **kw):
        return qn.AdamW([torch.nn.Parameter(torch.ones(n)) for n in sizes], **kw)
    for bits in (32, 8):
        saved = opt(300, 64, bits=bits).state_dict()
        opt(300, 64, bits=bits).load_state_dict(saved)
        for other in (opt(64, 300, bits=bits), opt(301, 64, bits=bits), opt(256, 512, bits=bits)):
            other._kept[0]["state"].m.fill_(3)
            with pytest.raises(ValueError, match="other parameters"):
                other.load_state_dict(saved)
            assert (other._kept[0]["state"].m == 3).all()
    # the same number of elements in another shape
    a = qn.AdamW([torch.nn.Parameter(torch.ones(4, 75))])
    with pytest.raises(ValueError, match="other parameters"):
        a.load_state_dict(qn.AdamW([torch.nn.Parameter(torch.ones(75, 4))]).state_dict())
    # states saved without the shapes: by their sizes in all
    saved = opt(300, 64).state_dict()
    del saved["kept"][0]["shapes"]
    opt(300, 64).load_state_dict(saved)
    with pytest.raises(ValueError, match="other parameters"):
        opt(300, 640).load_state_dict(saved)


def test_groups_are_counted():
    ps = [torch.nn.Parameter(torch.ones(300)) for _ in range(2)]
    opt = qn.AdamW([{"params": ps[:1], "lr": 0.5}, {"params": ps[1:], "lr": 0.25}])
    for name in ("groups", "kept"):
        saved = opt.state_dict()
        saved[name] = saved[name][:1]
        with pytest.raises(ValueError, match="groups"):
            opt.load_state_dict(saved)
        assert [g["lr"] for g in opt.param_groups] == [0.5, 0.25]


def test_saved_states_are_plain(tmp_path):
    """They pass through torch's file format without code."""
    ps = [torch.nn.Parameter(torch.ones(4, 75)), torch.nn.Parameter(torch.ones(7).bfloat16())]
    opt = qn.AdamW(ps, bits=8, masters=True, betas=(0.8, 0.9))
    torch.save(opt.state_dict(), tmp_path / "s.pt")
    saved = torch.load(tmp_path / "s.pt", weights_only=True)
    other = qn.AdamW([torch.nn.Parameter(p.detach().clone()) for p in ps], bits=8, masters=True)
    other.load_state_dict(saved)
    assert other.param_groups[0]["betas"] == (0.8, 0.9)


def test_groups_without_parameters(monkeypatch):
    """As torch's optimizers: such a group is there, and has nothing to do."""
    monkeypatch.setattr(optim, "adamw_step", lambda *a, **k: None)
    ps, opt = _opt(1, bits=8, masters=True)
    opt.add_param_group({"params": [], "lr": 0.5})
    ps[0].grad = torch.ones_like(ps[0])
    opt.step()
    opt.take_masters()
    saved = opt.state_dict()
    assert [k["step"] for k in saved["kept"]] == [[1], []]
    opt.param_groups[1]["lr"] = 0.25
    opt.load_state_dict(saved)
    assert opt.param_groups[1]["lr"] == 0.5


def test_a_group_that_fails_is_not_added(monkeypatch):
    ps, opt = _opt(1)

    def no_room(*a):
        raise MemoryError
    monkeypatch.setattr(optim, "adamw_init", no_room)
    with pytest.raises(MemoryError):
        opt.add_param_group({"params": [torch.nn.Parameter(torch.ones(3))]})
    assert len(opt.param_groups) == len(opt._kept) == 1
