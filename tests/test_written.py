"""Versions of tensors that the kernels write into (the calls: on the GPU)."""

import pytest
import torch

from quantized_base_lora_nf4_amd._lib import tensors, written


def test_versions_are_counted():
    x = torch.zeros(10)
    view, apart = x[2:5], torch.zeros(3, dtype=torch.bfloat16)
    written(view, None, apart)
    assert (x._version, view._version, apart._version) == (1, 1, 1)
    tensors().written([x.detach(), x])
    assert x._version == 3 and apart._version == 1
    written()
    tensors().written([])
    p = torch.nn.Parameter(torch.ones(3))
    y = p * p
    written(p.detach())
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    with torch.inference_mode():
        z = torch.zeros(3)
        written(z, p)
    written(z)
    assert p._version == 2


def test_what_is_refused():
    x = torch.zeros(3)
    for bad in (3, None):
        with pytest.raises(TypeError, match="list or tuple"):
            tensors().written(bad)
    with pytest.raises(TypeError, match="expected tensors"):
        written(x, "x")
