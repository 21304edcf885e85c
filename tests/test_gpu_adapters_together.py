"""Rotary positions, the AdamW step and the many-adapter layer together, as they
are used: blocks with rotary positions are trained by the package's AdamW, and
their adapters are then served beside the one base that they share.

Tolerance of a training step's gradients: as for the block without positions
(about ten bf16 roundings in a row, 2^-8 / sqrt(6) rms each, both passes, with
residual branches: 3e-2); the rotation adds one rounding to q, k and to each of
their gradients.
"""

import importlib.util
import os

import pytest
import torch

import quantized_base_lora_nf4_amd as qn
from gpu_util import say

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOL = 3e-2
SMALL = dict(width=256, heads=4, kv_heads=2, inner=704)


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "finetune_block", os.path.join(ROOT, "examples", "finetune_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def turn(x, positions, f):
    """Halves, in fp32."""
    a = positions[:, None].double() * f
    c, s = a.cos().float()[:, None], a.sin().float()[:, None]
    u, v = x.chunk(2, -1)
    return torch.cat([u * c - v * s, v * c + u * s], -1)


def reference(block, x, lengths):
    leaves = {n: p.detach().float().requires_grad_() for n, p in block.named_parameters()}

    def linear(name, h):
        m = getattr(block, name)
        w = qn.nf4_dequantize(m.nf4).float()
        return h @ w.T + m.s * (h @ leaves[name + ".A"].T) @ leaves[name + ".B"].T

    def norm(name, h):
        m = getattr(block, name)
        return h * torch.rsqrt(h.square().mean(-1, keepdim=True) + m.eps) * leaves[name + ".weight"]

    x = x.float()
    h = norm("norm_attn", x)
    q, k, v = (linear(n, h).unflatten(-1, (-1, block.dim)) for n in "qkv")
    pos = torch.cat([torch.arange(n) for n in lengths]).cuda()
    q, k = turn(q, pos, block.inv_freq), turn(k, pos, block.inv_freq)
    share = q.shape[1] // k.shape[1]
    k, v = (t.repeat_interleave(share, 1) for t in (k, v))
    out = []
    for a, b, c in zip(q.split(lengths), k.split(lengths), v.split(lengths)):
        s = (a.transpose(0, 1) @ b.transpose(0, 1).transpose(1, 2)) * block.dim ** -0.5
        n = s.shape[-1]
        s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -torch.inf)
        out.append((s.softmax(-1) @ c.transpose(0, 1)).transpose(0, 1))
    x = x + linear("o", torch.cat(out).flatten(-2))
    h = norm("norm_mlp", x)
    return x + linear("down", torch.nn.functional.silu(linear("gate", h)) * linear("up", h)), leaves


def test_step_with_positions_against_plain_operations(example):
    say("[together] one step with positions")
    lengths = [70, 1, 129, 40]
    block = example.Block(rope=True, **SMALL)
    with torch.no_grad():
        for n, p in block.named_parameters():
            if n.endswith(".B"):
                p.copy_(0.05 * torch.randn(p.shape, generator=torch.Generator().manual_seed(len(n))))
    g = torch.Generator().manual_seed(3)
    x = torch.randn(sum(lengths), 256, generator=g).bfloat16().cuda()
    dy = torch.randn(sum(lengths), 256, generator=g).bfloat16().cuda()
    y = block(x, example.offsets(lengths))
    y.backward(dy)
    ry, leaves = reference(block, x, lengths)
    ry.backward(dy.float())

    def off(a, b):
        return float((a.detach().float() - b.detach()).norm() / b.detach().norm())
    assert off(y, ry) < TOL
    for n, p in block.named_parameters():
        say(f"    {n} {off(p.grad, leaves[n].grad):.2e}")
        assert off(p.grad, leaves[n].grad) < TOL, n


def test_example_runs_as_a_program(example, monkeypatch, capsys):
    import sys
    for flags in (["--rope", "--adamw", "8"], ["--adamw", "32"]):
        monkeypatch.setattr(sys, "argv", ["finetune_block.py", "--steps", "2", "--tokens", "100", *flags])
        example.main()
        assert "step 1: loss" in capsys.readouterr().out


@pytest.mark.parametrize("bits", [32, 8])
def test_trained_adapters_served_together(example, bits):
    """Two blocks of one base, trained towards different targets; their
    projections then serve a mixed batch, from single tokens to prompts."""
    say(f"[together] {bits} bits")
    lengths = [60, 4, 36]
    cu = example.offsets(lengths)
    x = torch.randn(100, 256, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    blocks = []
    for seed in (9, 10):
        block = example.Block(rope=True, **SMALL)
        with torch.no_grad():
            target = example.Block(rope=True, seed=seed, **SMALL)(x, cu).float()
        before = {n: p.detach().clone() for n, p in block.named_parameters()}
        losses, norms = example.train(block, x, target, cu, 4, max_norm=0.05, report=say, bits=bits)
        assert all(torch.isfinite(torch.tensor(losses + norms))) and norms[0] > 0
        assert any(not torch.equal(p, before[n]) for n, p in block.named_parameters() if n.endswith(".B"))
        blocks.append(block)
    for name in ("q", "k", "gate", "down"):
        layers = [getattr(b, name) for b in blocks]
        assert torch.equal(layers[0].nf4.codes, layers[1].nf4.codes)   # the base was not trained
        many = qn.QLoRAMultiLinear(layers[0], slots=4, r=8)
        many.load(0, layers[0])
        many.load(2, layers[1])
        for rows in (1, 9, 50, 300):
            h = torch.randn(rows, many.nf4.K, generator=torch.Generator().manual_seed(rows)).bfloat16().cuda()
            index = torch.tensor([0, 2, -1], dtype=torch.int32).repeat(-(-rows // 3))[:rows].cuda()
            y = many(h, index)
            with torch.no_grad():
                for slot, layer in ((0, layers[0]), (2, layers[1])):
                    mine = index == slot
                    if mine.any():
                        z = layer(h[mine]).double()
                        # both round the output, and U or the weight's levels
                        assert float((y[mine].double() - z).norm() / z.norm()) <= 2.0 ** -8
