"""The operators together, as a finetuning step uses them: the example block's
output and gradients against the same block in fp32 torch operations on the
dequantized weights, and a short training run.

Tolerance of one step: the chain rounds its activations and gradients to bf16
about ten times in a row (2^-8 at most, 2^-8 / sqrt(6) rms each); rms errors
add in quadrature to 5e-3 of a tensor's norm per pass and gradients see both
passes, with residual branches that keep relative errors from growing: 3e-2.
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


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.fail("GPU tests need a ROCm GPU")
    spec = importlib.util.spec_from_file_location(
        "finetune_block", os.path.join(ROOT, "examples", "finetune_block.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def reference(block, x, lengths):
    """The block in fp32 torch operations; returns the output and its leaves
    by the block's parameter names."""
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
    y = x + linear("down", torch.nn.functional.silu(linear("gate", h)) * linear("up", h))
    return y, leaves


def test_step_against_plain_operations(example):
    say("[block] one step")
    lengths = [70, 1, 129, 40]
    block = example.Block(width=256, heads=4, kv_heads=2, inner=704)
    with torch.no_grad():   # adapters that do something
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
    say(f"    y {off(y, ry):.2e}")
    assert off(y, ry) < TOL
    for n, p in block.named_parameters():
        say(f"    {n} {off(p.grad, leaves[n].grad):.2e}")
        assert off(p.grad, leaves[n].grad) < TOL, n


def test_training_lowers_the_loss_and_clips(example):
    say("[block] training")
    block = example.Block(width=256, heads=4, kv_heads=1, inner=704)
    x = torch.randn(300, 256, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    cu = example.offsets([200, 100])
    with torch.no_grad():
        target = example.Block(width=256, heads=4, kv_heads=1, inner=704, seed=9)(x, cu).float()
    losses, norms = example.train(block, x, target, cu, 15, max_norm=0.05, report=say)
    assert losses[-1] < losses[0] and all(n > 0.05 for n in norms)
    # what the optimizer sees is clipped (each bf16 gradient is rounded once more)
    params = [p for p in block.parameters() if p.grad is not None]
    total = torch.stack([p.grad.float().square().sum() for p in params]).sum().sqrt()
    assert abs(float(total) - 0.05) <= 0.05 * 2.0 ** -8


def test_captured_step_replays(example):
    """Attention, norms and their backward passes in a HIP graph, replayed on
    new inputs: the same bits as the eager calls every time."""
    say("[block] graph")
    q, k, v, do = (torch.zeros(2, 150, h, 64, dtype=torch.bfloat16, device="cuda")
                   for h in (4, 2, 2, 4))
    x, dy = torch.zeros(300, 256, device="cuda"), torch.zeros(300, 256, device="cuda")
    w = torch.ones(256, device="cuda")

    def run():
        o, lse = qn.attention_fwd(q, k, v)
        y, mean, rstd = qn.norm_fwd(x, w, w)
        return [o, lse, *qn.attention_bwd(q, k, v, o, lse, do), y, *qn.norm_bwd(dy, x, w, mean, rstd)]
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for i in range(4):
        g = torch.Generator(device="cuda").manual_seed(i)
        for t in (q, k, v, do, x, dy):
            t.copy_(torch.randn(t.shape, generator=g, device="cuda"))
        expect = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, expect):
            assert torch.equal(a, b)
