"""One finetuning step after the other of a pre-norm decoder block whose
projections are frozen NF4 weights with LoRA adapters.

    python examples/finetune_block.py --steps 20 --rope --adamw 8

Everything of a step runs through this package: the q, k, v, o, gate, up and
down projections (QLoRALinear), root-mean-square norms, rotary positions
(--rope), causal attention with shared key/value heads over packed examples of
unequal length, the clipping of all adapters' and norms' gradients by their
global norm and, with --adamw 8 or 32, the AdamW step with states in so many
bits, which clips on the way.  The rest (SiLU, residual sums, loss, and by
default AdamW) is plain torch.  Weights and data are synthetic: the block
learns to reproduce another block's output.
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import quantized_base_lora_nf4_amd as qn  # noqa: E402


class Block(torch.nn.Module):
    def __init__(self, width=512, heads=8, kv_heads=2, inner=1408, r=8, alpha=16.0, seed=0,
                 rope=False):
        super().__init__()
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dim = width // heads
        self.inv_freq = qn.rope_frequencies(self.dim)[0] if rope else None
        kv = kv_heads * self.dim

        def linear(n, k):
            # frozen base at the scale of a trained layer, B = 0: the adapter starts as nothing
            w = torch.randn(n, k, generator=g, device="cuda") * k ** -0.5
            a = (torch.randn(r, k, generator=g, device="cuda") * 0.01).bfloat16()
            return qn.QLoRALinear(w, r, alpha, A=a)

        self.norm_attn, self.norm_mlp = qn.RMSNorm(width), qn.RMSNorm(width)
        self.q, self.k, self.v, self.o = (linear(width, width), linear(kv, width),
                                          linear(kv, width), linear(width, width))
        self.gate, self.up, self.down = (linear(inner, width), linear(inner, width),
                                         linear(width, inner))

    def forward(self, x, cu_seqlens):
        """x [tokens, width] bf16; cu_seqlens: the packed examples' offsets."""
        h = self.norm_attn(x)
        q, k, v = (p(h).unflatten(-1, (-1, self.dim)) for p in (self.q, self.k, self.v))
        if self.inv_freq is not None:
            q, k = qn.rope(q, k, self.inv_freq, cu_seqlens=cu_seqlens)
        x = x + self.o(qn.attention(q, k, v, causal=True, cu_seqlens=cu_seqlens).flatten(-2))
        h = self.norm_mlp(x)
        return x + self.down(torch.nn.functional.silu(self.gate(h)) * self.up(h))


def offsets(lengths):
    """int32 device offsets of packed examples."""
    ends = torch.cumsum(torch.tensor([0, *lengths]), 0)
    return ends.to(torch.int32).cuda()


def train(block, x, target, cu_seqlens, steps, lr=2e-3, max_norm=0.3, report=print, bits=None):
    """Returns the loss of each step, and the gradients' norms before clipping.
    bits: of the optimizer's states (32 or 8: this package's AdamW, which clips
    within its step and keeps fp32 masters; None: torch's)."""
    params = [p for p in block.parameters() if p.requires_grad]
    if bits is None:
        opt = torch.optim.AdamW(params, lr=lr, weight_decay=0.0)
    else:
        opt = qn.AdamW(params, lr=lr, weight_decay=0.0, bits=bits, max_norm=max_norm, masters=True)
    losses, norms = [], []
    for step in range(steps):
        opt.zero_grad(set_to_none=True)
        y = block(x, cu_seqlens)
        loss = (y.float() - target).square().mean()
        loss.backward()
        if bits is None:
            norms.append(qn.clip_grad_norm([p.grad for p in params], max_norm))
        opt.step()
        if bits is not None:
            norms.append(opt.last_norm)
        losses.append(loss.detach())
        report(f"step {step}: loss {float(losses[-1]):.5f}, gradient norm {float(norms[-1]):.4f}")
    return [float(v) for v in losses], [float(v) for v in norms]


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=1500)
    ap.add_argument("--rope", action="store_true", help="rotary positions of q and k")
    ap.add_argument("--adamw", choices=("torch", "32", "8"), default="torch",
                    help="AdamW: torch's, or this package's with 32- or 8-bit states")
    a = ap.parse_args()
    lengths = [a.tokens // 2, a.tokens // 3, a.tokens - a.tokens // 2 - a.tokens // 3]
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.tokens, 512, generator=g, device="cuda").bfloat16()
    cu = offsets(lengths)
    block = Block(rope=a.rope)
    with torch.no_grad():
        target = Block(seed=7, rope=a.rope)(x, cu).float()
    train(block, x, target, cu, a.steps, bits=None if a.adamw == "torch" else int(a.adamw))


if __name__ == "__main__":
    main()
