"""Train a gated feed-forward block, quantise it to 4 bits and serve it.

    python examples/gated_block.py [--steps 60] [--tokens 2048] [--dim 512] [--hidden 1024]

A student block y = (silu(x Wg^T) * (x Wu^T)) Wd^T learns a fixed random teacher
from its outputs.  Every step runs the block forward and backward
(gated_ffn, gated_ffn_backward), keeps a momentum of each weight gradient and
moves the weights along its orthogonalised form (orthogonalize; the gate and up
halves as a batch of two).  The trained weights are then rounded to 4-bit codes
(w4_quantize), and single tokens go through w4_gated and w4_linear.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_fp16_gemm_04_gb300 as g  # noqa: E402


def block(gen, dim, hidden):
    """fp32 master weights of a block: w_in [2, hidden, dim], w_down [dim, hidden]."""
    return (torch.randn(2, hidden, dim, generator=gen, device="cuda") * dim ** -0.5,
            torch.randn(dim, hidden, generator=gen, device="cuda") * hidden ** -0.5)


def train(steps=60, tokens=2048, dim=512, hidden=1024, lr=0.05, beta=0.9, dtype=torch.float16, seed=0):
    """Returns the losses and the trained 16-bit weights (w_in [2 hidden, dim], w_down)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    teacher = [w.to(dtype) for w in block(gen, dim, hidden)]
    masters = block(gen, dim, hidden)
    momenta = [torch.zeros_like(w) for w in masters]
    losses = []
    for step in range(steps):
        x = torch.randn(tokens, dim, generator=gen, device="cuda").to(dtype)
        want = g.gated_ffn(x, teacher[0].view(2 * hidden, dim), teacher[1])
        w_in, w_down = (w.to(dtype) for w in masters)
        w_in = w_in.view(2 * hidden, dim)
        y, gu = g.gated_ffn(x, w_in, w_down, save=True)
        diff = y.float() - want.float()
        losses.append(diff.square().mean())
        _, dw_in, dw_down = g.gated_ffn_backward(diff.to(dtype), x, w_in, w_down, gu)
        rate = lr * (1 - step / steps)
        for w, m, d in zip(masters, momenta, (dw_in.view(2, hidden, dim), dw_down)):
            m.mul_(beta).add_(d.float())
            # A step of the same size whatever the gradient's: every singular
            # value of the update is about rate * sqrt(rows / columns).
            w.add_(g.orthogonalize(m), alpha=-rate * max(1.0, w.shape[-2] / w.shape[-1]) ** 0.5)
    return torch.stack(losses), masters[0].to(dtype).view(2 * hidden, dim), masters[1].to(dtype)


class W4Block:
    """The block with weights of 4 bits, for a few tokens at a time."""

    def __init__(self, w_in, w_down, group=64):
        self.w_in = g.w4_quantize(w_in, group, zero_point=True)
        self.w_down = g.w4_quantize(w_down, group, zero_point=True)

    def __call__(self, x):
        return g.w4_linear(g.w4_gated(x, *self.w_in), *self.w_down)


def main(argv=None):
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--steps", type=int, default=60)
    p.add_argument("--tokens", type=int, default=2048)
    p.add_argument("--dim", type=int, default=512)
    p.add_argument("--hidden", type=int, default=1024)
    a = p.parse_args(argv)
    losses, w_in, w_down = train(a.steps, a.tokens, a.dim, a.hidden)
    g.default_ops().check_error()
    shown = losses.tolist()
    print("loss %.4f -> %.4f in %d steps" % (shown[0], shown[-1], a.steps))
    served = W4Block(w_in, w_down)
    token = torch.randn(1, a.dim, device="cuda").to(w_in.dtype)
    full, quant = g.gated_ffn(token, w_in, w_down).float(), served(token).float()
    print("one token: 4-bit weights differ from 16-bit ones by %.3f of the output" % float((quant - full).norm() / full.norm()))
    return 0


if __name__ == "__main__":
    sys.exit(main())
