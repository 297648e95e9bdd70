"""A transformer's MLP block trained on one GPU with the library's own operators, end to end:

  layer norm -> product, GELU -> product + residual      forward, keeping 8-bit checkpoints only
  the same backward                                      into one flat bf16 gradient
  compensate-quantize -> dequant-reduce + Adam           LoCo's low-bit path from that gradient
                                                         to the next step's weights

Of a token's activations the backward pass needs the norm's input (bf16, the residual stream
that is kept anyway), the norm's output and the pre-activation.  The last two are kept as
8-bit checkpoints, at half their bf16 size; the activation itself is recomputed from the
pre-activation's checkpoint.

  python examples/mlp_step.py [--tokens 4096] [--hidden 512] [--inner 2048] [--steps 20]
"""

from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from bit_gradient_compression_amd import loco  # noqa: E402

BF, F32 = torch.bfloat16, torch.float32
BLOCK = 64  # elements per step of a checkpoint


def empty(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def checkpoint(rows, cols):
    return empty(rows, cols, dtype=torch.int8), empty(rows, -(-cols // BLOCK), dtype=torch.uint8)


class MlpBlock:
    """out = x + W2 gelu(W1 norm(x) + b1) + b2.  Parameters and gradients are views of flat
    buffers, as a sharded data-parallel step hands them over; sizes are multiples of 8, so that
    every view starts on 16 bytes."""

    def __init__(self, tokens, hidden, inner, seed=0):
        self.t, self.h, self.f = tokens, hidden, inner
        shapes = {"gamma": (hidden,), "beta": (hidden,), "w1": (inner, hidden), "b1": (inner,), "w2": (hidden, inner),
                  "b2": (hidden,)}
        self.n = sum(torch.Size(s).numel() for s in shapes.values())
        self.master, self.param, self.grad = (empty(self.n, dtype=F32), empty(self.n), empty(self.n))
        gen = torch.Generator("cuda").manual_seed(seed)
        self.p, self.g, at = {}, {}, 0
        for name, shape in shapes.items():
            n = torch.Size(shape).numel()
            view = self.master[at:at + n].view(shape)
            if name in ("w1", "w2"):
                view.normal_(generator=gen).mul_(shape[1] ** -0.5)
            else:
                view.fill_(1.0 if name == "gamma" else 0.0)
            self.p[name], self.g[name] = self.param[at:at + n].view(shape), self.grad[at:at + n].view(shape)
            at += n
        self.param.copy_(self.master)
        self.y, self.a, self.out = empty(tokens, hidden), empty(tokens, inner), empty(tokens, hidden)
        self.mean, self.rstd = empty(tokens, dtype=F32), empty(tokens, dtype=F32)
        self.y8, self.z8 = checkpoint(tokens, hidden), checkpoint(tokens, inner)
        self.dz, self.dy, self.dx = empty(tokens, inner), empty(tokens, hidden), empty(tokens, hidden)
        self.ws = empty(max(loco.linear_workspace(tokens, inner, hidden), loco.linear_workspace(tokens, hidden, inner),
                            loco.linear_input_grad_workspace(tokens, inner, hidden),
                            loco.linear_input_grad_workspace(tokens, hidden, inner),
                            loco.linear_weight_grad_workspace(tokens, inner, hidden),
                            loco.linear_weight_grad_workspace(tokens, hidden, inner, loco.LOCO_ACT_GELU),
                            loco.layer_norm_backward_workspace(tokens, hidden)), dtype=torch.uint8)

    def forward(self, x):
        p = self.p
        loco.layer_norm(x, p["gamma"], p["beta"], out=self.y, mean=self.mean, rstd=self.rstd, checkpoint=self.y8,
                        block=BLOCK)
        loco.linear(self.y, p["w1"], bias=p["b1"], act=loco.LOCO_ACT_GELU, out=self.a, checkpoint=self.z8, block=BLOCK,
                    workspace=self.ws)
        loco.linear(self.a, p["w2"], bias=p["b2"], residual=x, out=self.out, workspace=self.ws)
        return self.out

    def backward(self, x, dout):
        """Fills the flat gradient and returns the gradient of x.  Reads the checkpoints only: y
        and a may have been overwritten by other layers since."""
        p, g, gelu, ws = self.p, self.g, loco.LOCO_ACT_GELU, self.ws
        loco.linear_weight_grad(dout, self.z8, act=gelu, block=BLOCK, out=g["w2"], dbias=g["b2"], workspace=ws)
        loco.linear_input_grad(dout, p["w2"], act=gelu, checkpoint=self.z8, block=BLOCK, out=self.dz, workspace=ws)
        loco.linear_weight_grad(self.dz, self.y8, block=BLOCK, out=g["w1"], dbias=g["b1"], workspace=ws)
        loco.linear_input_grad(self.dz, p["w1"], out=self.dy, workspace=ws)
        loco.layer_norm_backward(self.dy, x, p["gamma"], self.mean, self.rstd, dx=self.dx, dweight=g["gamma"],
                                 dbias=g["beta"], residual=dout, workspace=ws)
        return self.dx


class LocoStep:
    """The low-bit path of the flat gradient on one rank: 4-bit codes with the local error, then
    their average (of one payload here; of every rank's, after the exchange) into Adam."""

    def __init__(self, block, bits=4, scale_block=128):
        self.block, self.bits, self.scale_block = block, bits, scale_block
        n = block.n
        self.err = torch.zeros(n, device="cuda")
        self.codes = empty(loco.code_bytes(n, bits), dtype=torch.uint8)
        self.absmax = empty(loco.num_blocks(n, scale_block), dtype=F32)
        self.m, self.v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")

    def __call__(self, lr):
        b = self.block
        loco.compensate_quantize([(b.grad, self.err, self.codes, self.absmax)], bits=self.bits, block=self.scale_block,
                                 beta=0.9)
        loco.dequant_reduce_adam([(self.codes, self.absmax)], b.n, bits=self.bits, block=self.scale_block, out_scale=1.0,
                                 param=b.master, m=self.m, v=self.v, param_bf16=b.param, lr=lr, beta1=0.1, beta2=0.01,
                                 delta=1e-12)


def train(tokens=4096, hidden=512, inner=2048, steps=20, lr=5e-4, seed=0):
    """Fits the block to another block of the same shape; returns the mean squared error before
    each step."""
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").to(BF)
    target = MlpBlock(tokens, hidden, inner, seed=seed + 2).forward(x).clone()
    block = MlpBlock(tokens, hidden, inner, seed=seed)
    step, losses = LocoStep(block), []
    for _ in range(steps):
        diff = block.forward(x) - target
        losses.append(float(diff.float().square().mean()))
        block.backward(x, diff * (1.0 / tokens))
        step(lr)
    return losses


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, value in (("tokens", 4096), ("hidden", 512), ("inner", 2048), ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=value)
    a = ap.parse_args()
    for i, loss in enumerate(train(a.tokens, a.hidden, a.inner, a.steps)):
        print(f"step {i:3d}  mean squared error {loss:.5f}", flush=True)


if __name__ == "__main__":
    main()
