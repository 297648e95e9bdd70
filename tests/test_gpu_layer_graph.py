"""The layer operators on other streams, in HIP graphs and one after another as a training step
uses them."""
import numpy as np
import pytest
import torch

from layer_util import f64
from oracle import layer_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
T, H, F = 700, 256, 1040


def e(*shape, dtype=BF):
    return torch.empty(*shape, dtype=dtype, device="cuda")


class Block:
    """x -> layer norm -> product, GELU -> product + x, forward and backward, from the 8-bit
    checkpoints of the norm's output and of the pre-activation."""

    def __init__(self, lib, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def randn(*shape, scale=1.0):
            return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF)

        self.lib = lib
        self.x, self.dout = randn(T, H), randn(T, H, scale=0.01)
        self.gamma, self.beta = randn(H, scale=0.1) + 1, randn(H, scale=0.1)
        self.w1, self.b1, self.w2, self.b2 = randn(F, H, scale=H ** -0.5), randn(F), randn(H, F, scale=F ** -0.5), randn(H)
        self.y, self.a, self.out = e(T, H), e(T, F), e(T, H)
        self.mean, self.rstd = e(T, dtype=F32), e(T, dtype=F32)
        self.cy = (e(T, H, dtype=torch.int8), e(T, -(-H // 64), dtype=torch.uint8))
        self.cz = (e(T, F, dtype=torch.int8), e(T, -(-F // 64), dtype=torch.uint8))
        self.dz, self.dy, self.dx = e(T, F), e(T, H), e(T, H)
        self.dw1, self.db1, self.dw2, self.db2 = e(F, H), e(F), e(H, F), e(H)
        self.dgamma, self.dbeta = e(H), e(H)
        need = max(lib.linear_workspace(T, F, H), lib.linear_workspace(T, H, F), lib.linear_input_grad_workspace(T, H, F),
                   lib.linear_input_grad_workspace(T, F, H), lib.linear_weight_grad_workspace(T, F, H),
                   lib.linear_weight_grad_workspace(T, H, F, lib.LOCO_ACT_GELU), lib.layer_norm_backward_workspace(T, H))
        self.ws = e(need, dtype=torch.uint8)

    def step(self):
        lib, ws, gelu = self.lib, self.ws, self.lib.LOCO_ACT_GELU
        lib.layer_norm(self.x, self.gamma, self.beta, out=self.y, mean=self.mean, rstd=self.rstd, checkpoint=self.cy)
        lib.linear(self.y, self.w1, bias=self.b1, act=gelu, out=self.a, checkpoint=self.cz, workspace=ws)
        lib.linear(self.a, self.w2, bias=self.b2, residual=self.x, out=self.out, workspace=ws)
        lib.linear_weight_grad(self.dout, self.cz, act=gelu, out=self.dw2, dbias=self.db2, workspace=ws)
        lib.linear_input_grad(self.dout, self.w2, act=gelu, checkpoint=self.cz, out=self.dz, workspace=ws)
        lib.linear_weight_grad(self.dz, self.cy, out=self.dw1, dbias=self.db1, workspace=ws)
        lib.linear_input_grad(self.dz, self.w1, out=self.dy, workspace=ws)
        lib.layer_norm_backward(self.dy, self.x, self.gamma, self.mean, self.rstd, dx=self.dx, dweight=self.dgamma,
                                dbias=self.dbeta, residual=self.dout, workspace=ws)

    def results(self):
        return [t.clone() for t in (self.out, self.dx, self.dw1, self.db1, self.dw2, self.db2, self.dgamma, self.dbeta,
                                    *self.cy, *self.cz)]


def equal(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


def test_block_gradients(gpu_lib):
    """The block's gradients against the 64-bit formulas on unrounded intermediates.  Rounding each
    of the chain's tensors to bf16 (2^-9 of a value at random, root mean square) and each
    checkpoint to 8 bits (steps of 1/64 to 1/127.5 of a block's largest value, about 3 times
    the root mean square: an error of about 1% of it) leaves each gradient within 5% in norm."""
    b = Block(gpu_lib)
    b.step()
    y, mean, rstd = O.layer_norm(f64(b.x), f64(b.gamma), f64(b.beta), 1e-5)
    a, z = O.linear(y, f64(b.w1), f64(b.b1), "gelu", None)
    out, _ = O.linear(a, f64(b.w2), f64(b.b2), "none", f64(b.x))
    dw2, db2 = O.linear_weight_grad(f64(b.dout), z, "gelu")
    dz = O.linear_input_grad(f64(b.dout), f64(b.w2), z, "gelu", None)
    dw1, db1 = O.linear_weight_grad(dz, y, "none")
    dy = O.linear_input_grad(dz, f64(b.w1), None, "none", None)
    dx, dg, dbt = O.layer_norm_backward(dy, f64(b.x), f64(b.gamma), mean, rstd, f64(b.dout))
    for got, want in ((b.out, out), (b.dw2, dw2), (b.db2, db2), (b.dw1, dw1), (b.db1, db1), (b.dx, dx), (b.dgamma, dg),
                      (b.dbeta, dbt)):
        assert np.linalg.norm(f64(got) - want) <= 0.05 * np.linalg.norm(want)


def test_other_streams(gpu_lib):
    """The same bits on a side stream, given by the context or by argument, and with two streams at
    work at once."""
    want = Block(gpu_lib)
    want.step()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    b1, b2 = Block(gpu_lib), Block(gpu_lib)
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(s1):
            b1.step()
        with torch.cuda.stream(s2):
            b2.step()
    s1.synchronize()
    s2.synchronize()
    assert equal(b1.results(), want.results()) and equal(b2.results(), want.results())
    out = e(T, H)
    torch.cuda.synchronize()
    gpu_lib.linear(b1.a, b1.w2, bias=b1.b2, residual=b1.x, out=out, workspace=b1.ws, stream=s1)
    s1.synchronize()
    assert torch.equal(out, want.out)


def test_graph(gpu_lib):
    """A captured step, replayed with fresh inputs and eager work and synchronisations between the
    replays, equals the eager step bit for bit."""
    b, twin = Block(gpu_lib), Block(gpu_lib)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step()
    for i in range(4):
        x = (torch.randn(T, H, generator=torch.Generator("cuda").manual_seed(100 + i), device="cuda") * (1 + i)).to(BF)
        b.x.copy_(x)
        twin.x.copy_(x)
        graph.replay()
        twin.step()
        torch.cuda.synchronize()
        assert equal(b.results(), twin.results())
        torch.randn(1 << 16, device="cuda").sum().item()
