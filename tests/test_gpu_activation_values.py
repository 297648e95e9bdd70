"""GELU and SiLU in fp32 where the activation is of the order of its argument, within a bound
that counts each rounding."""
import numpy as np
import pytest
import torch

from layer_util import ACT, U, assert_near, f64, guarded, randn
from oracle import layer_oracle as O

pytestmark = pytest.mark.gpu
F32 = torch.float32


def value_bound(z, name):
    """z * s, s = 1 / (1 + t), t = 2^y, y = -x log2(e).  y has the rounding of the product and of the
    constant, each half a step of |y| < 1.45 |x|: 2 * 1.45 U |x|, which ln 2 turns into 2.01 U |x| of
    t's relative error; exp2 adds one unit in the last place, 2 U.  s takes a share 1 - s of t's
    error, a rounding of 1 + t (U), the reciprocal's last place (2 U) and the product with z (U).
    GELU's x = z (c1 z^2 + c2) has six of its own on the cubic term (three in c1, the products with
    z and the multiply-add), each of at most U |x|."""
    x = np.abs(O.act_arg(z, name))
    q = 1.0 / (1.0 + np.exp(O.act_arg(z, name)))
    return ((2.01 * x + 2 + (6 * x if name == "gelu" else 0)) * q + 4) * U * np.abs(O.act(z, name)) + 2.0 ** -140


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_read(gpu_lib, act):
    """Every code at steps that put |z| from 2^-12 to 16."""
    codes = torch.arange(-128, 128, dtype=torch.int16).to(torch.int8).repeat(6, 1).cuda()
    exps = torch.tensor([115, 118, 120, 121, 122, 124], dtype=torch.uint8)[:, None].repeat(1, 4).cuda()
    z = O.checkpoint_read(codes.cpu().numpy(), exps.cpu().numpy(), 64)
    out = guarded((6, 256), F32)
    gpu_lib.checkpoint_read(codes, exps, out=out.t, block=64, act=ACT[act])
    torch.cuda.synchronize()
    out.check()
    assert_near(out.t, O.act(z, act), value_bound(z, act), act)


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_linear(gpu_lib, act):
    """x times the identity: z is x exactly, with fp32 outputs."""
    x = randn(5, 300, 128, scale=1.5)
    w = torch.eye(128, dtype=torch.bfloat16, device="cuda")
    out = guarded((300, 128), F32)
    need = gpu_lib.linear_workspace(300, 128, 128)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    gpu_lib.linear(x, w, out=out.t, act=ACT[act], workspace=ws)
    torch.cuda.synchronize()
    out.check()
    assert_near(out.t, O.act(f64(x), act), value_bound(f64(x), act), act)
