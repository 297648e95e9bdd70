"""The slopes that linear_input_grad multiplies by, over every value a checkpoint can hold, and
blocks that were lost to an overflow."""
import numpy as np
import pytest
import torch

from layer_util import ACT, U, assert_near, f64, guarded, random_checkpoint, randn, slope_bound
from oracle import layer_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def every_checkpoint():
    """All 256 codes at all 256 steps, [256, 256] in blocks of 64: z from 2^-133 past 16, 87 and
    1e12 up to the infinities, and NaN where the byte is 255 and the code 0."""
    codes = torch.arange(-128, 128, dtype=torch.int16).to(torch.int8).repeat(256, 1).cuda()
    exps = torch.arange(256, dtype=torch.int16).to(torch.uint8)[:, None].repeat(1, 4).cuda()
    return codes, exps


@pytest.mark.parametrize("act", sorted(set(ACT) - {"none"}))
def test_slope_of_every_value(gpu_lib, act):
    """dy W is exactly 1 everywhere, so an fp32 dx is the slope itself.  Past |x| = 100 of the
    sigmoid's argument x the slope is 0 or 1 to within 100 e^-100 < 2^-135; near 0 the kernel's
    exponential is 0 below 2^-126 and its factor z at most 88 there: 2^-119 covers both."""
    codes, exps = every_checkpoint()
    dy, w = torch.zeros(256, 8, dtype=BF, device="cuda"), torch.zeros(8, 256, dtype=BF, device="cuda")
    dy[:, 0], w[0] = 1.0, 1.0
    out = guarded((256, 256), F32)
    need = gpu_lib.linear_input_grad_workspace(256, 8, 256)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    gpu_lib.linear_input_grad(dy, w, out=out.t, act=ACT[act], checkpoint=(codes, exps), block=64, workspace=ws)
    torch.cuda.synchronize()
    out.check()
    got = f64(out.t)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        z = O.checkpoint_read(codes.cpu().numpy(), exps.cpu().numpy(), 64).astype(np.float32).astype(np.float64)
        want = O.act_slope(z, act)
        x = np.abs(O.act_arg(z, act))
        bound = np.where(x < 100, slope_bound(z, act), 8 * U * np.abs(want)) + 2.0 ** -119
    nan, inf = np.isnan(z), np.isinf(z)
    assert nan.sum() == 1 and inf.sum() > 100
    assert np.isnan(got[nan]).all(), "a lost value has a finite slope"
    # at an infinity the formula's inf * 0 is NaN and its limit 0 or 1
    assert (np.isnan(got[inf]) | (got[inf] == np.where(z[inf] > 0, 1.0, 0.0))).all()
    fine = ~nan & ~inf
    assert_near(got[fine], want[fine], np.broadcast_to(bound, z.shape)[fine], act)


@pytest.mark.parametrize("act", sorted(set(ACT) - {"none"}))
@pytest.mark.parametrize("rows,n,k,block", [(300, 64, 264, 64), (40, 72, 150, 32), (5, 33, 70, 32)])
def test_lost_blocks(gpu_lib, act, rows, n, k, block):
    """A block written from an overflow (byte 255, codes 0) reads as NaN: its own elements of dx
    are NaN, every other one keeps its bits.  Blocks inside whole tiles and at the ends."""
    dy, w = randn(1, rows, n), randn(2, n, k, scale=n ** -0.5)
    codes, exps = random_checkpoint(3, rows, k, block)

    def run():
        out = guarded((rows, k), BF)
        need = gpu_lib.linear_input_grad_workspace(rows, n, k)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
        gpu_lib.linear_input_grad(dy, w, out=out.t, act=ACT[act], checkpoint=(codes, exps), block=block, workspace=ws)
        torch.cuda.synchronize()
        out.check()
        return out.t

    clean = run()
    last = exps.shape[1] - 1
    lost = torch.zeros(rows, k, dtype=torch.bool, device="cuda")
    for r, b in ((0, 0), (rows // 2, 1), (rows - 1, last)):
        exps[r, b] = 255
        codes[r, b * block:(b + 1) * block] = 0
        lost[r, b * block:(b + 1) * block] = True
    out = run()
    assert bool(torch.isnan(out[lost]).all()), "a lost value gave a finite gradient"
    assert torch.equal(out[~lost], clean[~lost]) and not bool(torch.isnan(out[~lost]).any())
