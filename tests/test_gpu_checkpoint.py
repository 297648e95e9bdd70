"""8-bit activation checkpoints, written and read, against the definition."""
import numpy as np
import pytest
import torch

from layer_util import ACT, act_bound, assert_near, f64, guarded, new_checkpoint, randn, round_bound
from oracle import layer_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def write(lib, x, block):
    rows, cols = x.shape
    codes, exps = new_checkpoint(rows, cols, block)
    lib.checkpoint_write(x, codes=codes.t, exps=exps.t, block=block)
    torch.cuda.synchronize()
    codes.check()
    exps.check()
    return codes.t, exps.t


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block", [32, 64])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (5, 31), (4, 32), (3, 33), (2, 63), (3, 64), (9, 65), (7, 1001),
                                       (2, 4096), (333, 100), (1000, 8), (1, 70000)])
def test_write_is_exact(gpu_lib, rows, cols, block, dtype):
    x = randn(rows + cols, rows, cols, dtype=dtype, scale=3.0)
    x *= torch.exp2(torch.randint(-20, 20, (rows, 1), generator=torch.Generator().manual_seed(1))).to(dtype).cuda()
    codes, exps = write(gpu_lib, x, block)
    wc, we = O.checkpoint_write(f64(x), block)
    assert np.array_equal(exps.cpu().numpy(), we)
    assert np.array_equal(codes.cpu().numpy(), wc)


@pytest.mark.parametrize("block", [32, 64])
def test_write_hard_values(gpu_lib, block):
    """The border between two steps and its neighbours, exact ties, zeros of both signs, subnormal
    and largest values, infinities and NaNs."""
    rows = []
    for s in (-140, -133, -126, -120, -60, 0, 7, 100, 120):
        edge = np.float32(127.5 * 2.0 ** s) if s > -149 + 8 else np.float32(2.0 ** s)
        for top in (edge, np.nextafter(edge, np.float32(0)), np.nextafter(edge, np.float32(np.inf))):
            r = np.zeros(96, np.float32)
            r[:64] = (np.arange(64, dtype=np.float64) - 31.5) * float(top) / 127.5
            r[10], r[64], r[70] = top, -top, np.float32(float(top) * 2.5 / 127)
            rows.append(r)
    for bad in (np.inf, -np.inf, np.nan):
        for at in (0, 40, 95):
            r = np.linspace(-1, 1, 96, dtype=np.float32)
            r[at] = bad
            rows.append(r)
    rows += [np.zeros(96, np.float32), np.full(96, -0.0, np.float32), np.full(96, np.finfo(np.float32).max, np.float32),
             np.full(96, -np.finfo(np.float32).max, np.float32), np.full(96, 2.0 ** -149, np.float32)]
    x = np.stack(rows)
    codes, exps = write(gpu_lib, torch.from_numpy(x).cuda(), block)
    wc, we = O.checkpoint_write(x, block)
    assert np.array_equal(exps.cpu().numpy(), we)
    assert np.array_equal(codes.cpu().numpy(), wc)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", sorted(ACT))
def test_read_every_code_and_byte(gpu_lib, act, dtype):
    """All 256 codes at all 256 steps; values are exact, activations within their bound."""
    codes = torch.arange(-128, 128, dtype=torch.int16).to(torch.int8).repeat(256, 1).cuda()
    exps = torch.arange(256, dtype=torch.int16).to(torch.uint8)[:, None].repeat(1, 4).cuda()
    out = guarded((256, 256), dtype)
    gpu_lib.checkpoint_read(codes, exps, out=out.t, block=64, act=ACT[act])
    torch.cuda.synchronize()
    out.check()
    with np.errstate(over="ignore", invalid="ignore"):
        z = O.checkpoint_read(codes.cpu().numpy(), exps.cpu().numpy(), 64)
        z = z.astype(np.float32).astype(np.float64)  # -128 * 2^127 overflows, as any fp32 value of that size does
    if act == "none":
        assert np.array_equal(f64(out.t), z, equal_nan=True)
        return
    fine = np.abs(z) < 1e12  # GELU's cube overflows fp32 past it; its value there is checked apart
    with np.errstate(over="ignore", invalid="ignore"):
        want = np.where(fine, O.act(z, act), 0.0)
        bound = np.where(fine, act_bound(z, 0.0, act), 0.0) + round_bound(want, dtype) + 2.0 ** -126
    got = np.where(fine, f64(out.t), 0.0)
    assert_near(got, want, bound, act)
    big = np.isfinite(z) & ~fine  # there an activation is z, or 0 for z < 0
    want = np.maximum(z, 0.0)
    assert_near(np.where(big, f64(out.t), 0.0), np.where(big, want, 0.0),
                np.where(big, (1 if dtype == BF else 4) * round_bound(want, dtype), 0.0), act)
    assert np.isnan(f64(out.t)[np.isnan(z)]).all()


@pytest.mark.parametrize("block", [32, 64])
@pytest.mark.parametrize("rows,cols", [(1, 1), (5, 31), (3, 33), (9, 65), (7, 1001), (2, 4096), (333, 100)])
def test_read_shapes(gpu_lib, rows, cols, block):
    x = randn(rows * cols, rows, cols, dtype=F32)
    codes, exps = write(gpu_lib, x, block)
    want = O.checkpoint_read(codes.cpu().numpy(), exps.cpu().numpy(), block)
    for dtype in (BF, F32):
        out = guarded((rows, cols), dtype)
        gpu_lib.checkpoint_read(codes, exps, out=out.t, block=block)
        torch.cuda.synchronize()
        out.check()
        assert np.array_equal(f64(out.t), want)


def test_nothing_to_do(gpu_lib):
    for shape in ((0, 64), (5, 0)):
        x = torch.empty(*shape, dtype=BF, device="cuda")
        c = torch.empty(shape, dtype=torch.int8, device="cuda")
        e = torch.empty(shape[0], -(-shape[1] // 64), dtype=torch.uint8, device="cuda")
        gpu_lib.checkpoint_write(x, codes=c, exps=e, block=64)
        gpu_lib.checkpoint_read(c, e, out=x, block=64)


@pytest.mark.parametrize("cols", [16384, 16391])
def test_past_2_31_elements(gpu_lib, cols):
    rows = (1 << 31) // cols + 300
    x = torch.empty(rows, cols, dtype=BF, device="cuda")
    for lo in range(0, rows, 16384):
        x[lo:lo + 16384].normal_(generator=torch.Generator("cuda").manual_seed(lo))
    codes = torch.empty(rows, cols, dtype=torch.int8, device="cuda")
    exps = torch.empty(rows, -(-cols // 64), dtype=torch.uint8, device="cuda")
    gpu_lib.checkpoint_write(x, codes=codes, exps=exps, block=64)
    at = torch.tensor([0, (1 << 31) // cols - 1, (1 << 31) // cols, (1 << 31) // cols + 1, rows - 1]).cuda()
    wc, we = O.checkpoint_write(f64(x[at]), 64)
    assert np.array_equal(exps[at].cpu().numpy(), we) and np.array_equal(codes[at].cpu().numpy(), wc)
    gpu_lib.checkpoint_read(codes, exps, out=x, block=64)
    assert np.array_equal(f64(x[at]), O.checkpoint_read(wc, we, 64))
