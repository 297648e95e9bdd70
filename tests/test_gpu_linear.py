"""The products of a linear layer and their epilogues against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from layer_util import (ACT, HALF, U, Guarded, act_bound, assert_near, check_checkpoint, f64, guarded, new_checkpoint,
                        randn, random_checkpoint, round_bound, slope_bound)
from oracle import layer_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

# rows, out features, in features: one of everything, sizes below, at and past a tile, a step of
# the contraction and a chunk of eight, few tiles with a long contraction, single tokens
SHAPES = [(1, 1, 1), (3, 5, 7), (1, 64, 64), (2, 8, 4104), (17, 130, 72), (128, 128, 64), (129, 257, 193), (64, 96, 1000),
          (300, 320, 520), (16, 64, 8192), (1, 4096, 512), (5, 33, 2049), (257, 264, 136), (512, 512, 256), (33, 1000, 31)]


def product_bound(a, b, k):
    """Error of fp32 sums of k exact products: each passes through k / 8 additions of the matrix
    cores at most, 16 inside one instruction and 64 partial sums."""
    return 2 * (k / 8 + 80) * U * (np.abs(a) @ np.abs(b))


def workspace(nbytes):
    return Guarded((nbytes,), torch.uint8, 0xCC) if nbytes else None


def run_linear(lib, x, w, bias, act, residual, out_dtype=BF, block=0):
    rows, n = x.shape[0], w.shape[0]
    out = guarded((rows, n), out_dtype)
    ck = new_checkpoint(rows, n, block) if block else None
    ws = workspace(lib.linear_workspace(rows, n, x.shape[1]))
    lib.linear(x, w, out=out.t, bias=bias, act=ACT[act], residual=residual,
               checkpoint=(ck[0].t, ck[1].t) if ck else None, block=block or 64, workspace=ws.t if ws else None)
    torch.cuda.synchronize()
    for g in (out, ws) + (ck or ()):
        if g is not None:
            g.check()
    return out.t, ck


def check_linear(lib, rows, n, k, act="none", bias=True, residual=True, out_dtype=BF, block=0, seed=3):
    x, w = randn(seed, rows, k), randn(seed + 1, n, k, scale=max(k, 1) ** -0.5)
    b = randn(seed + 2, n) if bias else None
    res = randn(seed + 3, rows, n) if residual else None
    out, ck = run_linear(lib, x, w, b, act, res, out_dtype, block)
    want, z = O.linear(f64(x), f64(w), None if b is None else f64(b), act, None if res is None else f64(res))
    dz = product_bound(f64(x), f64(w).T, k) + 2 * U * np.abs(z) + (0 if b is None else U * np.abs(f64(b)))
    bound = act_bound(z, dz, act) + 2 * U * np.abs(want) + (0 if res is None else U * np.abs(f64(res)))
    assert_near(out, want, bound + round_bound(want, out_dtype) + 2.0 ** -126, "out")
    if ck:
        check_checkpoint(ck[0].t, ck[1].t, block, z, dz)


@pytest.mark.parametrize("rows,n,k", SHAPES)
def test_linear(gpu_lib, rows, n, k):
    check_linear(gpu_lib, rows, n, k)
    check_linear(gpu_lib, rows, n, k, "gelu", residual=False, block=64, seed=11)
    check_linear(gpu_lib, rows, n, k, "silu", bias=False, out_dtype=F32, block=32, seed=12)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 7, 8, 15, 16, 31, 32, 33, 63, 64, 65, 127])
def test_linear_few_rows(gpu_lib, rows):
    check_linear(gpu_lib, rows, 384, 1024, "relu", block=64)
    check_linear(gpu_lib, rows, 200, 777, "none")


@pytest.mark.parametrize("act", sorted(ACT))
@pytest.mark.parametrize("out_dtype", [BF, F32])
def test_linear_epilogues(gpu_lib, act, out_dtype):
    for bias in (False, True):
        for residual in (False, True):
            for block in (0, 32, 64):
                check_linear(gpu_lib, 70, 150, 96, act, bias, residual, out_dtype, block)


def test_linear_of_no_features(gpu_lib):
    """An empty contraction leaves the bias: out = act(bias) + residual."""
    check_linear(gpu_lib, 5, 40, 0, "gelu", block=32)
    out, _ = run_linear(gpu_lib, randn(1, 0, 64), randn(2, 32, 64), None, "none", None)
    assert out.numel() == 0


def test_linear_non_finite_rows_stay_alone(gpu_lib):
    for rows, n, k in ((150, 200, 100), (9, 100, 72), (300, 264, 1032)):
        x, w = randn(1, rows, k), randn(2, n, k)
        clean, _ = run_linear(gpu_lib, x, w, None, "none", None)
        x[rows // 2, k - 1] = float("nan")
        w[n // 3, 0] = float("inf")
        out, _ = run_linear(gpu_lib, x, w, None, "none", None)
        assert bool(torch.isnan(out[rows // 2]).all())
        keep_r = torch.arange(rows, device="cuda") != rows // 2
        keep_n = torch.arange(n, device="cuda") != n // 3
        assert torch.equal(out[keep_r][:, keep_n], clean[keep_r][:, keep_n])
        assert not bool(torch.isfinite(out[:, n // 3]).any())


# -- input gradient ---------------------------------------------------------------------

def run_input_grad(lib, dy, w, act, ck, residual, out_dtype=BF, block=64):
    rows, k = dy.shape[0], w.shape[1]
    out = guarded((rows, k), out_dtype)
    ws = workspace(lib.linear_input_grad_workspace(rows, w.shape[0], k))
    lib.linear_input_grad(dy, w, out=out.t, act=ACT[act], checkpoint=ck, block=block, residual=residual,
                          workspace=ws.t if ws else None)
    torch.cuda.synchronize()
    out.check()
    if ws:
        ws.check()
    return out.t


def check_input_grad(lib, rows, n, k, act="none", residual=False, out_dtype=BF, block=64, seed=5):
    dy, w = randn(seed, rows, n), randn(seed + 1, n, k, scale=max(n, 1) ** -0.5)
    res = randn(seed + 2, rows, k) if residual else None
    ck = random_checkpoint(seed + 3, rows, k, block) if act != "none" else None
    out = run_input_grad(lib, dy, w, act, ck, res, out_dtype, block)
    z = O.checkpoint_read(ck[0].cpu().numpy(), ck[1].cpu().numpy(), block) if ck else None
    want = O.linear_input_grad(f64(dy), f64(w), z, act, None if res is None else f64(res))
    s = np.abs(f64(dy) @ f64(w))
    bound = product_bound(f64(dy), f64(w), n)
    if ck:
        bound = bound * (np.abs(O.act_slope(z, act)) + 1e-3) + s * slope_bound(z, act)
    bound = bound + 4 * U * np.abs(want) + (0 if res is None else 2 * U * np.abs(f64(res)))
    assert_near(out, want, bound + round_bound(want, out_dtype) + 2.0 ** -126, "dx")


@pytest.mark.parametrize("rows,n,k", SHAPES)
def test_input_grad(gpu_lib, rows, n, k):
    check_input_grad(gpu_lib, rows, n, k, residual=True)
    check_input_grad(gpu_lib, rows, n, k, "gelu", seed=21)
    check_input_grad(gpu_lib, rows, n, k, "silu", True, F32, 32, seed=22)


@pytest.mark.parametrize("rows", [1, 2, 3, 4, 7, 8, 15, 16, 31, 32, 33, 63, 64, 65, 127])
def test_input_grad_few_rows(gpu_lib, rows):
    check_input_grad(gpu_lib, rows, 1024, 384, "relu")
    check_input_grad(gpu_lib, rows, 777, 200)


@pytest.mark.parametrize("act", sorted(ACT))
@pytest.mark.parametrize("block", [32, 64])
def test_input_grad_epilogues(gpu_lib, act, block):
    for residual in (False, True):
        for out_dtype in (BF, F32):
            check_input_grad(gpu_lib, 70, 96, 150, act, residual, out_dtype, block)


def test_input_grad_of_no_features(gpu_lib):
    check_input_grad(gpu_lib, 5, 0, 40, "gelu", True)


# -- weight gradient --------------------------------------------------------------------

def run_weight_grad(lib, dy, ck, k, act, grad, block=64, bias=True, accumulate=None):
    rows, n = dy.shape
    out = guarded((n, k), grad)
    db = guarded((n,), grad) if bias else None
    if accumulate is not None:
        out.t.copy_(accumulate[0])
        if db:
            db.t.copy_(accumulate[1])
    ws = workspace(lib.linear_weight_grad_workspace(rows, n, k, ACT[act]))
    lib.linear_weight_grad(dy, ck, out=out.t, block=block, act=ACT[act], dbias=db.t if db else None,
                           accumulate=accumulate is not None, workspace=ws.t if ws else None)
    torch.cuda.synchronize()
    for g in (out, db, ws):
        if g is not None:
            g.check()
    return out.t, db.t if db else None


def check_weight_grad(lib, rows, n, k, act="none", grad=BF, block=64, accumulate=False, seed=9):
    dy = randn(seed, rows, n)
    ck = random_checkpoint(seed + 1, rows, k, block)
    start = (randn(seed + 2, n, k, dtype=grad), randn(seed + 3, n, dtype=grad)) if accumulate else None
    out, db = run_weight_grad(lib, dy, ck, k, act, grad, block, True, start)
    z = O.checkpoint_read(ck[0].cpu().numpy(), ck[1].cpu().numpy(), block)
    a = O.act(z, act)
    want, wb = O.linear_weight_grad(f64(dy), z, act)
    bound = product_bound(f64(dy).T, a, rows)
    if act not in ("none", "relu"):  # the product's operand is the activation rounded to bf16
        bound = bound + np.abs(f64(dy)).T @ (HALF[BF] * np.abs(a) + act_bound(z, 0.0, act))
    db_bound = 2 * (rows / 4 + 80) * U * np.abs(f64(dy)).sum(0)
    if start:
        want, wb = want + f64(start[0]), wb + f64(start[1])
    assert_near(out, want, bound + 2 * U * np.abs(want) + round_bound(want, grad), "dweight")
    assert_near(db, wb, db_bound + 2 * U * np.abs(wb) + round_bound(wb, grad), "dbias")


@pytest.mark.parametrize("rows,n,k", SHAPES + [(8192, 64, 16), (2049, 33, 5), (4100, 130, 260), (1, 520, 264)])
def test_weight_grad(gpu_lib, rows, n, k):
    check_weight_grad(gpu_lib, rows, n, k)
    check_weight_grad(gpu_lib, rows, n, k, grad=F32, block=32, accumulate=True, seed=31)
    check_weight_grad(gpu_lib, rows, n, k, "gelu", BF, 32, seed=32)


@pytest.mark.parametrize("act", sorted(ACT))
@pytest.mark.parametrize("block", [32, 64])
@pytest.mark.parametrize("grad", [BF, F32])
def test_weight_grad_options(gpu_lib, act, block, grad):
    for accumulate in (False, True):
        check_weight_grad(gpu_lib, 90, 70, 150, act, grad, block, accumulate)


def test_weight_grad_of_no_rows(gpu_lib):
    """No tokens: zero gradients, or what was there where they accumulate."""
    dy = randn(1, 0, 24)
    ck = random_checkpoint(2, 0, 40, 64)
    out, db = run_weight_grad(gpu_lib, dy, ck, 40, "none", F32)
    assert bool((out == 0).all()) and bool((db == 0).all())
    start = (randn(3, 24, 40, dtype=F32), randn(4, 24, dtype=F32))
    out, db = run_weight_grad(gpu_lib, dy, ck, 40, "none", F32, accumulate=start)
    assert torch.equal(out, start[0]) and torch.equal(db, start[1])


def test_weight_grad_without_bias(gpu_lib):
    dy, ck = randn(1, 100, 72), random_checkpoint(2, 100, 136, 64)
    a, _ = run_weight_grad(gpu_lib, dy, ck, 136, "none", BF)
    b, none = run_weight_grad(gpu_lib, dy, ck, 136, "none", BF, bias=False)
    assert none is None and torch.equal(a, b)


def test_weight_grad_of_a_lost_block(gpu_lib):
    """A block written from an overflow reads as NaN and reaches its own columns only."""
    dy, ck = randn(1, 64, 40), random_checkpoint(2, 64, 192, 64)
    clean, _ = run_weight_grad(gpu_lib, dy, ck, 192, "none", BF)
    ck[1][17, 1] = 255
    ck[0][17, 64:128] = 0
    out, _ = run_weight_grad(gpu_lib, dy, ck, 192, "none", BF)
    assert bool(torch.isnan(out[:, 64:128]).all())
    assert torch.equal(out[:, :64], clean[:, :64]) and torch.equal(out[:, 128:], clean[:, 128:])


# -- every tile shape, with rows, columns and k that end inside a tile -------------------

# (m, n, k) of the product: the large tile, the middle one, the small ones with either side
# short, few rows with the contraction split, rows that are not whole chunks and are copied
# or (few) staged through registers
TILES = [(2100, 4200, 136), (4000, 4400, 72), (1000, 1100, 200), (70000, 40, 72), (20, 9000, 1032), (16, 4096, 11008),
         (2100, 4200, 137), (2101, 4201, 515), (701, 700, 65), (260, 264, 4136)]


@pytest.mark.parametrize("m,n,k", TILES)
def test_linear_tiles(gpu_lib, m, n, k):
    check_linear(gpu_lib, m, n, k, "silu", block=32)


@pytest.mark.parametrize("m,n,k", TILES)
def test_input_grad_tiles(gpu_lib, m, n, k):
    check_input_grad(gpu_lib, m, k, n, "gelu", True)


@pytest.mark.parametrize("m,n,k", TILES)
def test_weight_grad_tiles(gpu_lib, m, n, k):
    check_weight_grad(gpu_lib, k, m, n, "none", F32, accumulate=True)


# a few rows without a checkpoint: one launch, columns and k that end inside a block
@pytest.mark.parametrize("act", sorted(ACT))
@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (1, 16, 64), (3, 17, 63), (5, 100, 65), (16, 1001, 1003), (2, 33, 4095),
                                   (9, 250, 577), (16, 4096, 4096), (15, 4096, 200), (16, 4097, 256), (17, 64, 256)])
def test_linear_single_tokens(gpu_lib, m, n, k, act):
    check_linear(gpu_lib, m, n, k, act, block=0)


# just past whole rounds of the large tile: the last rows, or the last columns, in a second launch
TAILS = [(4100, 4104, 520), (2056, 8200, 520), (4400, 4097, 520)]


@pytest.mark.parametrize("m,n,k", TAILS)
def test_linear_tails(gpu_lib, m, n, k):
    check_linear(gpu_lib, m, n, k, "gelu", block=64)


@pytest.mark.parametrize("m,n,k", TAILS)
def test_input_grad_tails(gpu_lib, m, n, k):
    check_input_grad(gpu_lib, m, k, n, "silu", True)


@pytest.mark.parametrize("m,n,k", TAILS)
def test_weight_grad_tails(gpu_lib, m, n, k):
    check_weight_grad(gpu_lib, k, m, n, "relu", BF, accumulate=True)


# -- the calls together -------------------------------------------------------------------------------------------------------------------------------

def test_same_call_same_bits(gpu_lib):
    x, w, b = randn(1, 190, 2100), randn(2, 150, 2100), randn(3, 150)
    first = run_linear(gpu_lib, x, w, b, "gelu", None, block=64)
    dy, ck = randn(4, 3000, 200), random_checkpoint(5, 3000, 136, 64)
    g = run_weight_grad(gpu_lib, dy, ck, 136, "none", F32)
    for _ in range(3):
        again = run_linear(gpu_lib, x, w, b, "gelu", None, block=64)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1][0].t, again[1][0].t)
        h = run_weight_grad(gpu_lib, dy, ck, 136, "none", F32)
        assert torch.equal(g[0], h[0]) and torch.equal(g[1], h[1])


@pytest.mark.parametrize("rows,n,k", [((1 << 32) // 2048 // 2 + 300, 24, 2048), ((1 << 32) // 2048 // 2 + 301, 2056, 8)])
def test_offsets_past_32_bits(gpu_lib, rows, n, k):
    """x, or out, past 2^32 bytes: the first, last and middle rows of the forward product, and the
    input gradient of the same sizes."""
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(rows, k, generator=g, device="cuda", dtype=BF)
    w = torch.randn(n, k, generator=g, device="cuda", dtype=BF)
    out = torch.full((rows, n), float("nan"), device="cuda", dtype=BF)
    need = gpu_lib.linear_workspace(rows, n, k)
    gpu_lib.linear(x, w, out=out, workspace=torch.empty(need, dtype=torch.uint8, device="cuda") if need else None)
    at = torch.tensor([0, 1, rows // 2, (1 << 32) // 2 // max(n, k) - 1, (1 << 32) // 2 // max(n, k), rows - 1]).cuda()
    want = f64(x[at]) @ f64(w).T
    assert_near(out[at], want, product_bound(f64(x[at]), f64(w).T, k) + round_bound(want, BF), "out")
    need = gpu_lib.linear_input_grad_workspace(rows, n, k)
    gpu_lib.linear_input_grad(out, w, out=x, workspace=torch.empty(need, dtype=torch.uint8, device="cuda") if need else None)
    want = f64(out[at]) @ f64(w)
    assert_near(x[at], want, product_bound(f64(out[at]), f64(w), n) + round_bound(want, BF), "dx")
