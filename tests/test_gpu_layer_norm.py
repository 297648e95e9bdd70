"""Layer norm, forward and backward, against the 64-bit oracle."""
import numpy as np
import pytest
import torch

from layer_util import U, Guarded, assert_near, check_checkpoint, f64, guarded, new_checkpoint, randn, round_bound
from oracle import layer_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

SHAPES = [(1, 1), (3, 7), (5, 64), (6, 511), (4, 512), (7, 513), (9, 1000), (3, 1024), (5, 1025), (5, 2047),
          (2, 2048), (5, 4096), (2, 4097), (2, 8192), (3, 9001), (3, 14336), (2, 16384)]


def seq(cols):
    """Additions a term of a row's sum passes through: a lane's own chunks, then lanes and waves."""
    return cols / 512 + 24


def forward_bounds(x, w, b, eps, y, mean, rstd):
    """Errors of y, mean and rstd: the mean's is that of a sum of |x|; the variance is formed about
    the computed mean, whose own error enters squared."""
    ax = np.abs(x).mean(1)
    dm = 2 * (seq(x.shape[1]) + 2) * U * ax
    var = 1.0 / rstd ** 2
    dr = rstd * (2 * (seq(x.shape[1]) + 6) * U + dm ** 2 / var)
    xh = np.abs(x - mean[:, None]) * rstd[:, None]
    aw = 1.0 if w is None else np.abs(w)
    ab = 0.0 if b is None else np.abs(b)
    dy = aw * (xh * (dr / rstd)[:, None] + (rstd * dm)[:, None] + 4 * U * xh) + 2 * U * (np.abs(y) + ab)
    return dy, dm + 2.0 ** -149, dr


def run_forward(lib, x, w, b, eps=1e-5, block=0):
    rows, cols = x.shape
    y, mean, rstd = guarded((rows, cols), x.dtype), guarded((rows,), F32), guarded((rows,), F32)
    ck = new_checkpoint(rows, cols, block) if block else None
    lib.layer_norm(x, w, b, out=y.t, mean=mean.t, rstd=rstd.t, eps=eps,
                   checkpoint=(ck[0].t, ck[1].t) if ck else None, block=block or 64)
    torch.cuda.synchronize()
    for g in (y, mean, rstd) + (ck or ()):
        g.check()
    return y.t, mean.t, rstd.t, ck


def check_forward(lib, x, w, b, eps=1e-5, block=0):
    y, mean, rstd, ck = run_forward(lib, x, w, b, eps, block)
    w64, b64 = (None if t is None else f64(t) for t in (w, b))
    wy, wm, wr = O.layer_norm(f64(x), w64, b64, eps)
    dy, dm, dr = forward_bounds(f64(x), w64, b64, eps, wy, wm, wr)
    assert_near(y, wy, dy + round_bound(wy, x.dtype), "y")
    assert_near(mean, wm, dm, "mean")
    assert_near(rstd, wr, dr, "rstd")
    if ck:
        check_checkpoint(ck[0].t, ck[1].t, block, wy, dy + U * np.abs(wy))


@pytest.mark.parametrize("dtype,param", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(gpu_lib, rows, cols, dtype, param):
    x = randn(rows * 31 + cols, rows, cols, dtype=dtype, scale=2.0, shift=0.5)
    w, b = randn(1, cols, dtype=param, shift=1.0), randn(2, cols, dtype=param)
    check_forward(gpu_lib, x, w, b, block=[0, 32, 64][(rows + cols) % 3])


@pytest.mark.parametrize("block", [32, 64])
@pytest.mark.parametrize("cols", [1, 31, 32, 33, 64, 65, 100, 1023, 4096, 5000])
def test_forward_checkpoint(gpu_lib, cols, block):
    check_forward(gpu_lib, randn(cols, 6, cols), randn(1, cols), randn(2, cols), block=block)


def test_forward_without_weight_or_bias(gpu_lib):
    x = randn(5, 4, 777, dtype=F32)
    check_forward(gpu_lib, x, None, None)
    check_forward(gpu_lib, x, randn(1, 777), None)
    check_forward(gpu_lib, x, None, randn(1, 777, dtype=F32))


def test_forward_hard_rows(gpu_lib):
    """A constant row (variance 0), a large common offset, tiny and huge values, one column."""
    x = randn(3, 6, 2048, dtype=F32)
    x[0] = 3.0
    x[1] += 1e4
    x[2] *= 1e-18
    x[3] *= 1e15
    x[4] = 0.0
    check_forward(gpu_lib, x, None, None)
    check_forward(gpu_lib, x[:, :1].contiguous(), None, None)


def test_forward_non_finite_rows_stay_alone(gpu_lib):
    for cols in (300, 2000, 9000):
        x = randn(4, 9, cols)
        clean = run_forward(gpu_lib, x, None, None, block=64)
        x[2, cols // 2] = float("nan")
        x[5, 0] = float("inf")
        y, mean, rstd, ck = run_forward(gpu_lib, x, None, None, block=64)
        bad = torch.tensor([2, 5], device="cuda")
        ok = torch.tensor([0, 1, 3, 4, 6, 7, 8], device="cuda")
        assert bool(torch.isnan(y[bad]).all()) and bool(torch.isnan(rstd[bad]).all())
        assert torch.equal(y[ok], clean[0][ok]) and torch.equal(mean[ok], clean[1][ok])
        assert bool((ck[1].t[bad] == 255).all()) and bool((ck[0].t[bad] == 0).all())
        assert torch.equal(ck[0].t[ok], clean[3][0].t[ok]) and torch.equal(ck[1].t[ok], clean[3][1].t[ok])


# -- backward ---------------------------------------------------------------------------

def run_backward(lib, dy, x, w, mean, rstd, residual, grad, sums=(True, True)):
    rows, cols = x.shape
    dx = guarded((rows, cols), x.dtype)
    dw, db = (guarded((cols,), grad) if s else None for s in sums)
    need = lib.layer_norm_backward_workspace(rows, cols)
    ws = Guarded((need,), torch.uint8, 0xCC)
    lib.layer_norm_backward(dy, x, w, mean, rstd, dx=dx.t, dweight=dw.t if dw else None, dbias=db.t if db else None,
                            residual=residual, workspace=ws.t if any(sums) else None)
    torch.cuda.synchronize()
    for g in (dx, dw, db, ws):
        if g is not None:
            g.check()
    return dx.t, dw.t if dw else None, db.t if db else None


def backward_bounds(dy, x, w, mean, rstd, rows):
    """Roundings of g, xh and the two sums; the column sums pass each term through at most
    rows (a group's own) + 64 (the join) additions."""
    cols = x.shape[1]
    r = rstd[:, None]
    xh = np.abs((x - mean[:, None]) * r)
    g = np.abs(dy * (1.0 if w is None else w))
    k = 2 * (seq(cols) + 12) * U
    ddx = r * k * (g + g.mean(1, keepdims=True) + xh * (g * xh).mean(1, keepdims=True))
    per = rows / 256 + 64
    return ddx, 2 * (per + 4) * U * (np.abs(dy) * xh).sum(0), 2 * per * U * np.abs(dy).sum(0)


def check_backward(lib, rows, cols, dtype, param, grad, residual, seed=7, affine=True):
    x = randn(seed, rows, cols, dtype=dtype, scale=1.5, shift=0.3)
    dy = randn(seed + 1, rows, cols, dtype=dtype, scale=1e-3)
    w = randn(seed + 2, cols, dtype=param, shift=1.0) if affine else None
    res = randn(seed + 3, rows, cols, dtype=dtype, scale=1e-3) if residual else None
    _, m, r = O.layer_norm(f64(x), None, None, 1e-5)
    mean, rstd = torch.from_numpy(m).float().cuda(), torch.from_numpy(r).float().cuda()
    dx, dw, db = run_backward(lib, dy, x, w, mean, rstd, res, grad)
    args = f64(dy), f64(x), None if w is None else f64(w), f64(mean), f64(rstd)
    wx, ww, wb = O.layer_norm_backward(*args, None if res is None else f64(res))
    bx, bw, bb = backward_bounds(*args, rows)
    bx = bx + (0 if res is None else 2 * U * np.abs(f64(res)))
    assert_near(dx, wx, bx + round_bound(wx, dtype), "dx")
    assert_near(dw, ww, bw + round_bound(ww, grad), "dweight")
    assert_near(db, wb, bb + round_bound(wb, grad), "dbias")


@pytest.mark.parametrize("dtype,param,grad", [(BF, BF, BF), (F32, F32, F32), (BF, F32, F32), (F32, BF, BF)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(gpu_lib, rows, cols, dtype, param, grad):
    check_backward(gpu_lib, rows, cols, dtype, param, grad, residual=(rows + cols) % 2 == 0)


@pytest.mark.parametrize("rows,cols", [(1, 4096), (4097, 64), (5000, 100), (3001, 520), (2500, 1500), (1500, 4097)])
def test_backward_many_rows(gpu_lib, rows, cols):
    check_backward(gpu_lib, rows, cols, BF, BF, F32, residual=False)


def test_backward_without_weight(gpu_lib):
    check_backward(gpu_lib, 40, 300, F32, F32, F32, residual=True, affine=False)


def test_backward_parts(gpu_lib):
    """Each of dweight and dbias is optional, and the others are what they are with both."""
    dy, x, w = randn(1, 50, 640), randn(2, 50, 640), randn(3, 640)
    mean, rstd = randn(4, 50, dtype=F32, scale=0.1), randn(5, 50, dtype=F32, scale=0.1, shift=1.0)
    dx, dw, db = run_backward(gpu_lib, dy, x, w, mean, rstd, None, BF)
    for sums in ((True, False), (False, True), (False, False)):
        ox, ow, ob = run_backward(gpu_lib, dy, x, w, mean, rstd, None, BF, sums)
        assert torch.equal(ox, dx)
        assert ow is None or torch.equal(ow, dw)
        assert ob is None or torch.equal(ob, db)


def test_no_rows(gpu_lib):
    x = torch.empty(0, 96, dtype=BF, device="cuda")
    s = torch.empty(0, device="cuda")
    gpu_lib.layer_norm(x, None, None, out=x.clone(), mean=s, rstd=s.clone())
    dx, dw, db = run_backward(gpu_lib, x, x, None, s, s, None, F32)
    assert bool((dw == 0).all()) and bool((db == 0).all())


def test_past_2_31_elements(gpu_lib):
    """Rows on both sides of element 2^31 and the last ones, forward and backward."""
    cols, rows = 16000, (1 << 31) // 16000 + 5000
    x = torch.empty(rows, cols, dtype=BF, device="cuda")
    for lo in range(0, rows, 16384):
        x[lo:lo + 16384].normal_(generator=torch.Generator("cuda").manual_seed(lo))
    y = torch.empty_like(x)
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    gpu_lib.layer_norm(x, None, None, out=y, mean=mean, rstd=rstd)
    at = torch.tensor([0, (1 << 31) // cols - 1, (1 << 31) // cols, (1 << 31) // cols + 1, rows - 2, rows - 1])
    xs = f64(x[at.cuda()])
    wy, wm, wr = O.layer_norm(xs, None, None, 1e-5)
    dy, dm, dr = forward_bounds(xs, None, None, 1e-5, wy, wm, wr)
    assert_near(y[at.cuda()], wy, dy + round_bound(wy, BF), "y")
    gpu_lib.layer_norm_backward(y, x, None, mean, rstd, dx=(dx := torch.empty_like(x)))
    args = f64(y[at.cuda()]), xs, None, f64(mean[at.cuda()]), f64(rstd[at.cuda()])
    wx, _, _ = O.layer_norm_backward(*args)
    bx, _, _ = backward_bounds(*args, rows)
    assert_near(dx[at.cuda()], wx, bx + round_bound(wx, BF), "dx")
