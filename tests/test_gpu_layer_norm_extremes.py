"""Layer norm's backward pass where (x - mean) * rstd of a missing element would overflow."""
import numpy as np
import pytest
import torch

from layer_util import assert_near, f64, randn, round_bound
from oracle import layer_oracle as O
from test_gpu_layer_norm import backward_bounds, run_backward

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("cols", [1, 7, 8, 64, 100, 513, 1000, 2047, 4097, 9001, 14336])
def test_large_constant_rows(gpu_lib, cols, dtype):
    """Constant rows of 2^120 with eps = 1e-5: mean * rstd is past fp32's largest number, every
    (x - mean) * rstd is 0, and dx = rstd (g - mean g) is finite.  Lanes and chunks past the row's
    end have no x; what they hold must not reach the row's sums."""
    rows = 5
    x = torch.full((rows, cols), 2.0 ** 120, dtype=dtype, device="cuda")
    dy, w = randn(1, rows, cols, dtype=dtype), randn(2, cols, dtype=dtype, shift=1.0)
    mean = torch.full((rows,), 2.0 ** 120, device="cuda")
    rstd = torch.full((rows,), 1e-5 ** -0.5, device="cuda")
    dx, dw, db = run_backward(gpu_lib, dy, x, w, mean, rstd, None, F32)
    args = f64(dy), f64(x), f64(w), f64(mean), f64(rstd)
    wx, ww, wb = O.layer_norm_backward(*args)
    bx, bw, bb = backward_bounds(*args, rows)
    assert_near(dx, wx, bx + round_bound(wx, dtype), "dx")
    assert np.all(ww == 0) and bool((dw == 0).all())
    assert_near(db, wb, bb + round_bound(wb, F32), "dbias")
