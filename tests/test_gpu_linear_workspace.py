"""Up to 16 rows without a checkpoint run in one launch and need no scratch memory."""
import pytest
import torch

from layer_util import f64, guarded, assert_near, randn, round_bound
from test_gpu_linear import product_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rows,n,k", [(16, 1001, 1003), (1, 4096, 4096), (3, 17, 63)])
def test_few_rows_without_a_workspace(gpu_lib, rows, n, k):
    x, w = randn(1, rows, k), randn(2, n, k, scale=k ** -0.5)
    out = guarded((rows, n), torch.bfloat16)
    gpu_lib.linear(x, w, out=out.t)
    torch.cuda.synchronize()
    out.check()
    want = f64(x) @ f64(w).T
    assert_near(out.t, want, product_bound(f64(x), f64(w).T, k) + round_bound(want, torch.bfloat16), "out")
