"""The products' fp32 results over a whole matrix in the root mean square: split contractions, the
second launch, the few-rows kernel and rows that are copied keep fp32 sums throughout."""
import numpy as np
import pytest
import torch

from layer_util import f64, guarded, random_checkpoint, randn
from oracle import layer_oracle as O
from precision_util import product_rms_bound, rms

pytestmark = pytest.mark.gpu
F32 = torch.float32


def scratch(nbytes):
    return torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None


def check(got, a, b):
    want = a @ b
    err, bound = rms(f64(got) - want), product_rms_bound(a, b, want)
    assert err <= bound, (err, bound)


# rows, out features, in features, whether partial sums have to pass through memory
SIZES = [(16, 64, 8192, True), (128, 64, 16384, True), (1000, 264, 4104, True), (4100, 4104, 520, False),
         (2056, 8200, 520, False), (16, 1000, 4096, False), (3, 4001, 2047, False), (301, 333, 4099, False)]


@pytest.mark.parametrize("rows,n,k,split", SIZES)
def test_linear(gpu_lib, rows, n, k, split):
    x, w, out = randn(1, rows, k), randn(2, n, k, scale=k ** -0.5), guarded((rows, n), F32)
    need = gpu_lib.linear_workspace(rows, n, k)
    assert need >= 2 * rows * n * 4 or not split
    gpu_lib.linear(x, w, out=out.t, workspace=scratch(need))
    torch.cuda.synchronize()
    out.check()
    check(out.t, f64(x), f64(w).T)


@pytest.mark.parametrize("rows,k,n,split", SIZES)
def test_input_grad(gpu_lib, rows, n, k, split):
    dy, w, out = randn(1, rows, n), randn(2, n, k, scale=n ** -0.5), guarded((rows, k), F32)
    need = gpu_lib.linear_input_grad_workspace(rows, n, k)
    assert need >= 2 * rows * k * 4 or not split
    gpu_lib.linear_input_grad(dy, w, out=out.t, workspace=scratch(need))
    torch.cuda.synchronize()
    out.check()
    check(out.t, f64(dy), f64(w))


@pytest.mark.parametrize("n,k,rows,split", SIZES)
def test_weight_grad(gpu_lib, rows, n, k, split):
    dy, ck, out = randn(1, rows, n), random_checkpoint(2, rows, k, 64), guarded((n, k), F32)
    gpu_lib.linear_weight_grad(dy, ck, out=out.t,
                               workspace=scratch(gpu_lib.linear_weight_grad_workspace(rows, n, k)))
    torch.cuda.synchronize()
    out.check()
    check(out.t, f64(dy).T, O.checkpoint_read(ck[0].cpu().numpy(), ck[1].cpu().numpy(), 64))
