"""Weight gradients kept in fp32 of an activation that is recomputed from its checkpoint."""
import numpy as np
import pytest
import torch

from layer_util import ACT, U, act_bound, assert_near, f64, guarded, random_checkpoint, randn, round_bound
from oracle import layer_oracle as O

pytestmark = pytest.mark.gpu
F32 = torch.float32


@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("rows,n,k", [(1, 8, 8), (90, 70, 150), (1000, 33, 31), (4100, 130, 260), (520, 520, 264)])
def test_two_part_operand(gpu_lib, rows, n, k, accumulate, act):
    """act(z) enters as two bf16 numbers: its rounding, and the rounding of what that leaves
    (at most 2^-8 |a|, so a further 2^-8 of it is lost: 2^-16 |a|).  The two products' sums of k
    exact products each pass through k / 8 additions of the matrix cores, 16 inside an instruction
    and 64 partial sums, of at most two units each; the second is added to the first in fp32."""
    dy = randn(1, rows, n)
    ck = random_checkpoint(2, rows, k, 64)
    out, db = guarded((n, k), F32), guarded((n,), F32)
    start = randn(3, n, k, dtype=F32), randn(4, n, dtype=F32)
    if accumulate:
        out.t.copy_(start[0])
        db.t.copy_(start[1])
    need = gpu_lib.linear_weight_grad_workspace(rows, n, k, ACT[act])
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    gpu_lib.linear_weight_grad(dy, ck, out=out.t, act=ACT[act], dbias=db.t, accumulate=accumulate, workspace=ws)
    torch.cuda.synchronize()
    out.check()
    db.check()
    z = O.checkpoint_read(ck[0].cpu().numpy(), ck[1].cpu().numpy(), 64)
    a, ady = np.abs(O.act(z, act)), np.abs(f64(dy))
    want, wb = O.linear_weight_grad(f64(dy), z, act)
    bound = ady.T @ (2 * (rows / 8 + 80) * U * 1.01 * a + 2.0 ** -16 * a + act_bound(z, 0.0, act))
    if accumulate:
        want, wb = want + f64(start[0]), wb + f64(start[1])
    bound = bound + 4 * U * (np.abs(want) + ady.T @ a)
    assert_near(out.t, want, bound + round_bound(want, F32), "dweight")
    assert_near(db.t, wb, 2 * (rows / 4 + 80) * U * ady.sum(0) + 2 * U * np.abs(wb) + round_bound(wb, F32), "dbias")


@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_large_and_lost_values(gpu_lib, act):
    """A column with activations past bf16's largest number keeps an infinity, as one bf16 operand
    would, and a lost block its NaN; nothing else changes."""
    rows, n, k = 64, 40, 192
    dy, ck = randn(1, rows, n).abs() + 0.5, random_checkpoint(2, rows, k, 64)

    def run():
        out = guarded((n, k), F32)
        ws = torch.empty(gpu_lib.linear_weight_grad_workspace(rows, n, k, ACT[act]), dtype=torch.uint8, device="cuda")
        gpu_lib.linear_weight_grad(dy, ck, out=out.t, act=ACT[act], workspace=ws)
        torch.cuda.synchronize()
        out.check()
        return out.t

    clean = run()
    ck[1][17, 1] = 255
    ck[0][17, 64:128] = 0
    ck[1][3, 0] = 255
    ck[0][3, :64] = 1  # +inf
    out = run()
    assert bool(torch.isnan(out[:, 64:128]).all())
    assert bool((out[:, :64] == float("inf")).all())
    assert torch.equal(out[:, 128:], clean[:, 128:])
