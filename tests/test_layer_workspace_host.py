"""What a product asks for as its workspace is what the kernel it takes uses.  No GPU: the
pointers are fake and never dereferenced, and a call that passes its checks ends at the launch."""
import ctypes

import pytest
import torch

if torch.cuda.is_available():
    pytest.skip("host-only validation tests (fake device pointers)", allow_module_level=True)

from bit_gradient_compression_amd import loco  # noqa: E402

INV, HIP = loco.LOCO_ERR_INVALID, loco.LOCO_ERR_HIP
P = [0x100000000 * (i + 1) for i in range(12)]


def linear(rows, n, k, ws, nws, ckpt=None):
    return loco.load().loco_linear(P[0], P[1], None, None, rows, n, k, 0, P[4], loco.LOCO_BF16, ckpt, ws, nws, None)


@pytest.mark.parametrize("rows,n,k", [(16, 1001, 1003), (16, 4096, 4096), (1, 64, 8)])
def test_few_rows_need_none(rows, n, k):
    """The one-launch kernel of few rows takes no scratch memory (LOCO_ERR_HIP: every check passed);
    with a checkpoint the tiles take the call, within what the size function states."""
    assert linear(rows, n, k, None, 0) == HIP
    need = loco.linear_workspace(rows, n, k)
    ck = ctypes.byref(loco.Checkpoint(P[8], P[9], 64))
    assert linear(rows, n, k, P[5], need, ck) == HIP
    if need:
        assert linear(rows, n, k, P[5], need - 1, ck) == INV


@pytest.mark.parametrize("rows,n,k", [(17, 1001, 1003), (16, 4097, 4099), (128, 64, 16384)])
def test_tiles_need_theirs(rows, n, k):
    need = loco.linear_workspace(rows, n, k)
    assert need > 0
    assert linear(rows, n, k, None, 0) == INV and linear(rows, n, k, P[5], need - 1) == INV
    assert linear(rows, n, k, P[5], need) == HIP
