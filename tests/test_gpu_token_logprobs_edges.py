"""Log probabilities of tokens where two conditions meet, and at the largest vocabulary."""
import numpy as np
import pytest
import torch

from layer_util import U, assert_near, f64, round_bound
from oracle import step_oracle as O
from test_gpu_token_logprobs import (BF, F32, INF, backward_bounds, check_backward, check_forward, forward_bounds,
                                     random_logits)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [5, 2049])
@pytest.mark.parametrize("parts", [dict(), dict(entropy=False), dict(logprob=False)])
def test_rows_without_a_token_and_a_target_past_the_vocabulary(gpu_lib, vocab, dtype, parts):
    """A row of minus infinities, one with a NaN and one of one token, each with a target that is in range, not
    scored or past the vocabulary: that target makes the log probability and the gradient NaN in every row."""
    x = random_logits(1, 12, vocab)
    x[:3] = -INF
    x[3:6, 2] = np.nan
    x[6:9] = -INF
    x[6:9, 1] = 0.5
    t = np.array([1, -1, vocab] * 4)
    t[5], t[8] = vocab + 2 ** 32, 2 ** 62
    if not parts:
        check_forward(gpu_lib, x, dtype, targets=t)
    check_backward(gpu_lib, x, dtype, targets=t, **parts)


@pytest.mark.parametrize("dtype,rows", [(BF, 2), (F32, 1), (BF, 300), (BF, 513)])
def test_the_largest_vocabulary(gpu_lib, dtype, rows):
    """2^24 tokens: one row in pieces, and many, all alike, each by one workgroup; with the most alternatives, and the
    gradient."""
    vocab, top = 1 << 24, 32
    row = torch.from_numpy(random_logits(3, 1, vocab)).to(dtype).cuda()
    row[0, -3:] = 40.0  # the last three, tied
    row[0, 5] = -INF
    x = row.repeat(rows, 1)
    t = torch.full((rows,), vocab - 2, device="cuda")
    lp, ent, st = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda"), torch.empty(rows, 2, device="cuda")
    ids, tops = torch.empty(rows, top, dtype=torch.int32, device="cuda"), torch.empty(rows, top, device="cuda")
    need = gpu_lib.token_logprobs_workspace(rows, vocab, top)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    gpu_lib.token_logprobs(x, t, logprob=lp, entropy=ent, stats=st, top_ids=ids, top_logprobs=tops, scale=0.5, workspace=ws)
    for got in (lp, ent, st, ids, tops):
        assert torch.equal(got, got[:1].expand_as(got))
    x64, t64 = f64(row), np.array([vocab - 2])
    want = O.token_logprobs(x64, t64, 0.5, top)
    bound = forward_bounds(x64, t64, 0.5, want)
    assert np.array_equal(ids[:1].cpu().numpy(), want["top_ids"]) and ids[0, :3].tolist() == [vocab - 3, vocab - 2, vocab - 1]
    for k, got in (("logprob", lp), ("entropy", ent), ("stats", st), ("top_logprobs", tops)):
        assert_near(got[:1], want[k], bound[k] + 2 * U * np.abs(want[k]), k)
    dlp, dh = torch.full((rows,), 0.25, device="cuda"), torch.full((rows,), -0.125, device="cuda")
    st[:], ent[:] = torch.from_numpy(want["stats"]).cuda(), torch.from_numpy(want["entropy"]).cuda()
    gpu_lib.token_logprobs_backward(x, t, st, dlogprob=dlp, entropy=ent, dentropy=dh, dlogits=x, scale=0.5)
    assert all(torch.equal(x[i], x[0]) for i in range(0, rows, 37)) and torch.equal(x[-1], x[0])
    dx = O.token_logprobs_backward(x64, t64, 0.5, np.array([0.25]), np.array([-0.125]))
    b = backward_bounds(x64, t64, 0.5, want, np.array([0.25]), np.array([-0.125]))
    assert_near(x[:1], dx, b + round_bound(dx, dtype), "dlogits")
