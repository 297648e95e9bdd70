"""Log probabilities of tokens where two conditions meet."""
import numpy as np
import pytest
import torch

from test_gpu_token_logprobs import BF, F32, INF, check_backward, check_forward, random_logits

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
