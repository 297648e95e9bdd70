"""The oracle of the step operators against independent statements: gradients against central
differences, AdamW's fp32 form against the textbook's, the 8-bit states against the bounds that
their definition promises."""
import numpy as np
import pytest

from oracle import step_oracle as O


def rng(seed=0):
    return np.random.default_rng(seed)


def bf16(x):
    return (np.asarray(x, np.float32).view(np.uint32) & 0xFFFF0000).view(np.float32)


# -- 8-bit states ---------------------------------------------------------------------------

def test_float8_values_are_torchs():
    import torch
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.fp8_values(), want, equal_nan=True)


@pytest.mark.parametrize("block", [64, 128])
def test_first_moment_is_float8_of_the_scaled_block(block):
    import torch
    x = (rng(1).normal(size=1000) * np.exp(3 * rng(2).normal(size=1000)) * 1e-4).astype(np.float32)
    x[block:2 * block] = 0.0
    codes, exps = O.state_write(x, block, 1)
    for b in range(exps.size):
        v = x[b * block:(b + 1) * block]
        step = 2.0 ** (int(exps[b]) - 127)
        assert np.abs(v).max() <= 448 * step and (exps[b] == 10 or np.abs(v).max() > 224 * step)
        want = torch.from_numpy(v / np.float32(step)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        assert np.array_equal(codes[b * block:(b + 1) * block], want)


@pytest.mark.parametrize("moment", [1, 2])
def test_states_round_trip(moment):
    """Every value that a state can hold is stored as itself."""
    values = O.fp8_values()[:127] * 2.0 ** -20 if moment == 1 else O.second_values(100)
    v = np.concatenate([values, values[::-1]])
    x = np.zeros(512)
    x[:v.size] = v
    codes, exps = O.state_write(x, 512, moment)
    assert np.array_equal(O.state_read(codes, exps, 512, moment), x)


def test_states_rounding():
    r = rng(3)
    x = np.abs(r.normal(size=4096)) * 10.0 ** r.uniform(-12, 0, size=4096)
    # a first moment's largest value is above 224 steps (448 / 2) and its normal numbers start at 2^-6
    # steps, 1 / 14336 of that; a second moment's reach 31 binades below the largest's
    for moment, floor in ((1, 1 / 14336), (2, 2.0 ** -30)):
        got = O.state_read(*O.state_write(x, 256, moment), 256, moment)
        top = np.repeat(x.reshape(-1, 256).max(1), 256)
        normal = x > floor * top
        # half a step of four significant bits
        assert np.all(np.abs(got - x)[normal] <= 2.0 ** -4 * x[normal])
        assert moment == 1 or np.all(got > 0)


def test_states_without_a_finite_value():
    x = np.ones(256)
    x[70] = np.inf
    x[200] = np.nan
    for moment in (1, 2):
        codes, exps = O.state_write(x, 64, moment)
        assert exps.tolist()[1] == exps.tolist()[3] == 255 and not codes[64:128].any()
        got = O.state_read(codes, exps, 64, moment)
        assert np.isnan(got[64:128]).all() and np.isnan(got[192:]).all() and np.all(got[:64] == 1)
    assert O.state_write(np.full(64, 3.4e38), 64, 2)[1][0] == 255
    assert O.state_write(np.full(64, 3.2e38), 64, 2)[1][0] == 254


# -- AdamW -----------------------------------------------------------------------------------

@pytest.mark.parametrize("step,beta2", [(1, 0.999), (7, 0.95), (10 ** 6, 0.99)])
def test_adamw_is_the_textbook_form(step, beta2):
    r = rng(step)
    p, g = r.normal(size=500).astype(np.float32), r.normal(size=500).astype(np.float32)
    m, v = (0.1 * r.normal(size=500)).astype(np.float32), np.abs(r.normal(size=500)).astype(np.float32)
    hp = dict(lr=1e-2, beta1=0.9, beta2=beta2, eps=1e-8, step=step, weight_decay=0.1)
    for got, want, k in zip(O.adamw(p, g, m, v, **hp), O.adamw64(p, g, m, v, **hp), (3, 4, 5)):
        # a few roundings of terms no larger than these (1 - beta2 as a float: 2^-24 relative to itself)
        size = np.abs(want) + np.abs(p) * 0.01 * (k == 3) + (0.9 * np.abs(m) + 0.1 * np.abs(g)) * (k == 4)
        if k == 3:
            size = size + np.abs(p - want) + 1.0
        assert np.all(np.abs(got - want) <= 8 * 2.0 ** -24 * size)


# -- the norms around a block ------------------------------------------------------------------

@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("gate", [None, "column", "element"])
def test_residual_norm_backward_is_the_derivative(post, gate):
    r = rng(4)
    rows, cols, scale, eps = 4, 7, 0.7, 1e-5
    a = {"y": r.normal(size=(rows, cols)), "residual": r.normal(size=(rows, cols)), "weight": r.normal(size=cols),
         "post_weight": r.normal(size=cols) if post else None,
         "gate": None if gate is None else r.normal(size=cols if gate == "column" else (rows, cols))}
    dout, dh = r.normal(size=(rows, cols)), r.normal(size=(rows, cols))

    def loss(**kw):
        b = {**a, **kw}
        out, h, _, _ = O.residual_norm(b["y"], b["residual"], b["weight"], b["post_weight"], b["gate"], scale, eps, post)
        return float((out * dout).sum() + (h * dh).sum())

    _, h, rs, rp = O.residual_norm(a["y"], a["residual"], a["weight"], a["post_weight"], a["gate"], scale, eps, post)
    got = O.residual_norm_backward(dout, dh, h, rs, a["weight"], a["y"], rp, a["post_weight"], a["gate"], scale)
    if gate == "column":
        got["dgate"] = got["dgate"].sum(0)
    step = 1e-6
    for name in a:
        if a[name] is None:
            continue
        grad = got["d" + name]
        for i in np.ndindex(a[name].shape):
            lo, hi = a[name].copy(), a[name].copy()
            lo[i] -= step
            hi[i] += step
            # 2^-52 of sums near 50, over the step; step^2 of third derivatives below 1e3
            assert abs((loss(**{name: hi}) - loss(**{name: lo})) / (2 * step) - grad[i]) <= 1e-7, (name, i)


def test_residual_norm_alone_is_an_rms_norm():
    x, w = rng(5).normal(size=(3, 8)), rng(6).normal(size=8)
    out, h, r, rp = O.residual_norm(None, x, w, None, None, 1.0, 1e-5, False)
    assert np.array_equal(h, x) and rp is None
    assert np.allclose(out, x / np.sqrt((x ** 2).mean(1) + 1e-5)[:, None] * w, rtol=1e-14)


# -- log probabilities -------------------------------------------------------------------------

def test_token_logprobs_of_known_rows():
    x = np.array([[0.0, 0.0, 0.0, 0.0], [0.0, np.log(3.0), -np.inf, -np.inf], [-np.inf] * 4, [1.0, np.nan, 2.0, 3.0],
                  [0.0, 5.0, 5.0, -1e300]])
    o = O.token_logprobs(x, np.array([1, 0, 2, 0, -5]), 1.0, 3)
    assert np.allclose(o["logprob"][:2], [-np.log(4), -np.log(4)]) and o["logprob"][2] == -np.inf
    assert np.isnan(o["logprob"][3]) and o["logprob"][4] == 0.0
    assert np.allclose(o["entropy"][:2], [np.log(4), np.log(4) - 0.75 * np.log(3)]) and o["entropy"][2] == 0.0
    assert o["top_ids"].tolist() == [[0, 1, 2], [1, 0, 2], [0, 1, 2], [-1, -1, -1], [1, 2, 0]]


def test_token_logprobs_backward_is_the_derivative():
    r = rng(7)
    x, scale = 2 * r.normal(size=(3, 6)), 0.6
    t, dl, de = np.array([2, -1, 5]), r.normal(size=3), r.normal(size=3)
    got = O.token_logprobs_backward(x, t, scale, dl, de)

    def loss(x):
        o = O.token_logprobs(x, t, scale, 0)
        return float((dl * o["logprob"] + de * o["entropy"]).sum())

    for i in np.ndindex(x.shape):
        lo, hi = x.copy(), x.copy()
        lo[i] -= 1e-6
        hi[i] += 1e-6
        assert abs((loss(hi) - loss(lo)) / 2e-6 - got[i]) <= 1e-8
    masked = x.copy()
    masked[:, 3] = -np.inf
    g = O.token_logprobs_backward(masked, t, scale, dl, de)
    assert np.all(g[:, 3] == 0) and np.isfinite(g).all()
