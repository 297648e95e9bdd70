"""The layer oracle against independent statements: gradients against central differences,
the checkpoint against its definition's bounds and hand-worked values."""
import numpy as np
import pytest

from oracle import layer_oracle as O


def rng(seed=0):
    return np.random.default_rng(seed)


@pytest.mark.parametrize("name", O.ACTS)
def test_activation_slope_is_the_derivative(name):
    z = np.concatenate([np.linspace(-12, 12, 481) + 0.013, [1e-3, -1e-3, 30.0, -30.0]])
    h = 1e-5
    diff = (O.act(z + h, name) - O.act(z - h, name)) / (2 * h)
    # central differences: h^2/6 of the third derivative (below 4 here), 2^-53 |a| / h of rounding
    assert np.all(np.abs(diff - O.act_slope(z, name)) <= 4 * h * h + 2.0 ** -52 * (np.abs(z) + 1) / h)


def test_gelu_tanh_form_is_the_sigmoid_form():
    z = np.linspace(-8, 8, 1001)
    t = 0.5 * z * (1.0 + np.tanh(O.GELU_C * (z + 0.044715 * z ** 3)))
    assert np.all(np.abs(O.act(z, "gelu") - t) <= 1e-14 * (1 + np.abs(z)))


def test_layer_norm_backward_is_the_derivative():
    r = rng(1)
    x, w, b, dy = r.normal(size=(5, 9)), r.normal(size=9), r.normal(size=9), r.normal(size=(5, 9))
    res = r.normal(size=(5, 9))
    y, mean, rstd = O.layer_norm(x, w, b, 1e-5)
    dx, dw, db = O.layer_norm_backward(dy, x, w, mean, rstd, res)
    h = 1e-6

    def loss(x_, w_, b_):
        return float((O.layer_norm(x_, w_, b_, 1e-5)[0] * dy).sum() + (x_ * res).sum())

    for a, grad, at in ((x, dx, 0), (w, dw, 1), (b, db, 2)):
        for i in np.ndindex(a.shape):
            args = [x.copy(), w.copy(), b.copy()]
            args[at][i] += h
            hi = loss(*args)
            args[at][i] -= 2 * h
            assert abs((hi - loss(*args)) / (2 * h) - grad[i]) < 1e-7


@pytest.mark.parametrize("name", O.ACTS)
def test_linear_gradients_are_derivatives(name):
    r = rng(2)
    x, w, b, dout = r.normal(size=(4, 6)), r.normal(size=(5, 6)), r.normal(size=5), r.normal(size=(4, 3))
    w2 = r.normal(size=(3, 5))  # loss = sum(dout * act(x w^T + b) w2^T)

    def loss(w_):
        return float((O.linear(O.linear(x, w_, b, name, None)[0], w2, None, "none", None)[0] * dout).sum())

    z = O.linear(x, w, b, name, None)[1]
    dz = O.linear_input_grad(dout, w2, z, name, None)
    dw, _ = O.linear_weight_grad(dz, x, "none")
    dw2, _ = O.linear_weight_grad(dout, z, name)
    h = 1e-6
    for i in np.ndindex(w.shape):
        p, m = w.copy(), w.copy()
        p[i] += h
        m[i] -= h
        assert abs((loss(p) - loss(m)) / (2 * h) - dw[i]) < 1e-6
    assert np.allclose(dw2, dout.T @ O.act(z, name), rtol=1e-13, atol=1e-13)


def test_checkpoint_worked():
    # 127 * 2^s fits the step 2^s, 127.5 * 2^s does not; ties go to even
    x = np.array([[127.0, 0.5, 1.5, -2.5] + [0.0] * 28 + [127.5, 1.0, -3.0, 0.0]])
    codes, exps = O.checkpoint_write(x, 32)
    assert exps.tolist() == [[127, 128]]
    assert codes[0, :4].tolist() == [127, 0, 2, -2]
    assert codes[0, 32:].tolist() == [64, 0, -2, 0]  # 63.75, 0.5 and -1.5 at step 2
    assert O.checkpoint_read(codes, exps, 32)[0, 32:].tolist() == [128.0, 0.0, -4.0, 0.0]


@pytest.mark.parametrize("block", [32, 64])
def test_checkpoint_rounds_by_half_a_step_and_reads_as_bf16(block):
    r = rng(3)
    x = (r.normal(size=(7, 150)) * 2.0 ** r.integers(-130, 100, size=(7, 150))).astype(np.float32)
    x[2] = 0.0
    codes, exps = O.checkpoint_write(x, block)
    step = O.checkpoint_steps(exps, 150, block)
    v = O.checkpoint_read(codes, exps, block)
    assert np.all(np.abs(v - x) <= step / 2)
    assert np.abs(codes.astype(int)).max() <= 127
    # no smaller step would do, except at the smallest one
    for b, (lo, hi) in enumerate(O.blocks_of(150, block)):
        top = np.abs(x[:, lo:hi].astype(np.float64)).max(1)
        s = 2.0 ** (exps[:, b].astype(np.float64) - 127)
        assert np.all((exps[:, b] == 1) | (top >= 127.5 * s / 2))
    import torch
    t = torch.from_numpy(v)
    assert torch.equal(t.to(torch.bfloat16).double(), t)  # also where the value is subnormal


def test_checkpoint_of_non_finite_blocks():
    x = np.ones((3, 70))
    x[0, 3], x[1, 40], x[2, 69] = np.inf, np.nan, -np.inf
    codes, exps = O.checkpoint_write(x, 32)
    assert exps.tolist() == [[255, 121, 121], [121, 255, 121], [121, 121, 255]]
    v = O.checkpoint_read(codes, exps, 32)
    assert np.isnan(v[0, :32]).all() and np.isnan(v[1, 32:64]).all() and np.isnan(v[2, 64:]).all()
    assert (v[0, 32:] == 1).all() and (v[2, :64] == 1).all()
