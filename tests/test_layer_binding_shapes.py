"""The binding's checks of shapes: a matrix laid out the other way round is refused even though
it has as many elements; collapsed leading dimensions and flat storage are not.  Host tensors:
a call that passes the checks of shapes is refused for its memory, and says so."""
import pytest
import torch

from bit_gradient_compression_amd import loco

F32, I8, U8 = torch.float32, torch.int8, torch.uint8


@pytest.fixture(autouse=True)
def no_device(monkeypatch):
    monkeypatch.setattr(loco, "_device", lambda: 0)


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def wrong(fn, *a, **kw):
    with pytest.raises(ValueError, match="shape"):
        fn(*a, **kw)


def right(fn, *a, **kw):
    with pytest.raises(ValueError, match="device memory"):
        fn(*a, **kw)


def norm(x, **kw):
    a = dict(out=t(*x.shape), mean=t(x.shape[0], dtype=F32), rstd=t(x.shape[0], dtype=F32))
    return loco.layer_norm, (x, None, None), {**a, **kw}


def call(check, made):
    check(made[0], *made[1], **made[2])


def test_layer_norm():
    x = t(4, 96)
    call(right, norm(x))
    call(wrong, norm(x, out=t(96, 4)))
    call(wrong, norm(x, checkpoint=(t(96, 4, dtype=I8), t(4, 2, dtype=U8))))
    call(wrong, norm(x, checkpoint=(t(4, 96, dtype=I8), t(2, 4, dtype=U8))))
    call(right, norm(x, checkpoint=(t(4, 96, dtype=I8), t(4, 2, dtype=U8))))
    call(right, norm(x, checkpoint=(t(384, dtype=I8), t(8, dtype=U8))))  # flat storage
    call(right, norm(x, out=t(2, 2, 96)))
    call(right, norm(x, mean=t(4, 1, dtype=F32)))
    x = t(2, 3, 96)
    call(wrong, norm(x, out=t(3, 2, 96), mean=t(6, dtype=F32), rstd=t(6, dtype=F32)))
    call(wrong, norm(x, mean=t(3, 2, dtype=F32), rstd=t(6, dtype=F32)))
    call(right, norm(x, mean=t(2, 3, dtype=F32), rstd=t(2, 3, 1, dtype=F32)))
    call(right, norm(x, out=t(6, 96), mean=t(6, dtype=F32), rstd=t(6, dtype=F32)))


def test_layer_norm_backward():
    x, s = t(4, 96), t(4, dtype=F32)
    right(loco.layer_norm_backward, x, x, None, s, s, dx=x)
    wrong(loco.layer_norm_backward, t(96, 4), x, None, s, s, dx=x)
    wrong(loco.layer_norm_backward, x, x, None, s, s, dx=t(96, 4))
    wrong(loco.layer_norm_backward, x, x, None, s, s, dx=x, residual=t(96, 4))
    y = t(2, 3, 96)
    wrong(loco.layer_norm_backward, y, y, None, t(3, 2, dtype=F32), t(6, dtype=F32), dx=y)


def test_checkpoints():
    x = t(4, 96)
    right(loco.checkpoint_write, x, codes=t(4, 96, dtype=I8), exps=t(4, 2, dtype=U8))
    wrong(loco.checkpoint_write, x, codes=t(96, 4, dtype=I8), exps=t(4, 2, dtype=U8))
    wrong(loco.checkpoint_write, x, codes=t(4, 96, dtype=I8), exps=t(2, 4, dtype=U8))
    wrong(loco.checkpoint_read, t(96, 4, dtype=I8), t(4, 2, dtype=U8), out=x)


def test_products():
    x, w = t(4, 96), t(32, 96)
    right(loco.linear, x, w, out=t(4, 32))
    wrong(loco.linear, x, w, out=t(32, 4))
    wrong(loco.linear, x, w, out=t(4, 32), residual=t(32, 4))
    wrong(loco.linear, t(2, 3, 96), w, out=t(3, 2, 32))
    right(loco.linear, t(2, 3, 96), w, out=t(2, 3, 32))
    right(loco.linear, t(2, 3, 96), w, out=t(6, 32), residual=t(2, 3, 32))
    right(loco.linear, t(96), w, out=t(32))
    dy = t(4, 32)
    right(loco.linear_input_grad, dy, w, out=x)
    wrong(loco.linear_input_grad, dy, w, out=t(96, 4))
    wrong(loco.linear_input_grad, dy, w, out=x, residual=t(96, 4))
    wrong(loco.linear_input_grad, dy, w, out=x, act=2, checkpoint=(t(96, 4, dtype=I8), t(4, 2, dtype=U8)))
    right(loco.linear_weight_grad, dy, (t(4, 96, dtype=I8), t(4, 2, dtype=U8)), out=w)
    wrong(loco.linear_weight_grad, dy, (t(96, 4, dtype=I8), t(4, 2, dtype=U8)), out=w)
    wrong(loco.linear_weight_grad, dy, (t(4, 96, dtype=I8), t(2, 4, dtype=U8)), out=w)


def test_counts_are_still_refused():
    with pytest.raises(ValueError):
        loco.linear(t(4, 96), t(32, 96), out=t(4, 33))
    with pytest.raises(ValueError):
        loco.linear(t(4, 96), t(32, 96), out=t(127))
