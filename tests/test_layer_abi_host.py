"""Refusals of the layer operators' C calls, without a GPU: every bad argument gets its status
before any HIP call, and the workspace sizes are what the calls then ask for.  The pointers
are fake and never dereferenced."""
import ctypes

import pytest
import torch

if torch.cuda.is_available():
    # Fake pointers must never reach a real device: these checks run only where no GPU is.
    pytest.skip("host-only validation tests (fake device pointers)", allow_module_level=True)

from bit_gradient_compression_amd import loco  # noqa: E402

OK, INV, ALIGN, UNSUP = loco.LOCO_OK, loco.LOCO_ERR_INVALID, loco.LOCO_ERR_ALIGN, loco.LOCO_ERR_UNSUPPORTED
F32, BF16, I8 = loco.LOCO_F32, loco.LOCO_BF16, loco.LOCO_I8
NAN, INF = float("nan"), float("inf")
P = [0x100000000 * (i + 1) for i in range(12)]  # fake, aligned, 4 GiB apart


@pytest.fixture(scope="module")
def lib():
    return loco.load()


def ck(codes=P[8], exps=P[9], block=64):
    return ctypes.byref(loco.Checkpoint(codes, exps, block))


def norm(lib, **kw):
    a = dict(x=P[0], dtype=BF16, w=P[1], b=P[2], param=BF16, rows=4, cols=64, eps=1e-5, y=P[3], mean=P[4], rstd=P[5],
             ckpt=None)
    a.update(kw)
    return lib.loco_layer_norm(a["x"], a["dtype"], a["w"], a["b"], a["param"], a["rows"], a["cols"], a["eps"], a["y"],
                               a["mean"], a["rstd"], a["ckpt"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INV), (dict(cols=0), INV), (dict(cols=-5), INV), (dict(cols=16385), UNSUP),
    (dict(rows=1 << 50, cols=64), INV), (dict(dtype=I8), INV), (dict(dtype=7), INV), (dict(param=I8), INV),
    (dict(eps=-1e-5), INV), (dict(eps=NAN), INV), (dict(eps=INF), INV),
    (dict(x=None), INV), (dict(y=None), INV), (dict(mean=None), INV), (dict(rstd=None), INV),
    (dict(x=P[0] + 2), ALIGN), (dict(w=P[1] + 8), ALIGN), (dict(b=P[2] + 4), ALIGN), (dict(mean=P[4] + 4), ALIGN),
    (dict(y=P[0]), INV), (dict(y=P[0] + 496), INV), (dict(rstd=P[4]), INV), (dict(y=P[1]), INV),
    (dict(ckpt=ck(block=0)), INV), (dict(ckpt=ck(block=-64)), INV), (dict(ckpt=ck(block=128)), UNSUP),
    (dict(ckpt=ck(codes=None)), INV), (dict(ckpt=ck(exps=None)), INV), (dict(ckpt=ck(codes=P[3])), INV),
    (dict(ckpt=ck(exps=P[8] + 16)), INV), (dict(ckpt=ck(codes=P[8] + 1)), ALIGN),
    (dict(rows=0), OK), (dict(rows=0, x=None, y=None, mean=None, rstd=None), OK),
])
def test_layer_norm(lib, kw, want):
    assert norm(lib, **kw) == want


def norm_bwd(lib, **kw):
    a = dict(dy=P[0], x=P[1], dtype=BF16, w=P[2], param=F32, mean=P[3], rstd=P[4], res=None, rows=4, cols=64, dx=P[5],
             dw=P[6], db=P[7], grad=F32, ws=P[8], nws=1 << 20)
    a.update(kw)
    return lib.loco_layer_norm_backward(a["dy"], a["x"], a["dtype"], a["w"], a["param"], a["mean"], a["rstd"], a["res"],
                                        a["rows"], a["cols"], a["dx"], a["dw"], a["db"], a["grad"], a["ws"], a["nws"],
                                        None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INV), (dict(cols=0), INV), (dict(cols=16385), UNSUP), (dict(dtype=I8), INV), (dict(param=3), INV),
    (dict(grad=I8), INV), (dict(dy=None), INV), (dict(x=None), INV), (dict(mean=None), INV), (dict(rstd=None), INV),
    (dict(dx=None), INV), (dict(ws=None), INV), (dict(nws=0), INV), (dict(nws=-1), INV),
    (dict(dy=P[0] + 2), ALIGN), (dict(res=P[9] + 2), ALIGN), (dict(dw=P[6] + 4), ALIGN), (dict(ws=P[8] + 4), ALIGN),
    (dict(dx=P[0]), INV), (dict(dx=P[1]), INV), (dict(res=P[5]), INV), (dict(db=P[6]), INV), (dict(ws=P[0]), INV),
    (dict(ws=P[6]), INV), (dict(rows=0, dw=None, db=None, ws=None, nws=0), OK),
    (dict(rows=0, ws=None), INV),  # the zeros of dw and db go through the workspace
])
def test_layer_norm_backward(lib, kw, want):
    assert norm_bwd(lib, **kw) == want


def test_layer_norm_backward_workspace(lib):
    w = lib.loco_layer_norm_backward_workspace
    assert w(0, 64) >= 2 * 64 * 4 and w(1000, 4096) >= w(1, 4096) > 0
    assert w(-1, 64) == 0 and w(5, 0) == 0 and w(5, 16385) == 0
    assert norm_bwd(lib, rows=1000, cols=4096, dx=P[10], nws=w(1000, 4096) - 1) == INV


@pytest.mark.parametrize("kw,want", [
    (dict(ckpt=None), INV), (dict(rows=-1), INV), (dict(cols=-1), INV), (dict(rows=1 << 39, cols=1 << 39), INV),
    (dict(dtype=I8), INV), (dict(ckpt=ck(block=96)), UNSUP), (dict(ckpt=ck(block=0)), INV), (dict(x=None), INV),
    (dict(x=P[0] + 4), ALIGN), (dict(ckpt=ck(exps=P[9] + 1)), ALIGN), (dict(x=P[8]), INV), (dict(x=P[9]), INV),
    (dict(ckpt=ck(codes=None)), INV), (dict(rows=0), OK), (dict(cols=0), OK),
])
def test_checkpoint_write_and_read(lib, kw, want):
    a = dict(x=P[0], dtype=BF16, rows=4, cols=100, ckpt=ck())
    a.update(kw)
    assert lib.loco_checkpoint_write(a["x"], a["dtype"], a["rows"], a["cols"], a["ckpt"], None) == want
    assert lib.loco_checkpoint_read(a["ckpt"], a["rows"], a["cols"], 0, a["x"], a["dtype"], None) == want


def test_checkpoint_read_activation(lib):
    for act in (-1, 4, 100):
        assert lib.loco_checkpoint_read(ck(), 4, 64, act, P[0], BF16, None) == INV


PRODUCT_SIZES = [
    (dict(rows=-1), INV), (dict(n=-1), INV), (dict(k=-1), INV), (dict(n=(1 << 20) + 1), UNSUP),
    (dict(k=(1 << 20) + 1), UNSUP), (dict(rows=(1 << 28) + 1), UNSUP), (dict(rows=1 << 28, n=1 << 10), UNSUP),
    (dict(n=1 << 19, k=1 << 18), UNSUP), (dict(rows=1 << 40, n=1 << 20), INV), (dict(act=-1), INV), (dict(act=4), INV),
    (dict(dtype=I8), INV), (dict(ckpt=ck(block=16)), UNSUP), (dict(ckpt=ck(block=-1)), INV),
]


def linear(lib, **kw):
    a = dict(x=P[0], w=P[1], b=P[2], res=P[3], rows=4, n=64, k=96, act=2, out=P[4], dtype=BF16, ckpt=ck(), ws=P[5],
             nws=1 << 30)
    a.update(kw)
    return lib.loco_linear(a["x"], a["w"], a["b"], a["res"], a["rows"], a["n"], a["k"], a["act"], a["out"], a["dtype"],
                           a["ckpt"], a["ws"], a["nws"], None)


@pytest.mark.parametrize("kw,want", PRODUCT_SIZES + [
    (dict(x=None), INV), (dict(w=None), INV), (dict(out=None), INV), (dict(ckpt=ck(codes=None)), INV),
    (dict(x=P[0] + 2), ALIGN), (dict(w=P[1] + 2), ALIGN), (dict(b=P[2] + 2), ALIGN), (dict(res=P[3] + 2), ALIGN),
    (dict(out=P[0]), INV), (dict(out=P[3]), INV), (dict(out=P[1]), INV), (dict(ckpt=ck(codes=P[4])), INV),
    (dict(rows=0), OK), (dict(n=0), OK), (dict(rows=0, x=None, out=None), OK),
])
def test_linear(lib, kw, want):
    assert linear(lib, **kw) == want


def input_grad(lib, **kw):
    a = dict(dy=P[0], w=P[1], res=P[3], rows=4, n=64, k=96, act=2, out=P[4], dtype=BF16, ckpt=ck(), ws=P[5], nws=1 << 30)
    a.update(kw)
    return lib.loco_linear_input_grad(a["dy"], a["w"], a["res"], a["rows"], a["n"], a["k"], a["act"], a["ckpt"], a["out"],
                                      a["dtype"], a["ws"], a["nws"], None)


@pytest.mark.parametrize("kw,want", PRODUCT_SIZES + [
    (dict(dy=None), INV), (dict(w=None), INV), (dict(out=None), INV), (dict(ckpt=None), INV),
    (dict(ckpt=ck(exps=None)), INV), (dict(dy=P[0] + 2), ALIGN), (dict(out=P[0]), INV), (dict(out=P[8]), INV),
    (dict(out=P[3]), INV), (dict(rows=0), OK), (dict(k=0), OK),
])
def test_linear_input_grad(lib, kw, want):
    assert input_grad(lib, **kw) == want


def weight_grad(lib, **kw):
    a = dict(dy=P[0], ckpt=ck(), rows=4, n=64, k=96, act=2, acc=0, out=P[4], db=P[6], dtype=BF16, ws=P[5], nws=1 << 30)
    a.update(kw)
    return lib.loco_linear_weight_grad(a["dy"], a["ckpt"], a["rows"], a["n"], a["k"], a["act"], a["acc"], a["out"],
                                       a["db"], a["dtype"], a["ws"], a["nws"], None)


@pytest.mark.parametrize("kw,want", PRODUCT_SIZES + [
    (dict(ckpt=None), INV), (dict(dy=None), INV), (dict(out=None), INV), (dict(ckpt=ck(codes=None)), INV),
    (dict(dy=P[0] + 2), ALIGN), (dict(db=P[6] + 2), ALIGN), (dict(out=P[0]), INV), (dict(out=P[8]), INV),
    (dict(db=P[4]), INV), (dict(ws=P[4]), INV), (dict(nws=0), INV), (dict(n=0), OK),
])
def test_linear_weight_grad(lib, kw, want):
    assert weight_grad(lib, **kw) == want


def test_workspaces_of_refused_sizes(lib):
    for rows, n, k in ((-1, 64, 64), (4, -1, 64), (4, 64, -1), (4, (1 << 20) + 1, 64), (1 << 40, 64, 64)):
        assert lib.loco_linear_workspace(rows, n, k) == 0
        assert lib.loco_linear_input_grad_workspace(rows, n, k) == 0
        assert lib.loco_linear_weight_grad_workspace(rows, n, k, 0) == 0


def test_split_products_ask_for_their_workspace(lib):
    """Few rows and a long contraction: the call refuses less than the function returned."""
    need = lib.loco_linear_workspace(128, 64, 16384)
    assert need > 0
    assert linear(lib, rows=128, n=64, k=16384, nws=need - 1) == INV
    assert linear(lib, rows=128, n=64, k=16384, ws=None, nws=need) == INV
    need = lib.loco_linear_input_grad_workspace(128, 16384, 64)
    assert need > 0 and input_grad(lib, rows=128, n=16384, k=64, nws=need - 1) == INV
    need = lib.loco_linear_weight_grad_workspace(16384, 64, 64, 0)
    assert need > 0 and weight_grad(lib, rows=16384, n=64, k=64, nws=need - 1) == INV


# -- the binding's own checks (host tensors, refused before any pointer is taken) --------

@pytest.fixture
def no_device(monkeypatch):
    monkeypatch.setattr(loco, "_device", lambda: 0)


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def refuses(error, fn, *a, **kw):
    with pytest.raises(error):
        fn(*a, **kw)


def test_binding_shapes_and_types(no_device):
    f = torch.float32
    x, w = t(4, 64), t(64)
    s = t(4, dtype=f)
    refuses(ValueError, loco.layer_norm, x, t(63), None, out=x, mean=s, rstd=s)
    refuses(ValueError, loco.layer_norm, x, w, None, out=t(4, 63), mean=s, rstd=s)
    refuses(ValueError, loco.layer_norm, x, w, None, out=x, mean=t(3, dtype=f), rstd=s)
    refuses(TypeError, loco.layer_norm, x, w, None, out=t(4, 64, dtype=f), mean=s, rstd=s)
    refuses(TypeError, loco.layer_norm, x, w, t(64, dtype=f), out=x, mean=s, rstd=s)
    refuses(TypeError, loco.layer_norm, x.half(), w, None, out=x.half(), mean=s, rstd=s)
    refuses(TypeError, loco.layer_norm_backward, x, x, w, s, s, dx=x, dweight=w, dbias=t(64, dtype=f))
    refuses(ValueError, loco.layer_norm_backward, t(5, 64), x, w, s, s, dx=x)
    c, e = t(4, 64, dtype=torch.int8), t(4, 1, dtype=torch.uint8)
    refuses(ValueError, loco.checkpoint_write, x, codes=t(4, 63, dtype=torch.int8), exps=e)
    refuses(ValueError, loco.checkpoint_write, x, codes=c, exps=t(4, 2, dtype=torch.uint8))
    refuses(TypeError, loco.checkpoint_write, x, codes=c.to(torch.uint8), exps=e)
    refuses(ValueError, loco.checkpoint_read, c, e, out=t(4, 32))
    refuses(TypeError, loco.checkpoint_read, c, e, out=t(4, 64, dtype=torch.float16))
    wt = t(32, 64)
    refuses(ValueError, loco.linear, x, t(32, 63), out=t(4, 32))
    refuses(ValueError, loco.linear, x, wt, out=t(4, 33))
    refuses(ValueError, loco.linear, x, wt, out=t(4, 32), bias=t(64))
    refuses(TypeError, loco.linear, x.float(), wt, out=t(4, 32))
    refuses(ValueError, loco.linear_input_grad, t(4, 31), wt, out=x)
    refuses(ValueError, loco.linear_input_grad, t(4, 32), wt, out=x, residual=t(4, 63))
    refuses(ValueError, loco.linear_weight_grad, t(4, 31), (c, e), out=wt)
    refuses(TypeError, loco.linear_weight_grad, t(4, 32), (c, e), out=wt, dbias=t(32, dtype=f))
    refuses(ValueError, loco.linear_weight_grad, t(5, 32), (c, e), out=wt)


def test_binding_refuses_host_and_strided_tensors(no_device):
    x, s = t(4, 64), t(4, dtype=torch.float32)
    refuses(ValueError, loco.layer_norm, x, None, None, out=x.clone(), mean=s, rstd=s.clone())  # host memory
    refuses(ValueError, loco.linear, x, t(32, 64), out=t(4, 32))
