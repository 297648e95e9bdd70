"""Refusals of the step operators' C calls and of their binding, without a GPU: every bad argument
gets its status before any HIP call.  The pointers are fake and never dereferenced."""
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
P = [0x100000000 * (i + 1) for i in range(16)]  # fake, aligned, 4 GiB apart


@pytest.fixture(scope="module")
def lib():
    return loco.load()


# -- AdamW ------------------------------------------------------------------------------------

def tensor(param=P[0], grad=P[1], m=P[2], v=P[3], me=P[4], ve=P[5], copy=P[6], n=1000, wd=0.1):
    return loco.AdamwTensor(param, grad, m, v, me, ve, copy, n, wd)


def plan_of(lib, ts=None, nt=None, pd=F32, gd=BF16, bits=8, block=256, table=P[15], nbytes=1 << 20, null=False):
    """(status, plan, the array that it refers to) of loco_adamw_plan."""
    ts = [tensor()] if ts is None else ts
    arr, plan = (loco.AdamwTensor * max(1, len(ts)))(*ts), loco.AdamwPlan()
    st = lib.loco_adamw_plan(arr if ts else None, len(ts) if nt is None else nt, pd, gd, bits, block, table, nbytes,
                             None if null else ctypes.byref(plan), None)
    return st, plan, arr


def adamw(lib, ts=None, **kw):
    return plan_of(lib, ts, **kw)[0]


@pytest.mark.parametrize("kw,want", [
    (dict(nt=-1), INV), (dict(ts=[], nt=1), INV), (dict(ts=[]), OK), (dict(null=True), INV),
    (dict(pd=I8), INV), (dict(gd=I8), INV), (dict(pd=5), INV), (dict(bits=4), INV), (dict(bits=16), INV),
    (dict(block=0), INV), (dict(block=-64), INV), (dict(block=100), UNSUP), (dict(block=1024), UNSUP),
    (dict(table=None), INV), (dict(nbytes=64), INV), (dict(nbytes=-1), INV), (dict(table=P[15] + 8), ALIGN),
    (dict(table=P[1] + 16), INV), (dict(table=P[5]), INV), (dict(ts=[tensor(n=0)], table=None), OK),
])
def test_adamw_plan(lib, kw, want):
    assert adamw(lib, **kw) == want


def test_adamw_table_bytes(lib):
    w = lib.loco_adamw_table_bytes
    assert w(0) == w(-5) == 0 and 0 < w(1) < w(2) < w(1000)
    assert adamw(lib, nbytes=w(1) - 1) == INV


def step(lib, plan, lr=1e-3, b1=0.9, b2=0.99, eps=1e-8, t=1, scale=None, null=False):
    opt = loco.AdamwOptions(lr, b1, b2, eps, t)
    return lib.loco_adamw(plan and ctypes.byref(plan), None if null else ctypes.byref(opt), scale, None)


@pytest.mark.parametrize("kw,want", [
    (dict(null=True), INV), (dict(lr=NAN), INV), (dict(lr=INF), INV), (dict(lr=1e300), INV), (dict(b1=1.0), INV),
    (dict(b1=-0.1), INV), (dict(b2=1.0), INV), (dict(b2=NAN), INV), (dict(eps=0.0), INV), (dict(eps=-1e-8), INV),
    (dict(eps=1e-60), INV), (dict(eps=1e39), INV), (dict(eps=NAN), INV), (dict(t=0), INV), (dict(t=-3), INV),
    (dict(scale=P[7] + 4), ALIGN), (dict(), OK), (dict(scale=P[7]), OK),
])
def test_adamw_options(lib, kw, want):
    """Of a plan without tensors, which launches nothing."""
    st, plan, _ = plan_of(lib, [])
    assert st == OK and step(lib, plan, **kw) == want


def test_adamw_of_a_plan_that_is_none(lib):
    assert step(lib, None) == INV
    assert step(lib, loco.AdamwPlan()) == INV  # never filled
    states = loco.AdamwPlan()
    assert lib.loco_adamw_state_plan(None, 0, 256, BF16, None, 0, ctypes.byref(states), None) == OK
    assert step(lib, states) == INV
    _, plan, _ = plan_of(lib, [])
    for fn in (lib.loco_adamw_state_read, lib.loco_adamw_state_write):
        assert fn(None, None) == INV and fn(ctypes.byref(plan), None) == INV and fn(ctypes.byref(states), None) == OK


@pytest.mark.parametrize("kw,want", [
    (dict(scale=P[0] + 16), INV), (dict(scale=P[2]), INV), (dict(scale=P[3] + 992), INV), (dict(scale=P[4]), INV),
    (dict(scale=P[5]), INV), (dict(scale=P[6] + 16), INV), (dict(scale=P[7] + 4), ALIGN),
])
def test_adamw_grad_scale_of_a_plan(lib, kw, want):
    """The plan's tensors are looked at before the launch (which no refused call reaches)."""
    arr = (loco.AdamwTensor * 1)(tensor())
    _, plan, _ = plan_of(lib, [])
    plan.ntensors, plan.tensors = 1, arr
    assert step(lib, plan, **kw) == want
    arr[0].weight_decay = 1e300
    assert step(lib, plan) == INV


@pytest.mark.parametrize("kw,want", [
    (dict(n=-1), INV), (dict(n=(1 << 52) + 1), INV), (dict(wd=NAN), INV), (dict(wd=INF), INV),
    (dict(param=None), INV), (dict(grad=None), INV), (dict(m=None), INV), (dict(v=None), INV), (dict(me=None), INV),
    (dict(ve=None), INV), (dict(param=P[0] + 4), ALIGN), (dict(grad=P[1] + 2), ALIGN), (dict(m=P[2] + 1), ALIGN),
    (dict(v=P[3] + 8), ALIGN), (dict(me=P[4] + 1), ALIGN), (dict(ve=P[5] + 2), ALIGN), (dict(copy=P[6] + 2), ALIGN),
    (dict(grad=P[0]), INV), (dict(m=P[0] + 3984), INV), (dict(v=P[2]), INV), (dict(me=P[4], ve=P[4]), INV),
    (dict(copy=P[0]), INV), (dict(copy=P[1]), INV), (dict(ve=P[6] + 1984), INV),
    (dict(n=0, param=None, grad=None, m=None, v=None, me=None, ve=None, copy=None), OK),
])
def test_adamw_tensor(lib, kw, want):
    assert adamw(lib, [tensor(**kw)]) == want
    # the same with a good tensor before it, elsewhere
    far = tensor(*(p + (1 << 30) for p in P[8:15]))
    if want != OK:  # a plan that passes fills its table
        assert adamw(lib, [far, tensor(**kw)]) == want


def test_adamw_across_tensors(lib):
    far = [p + (1 << 30) for p in P[8:15]]
    assert adamw(lib, [tensor(), tensor()]) == INV  # the same tensor twice
    for i in (0, 2, 3, 4, 5, 6):  # one buffer shared with another tensor's
        q = list(far)
        q[i] = P[i]
        assert adamw(lib, [tensor(), tensor(*q)]) == INV, i
    q = list(far)
    q[1] = P[2]  # a gradient over another tensor's state
    assert adamw(lib, [tensor(), tensor(*q)]) == INV


def test_adamw_copy_needs_fp32_params(lib):
    assert adamw(lib, pd=BF16) == INV


def state(codes=P[0], exps=P[1], values=P[2], n=1000, moment=1):
    return loco.AdamwState(codes, exps, values, n, moment)


@pytest.mark.parametrize("s,kw,want", [
    ([], dict(), OK), ([], dict(ns=1), INV), ([state()], dict(ns=-1), INV), ([state()], dict(block=96), UNSUP),
    ([state()], dict(block=0), INV), ([state()], dict(dtype=I8), INV), ([state(n=-1)], dict(), INV),
    ([state(moment=0)], dict(), INV), ([state(moment=3)], dict(), INV), ([state(codes=None)], dict(), INV),
    ([state(exps=None)], dict(), INV), ([state(values=None)], dict(), INV), ([state(codes=P[0] + 1)], dict(), ALIGN),
    ([state(exps=P[1] + 4)], dict(), ALIGN), ([state(values=P[2] + 2)], dict(), ALIGN),
    ([state(values=P[0] + 16)], dict(), INV), ([state(values=P[1])], dict(), INV), ([state(n=0)], dict(table=None), OK),
    ([state()], dict(table=None), INV), ([state()], dict(table=P[15] + 8), ALIGN), ([state()], dict(table=P[1]), INV),
    ([state()], dict(nbytes=16), INV), ([state()], dict(null=True), INV),
    ([state(), state(codes=P[3], exps=P[4])], dict(), INV), ([state(), state(exps=P[4], values=P[5])], dict(), INV),
    ([state(), state(codes=P[3], values=P[5])], dict(), INV),
])
def test_adamw_state_plan(lib, s, kw, want):
    a = dict(ns=len(s), block=256, dtype=BF16, table=P[15], nbytes=1 << 20, null=False)
    a.update(kw)
    arr, plan = (loco.AdamwState * max(1, len(s)))(*s), loco.AdamwPlan()
    assert lib.loco_adamw_state_plan(arr if s else None, a["ns"], a["block"], a["dtype"], a["table"], a["nbytes"],
                                     None if a["null"] else ctypes.byref(plan), None) == want


@pytest.fixture
def no_device(monkeypatch):
    """Host tensors: what passes the checks of sizes and types is refused for its memory, and says so."""
    monkeypatch.setattr(loco, "_device", lambda: 0)


def t(n, dtype=torch.float32):
    return torch.zeros(n, dtype=dtype)


F8, U8, BF = torch.float8_e4m3fn, torch.uint8, torch.bfloat16


def eight(n, block=256):
    return (t(n, F8), t(-(-n // block), U8)), (t(n, U8), t(-(-n // block), U8))


@pytest.mark.parametrize("make,err,match", [
    (lambda: (t(8), t(8), t(8), t(8)), ValueError, "device memory"),
    (lambda: (t(8), t(8), *eight(8), None, 0.1), ValueError, "device memory"),
    (lambda: (t(8), t(8), t(8)), ValueError, "expected"),
    (lambda: (t(8), t(8), t(8), t(8), None, 0.1, 3), ValueError, "expected"),
    (lambda: (t(8), t(9), t(8), t(8)), ValueError, "9 elements"),
    (lambda: (t(8), t(8), t(7), t(8)), ValueError, "7 elements"),
    (lambda: (t(8), t(8), t(8), t(8), t(9, BF)), ValueError, "9 elements"),
    (lambda: (t(8, torch.float16), t(8), t(8), t(8)), TypeError, "float32 or bfloat16"),
    (lambda: (t(8), t(8), t(8, BF), t(8)), TypeError, "m must be"),
    (lambda: (t(8), t(8), t(8), t(8), t(8)), TypeError, "param_bf16"),
    (lambda: (t(8, BF), t(8), t(8), t(8), t(8, BF)), TypeError, "param_bf16"),
    (lambda: (t(8), t(8), t(8), eight(8)[1]), TypeError, "one kind"),
    (lambda: (t(8), t(8), eight(8)[1], eight(8)[1]), TypeError, "m codes"),
    (lambda: (t(8), t(8), eight(8)[0], eight(8)[0]), TypeError, "v codes"),
    (lambda: (t(600), t(600), *eight(600, 128)), ValueError, "exps"),
])
def test_adamw_binding(no_device, make, err, match):
    with pytest.raises(err, match=match):
        loco.AdamwTensors([make()])


def test_adamw_binding_kinds_and_plans(no_device, monkeypatch):
    monkeypatch.setattr(loco, "_ptr", lambda t, dev: None if t is None else t.data_ptr())
    monkeypatch.setattr(loco, "_stream", lambda stream, dev: 0)
    with pytest.raises(TypeError, match="one kind"):
        loco.AdamwTensors([(t(8), t(8), t(8), t(8)), (t(8), t(8, BF), t(8), t(8))])
    plan = loco.AdamwTensors([])
    with pytest.raises(ValueError, match="its own"):
        loco.adamw(plan, step=1, lr=1e-3, weight_decay=0.1)
    with pytest.raises(ValueError, match="its own"):
        loco.adamw(plan, step=1, lr=1e-3, block=256)
    monkeypatch.setattr(loco, "_device", lambda: 1)
    with pytest.raises(ValueError, match="current device"):
        loco.adamw(plan, step=1, lr=1e-3)
    states = loco.AdamwStates([])
    monkeypatch.setattr(loco, "_device", lambda: 0)
    with pytest.raises(ValueError, match="current device"):
        loco.adamw_state_read(states)
    with pytest.raises(ValueError, match="its own"):
        loco.adamw_state_write(loco.AdamwStates([]), block=128)


@pytest.mark.parametrize("make,err,match", [
    (lambda: ((t(8, F8), t(1, U8)), t(8)), ValueError, "device memory"),
    (lambda: ((t(8, torch.int8), t(1, U8)), t(8)), TypeError, "codes"),
    (lambda: ((t(8, F8), t(2, U8)), t(8)), ValueError, "exps"),
    (lambda: ((t(8, F8), t(1, U8)), t(9)), ValueError, "9 elements"),
    (lambda: ((t(8, U8), t(1, U8)), t(8, torch.float16)), TypeError, "values"),
])
def test_adamw_states_binding(no_device, make, err, match):
    with pytest.raises(err, match=match):
        loco.AdamwStates([make()])


# -- the norms around a block --------------------------------------------------------------------

def ck(codes=P[12], exps=P[13], block=64):
    return ctypes.byref(loco.Checkpoint(codes, exps, block))


def rnorm(lib, **kw):
    a = dict(y=P[0], res=P[1], dtype=BF16, gate=P[2], kind=1, pw=P[3], w=P[4], param=BF16, rows=4, cols=64, scale=1.0,
             eps=1e-5, h=P[5], out=P[6], pr=P[7], r=P[8], ckpt=None)
    a.update(kw)
    return lib.loco_residual_norm(a["y"], a["res"], a["dtype"], a["gate"], a["kind"], a["pw"], a["w"], a["param"],
                                  a["rows"], a["cols"], a["scale"], a["eps"], a["h"], a["out"], a["pr"], a["r"], a["ckpt"],
                                  None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INV), (dict(cols=0), INV), (dict(cols=16385), UNSUP), (dict(rows=1 << 50), INV), (dict(dtype=I8), INV),
    (dict(param=I8), INV), (dict(eps=-1.0), INV), (dict(eps=NAN), INV), (dict(scale=INF), INV), (dict(kind=3), INV),
    (dict(kind=-1), INV), (dict(kind=0), INV), (dict(gate=None), INV), (dict(y=None, res=None), INV),
    (dict(y=None), INV), (dict(y=None, gate=None, kind=0, pw=None), INV), (dict(y=None, gate=None, kind=0, pr=None), INV),
    (dict(h=None, out=None), INV), (dict(r=None), INV), (dict(out=None), INV), (dict(out=None, w=None, r=None, ckpt=ck()), INV),
    (dict(out=None, r=None), INV), (dict(pr=None), INV), (dict(ckpt=ck(block=0)), INV), (dict(ckpt=ck(block=16)), UNSUP),
    (dict(ckpt=ck(codes=None)), INV), (dict(ckpt=ck(exps=P[13] + 1)), ALIGN),
    (dict(y=P[0] + 2), ALIGN), (dict(res=P[1] + 2), ALIGN), (dict(gate=P[2] + 2), ALIGN), (dict(pw=P[3] + 2), ALIGN),
    (dict(w=P[4] + 4), ALIGN), (dict(h=P[5] + 2), ALIGN), (dict(out=P[6] + 8), ALIGN), (dict(pr=P[7] + 4), ALIGN),
    (dict(r=P[8] + 4), ALIGN), (dict(h=P[0]), INV), (dict(out=P[1] + 496), INV), (dict(out=P[5]), INV), (dict(r=P[7]), INV),
    (dict(h=P[2]), INV), (dict(kind=2, h=P[2] + 496), INV), (dict(ckpt=ck(codes=P[6])), INV),
    (dict(rows=0), OK), (dict(rows=0, y=None, res=None, gate=None, h=None, out=None), OK),
])
def test_residual_norm(lib, kw, want):
    assert rnorm(lib, **kw) == want


def rback(lib, **kw):
    a = dict(dout=P[0], dh=P[1], h=P[2], y=P[3], dtype=BF16, gate=P[4], kind=1, pw=P[5], w=P[6], param=BF16, pr=P[7], r=P[8],
             rows=4, cols=64, scale=1.0, dres=P[9], dy=P[10], dg=P[11], dpw=P[12], dw=P[13], grad=F32, ws=P[14], nws=1 << 20)
    a.update(kw)
    return lib.loco_residual_norm_backward(a["dout"], a["dh"], a["h"], a["y"], a["dtype"], a["gate"], a["kind"], a["pw"],
                                           a["w"], a["param"], a["pr"], a["r"], a["rows"], a["cols"], a["scale"],
                                           a["dres"], a["dy"], a["dg"], a["dpw"], a["dw"], a["grad"], a["ws"], a["nws"], None)


NONE = dict(dres=None, dy=None, dg=None, dpw=None, dw=None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INV), (dict(cols=0), INV), (dict(cols=16385), UNSUP), (dict(dtype=I8), INV), (dict(param=7), INV),
    (dict(grad=I8), INV), (dict(scale=NAN), INV), (dict(kind=5), INV), (dict(kind=0), INV), (dict(gate=None), INV),
    (dict(dout=None, dh=None), INV), (dict(h=None), INV), (dict(r=None), INV), (dict(dout=None), INV),
    (dict(pr=None), INV), (dict(pr=None, pw=None), INV), (dict(y=None), INV),
    (dict(y=None, pr=None, pw=None, dpw=None), INV), (NONE, INV), (dict(gate=None, kind=0), INV),
    (dict(ws=None), INV), (dict(nws=0), INV), (dict(ws=P[14] + 4), ALIGN), (dict(dout=P[0] + 2), ALIGN),
    (dict(dh=P[1] + 2), ALIGN), (dict(h=P[2] + 2), ALIGN), (dict(y=P[3] + 2), ALIGN), (dict(gate=P[4] + 2), ALIGN),
    (dict(dres=P[9] + 2), ALIGN), (dict(dy=P[10] + 2), ALIGN), (dict(dg=P[11] + 4), ALIGN), (dict(dw=P[13] + 4), ALIGN),
    (dict(dres=P[0]), INV), (dict(dy=P[9]), INV), (dict(dg=P[4]), INV), (dict(dw=P[12]), INV), (dict(ws=P[1]), INV),
    (dict(dy=P[3] + 496), INV), (dict(kind=2, dg=P[10]), INV),
    (dict(rows=0, **NONE, ws=None, nws=0), OK), (dict(rows=0, ws=None), INV),
])
def test_residual_norm_backward(lib, kw, want):
    assert rback(lib, **kw) == want


def test_residual_norm_backward_workspace(lib):
    w = lib.loco_residual_norm_backward_workspace
    assert w(0, 64) >= 3 * 64 * 4 and w(1000, 4096) >= w(1, 4096) > 0
    assert w(-1, 64) == 0 and w(5, 0) == 0 and w(5, 16385) == 0 and w(1 << 50, 64) == 0
    assert rback(lib, rows=1000, cols=4096, nws=w(1000, 4096) - 1) == INV


def b(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


def rows32(*shape):
    return torch.zeros(*shape)


def refused(match, fn, *a, err=ValueError, **kw):
    with pytest.raises(err, match=match):
        fn(*a, **kw)


def test_residual_norm_binding(no_device):
    f, x = loco.residual_norm, b(4, 96)
    ok = dict(out=b(4, 96), rstd=rows32(4))
    refused("device memory", f, x, b(4, 96), **ok)
    refused("device memory", f, None, x, **ok)
    refused("needed", f, None, None, **ok)
    refused("shape", f, x, b(96, 4), **ok)
    refused("shape", f, x, None, h=b(96, 4))
    refused("elements", f, x, b(4, 95), **ok)
    refused("must be", f, x, x.float(), err=TypeError, **ok)
    refused("elements", f, x, None, weight=b(95), **ok)
    refused("must be", f, x, None, weight=b(96), gate=rows32(96), err=TypeError, **ok)
    refused("must be", f, x, None, gate=rows32(4, 96), err=TypeError, **ok)
    refused("device memory", f, x, None, gate=rows32(96), weight=rows32(96), **ok)
    refused("shape", f, x, None, gate=b(96, 4), **ok)
    refused("elements", f, x, None, gate=b(4), **ok)
    refused("elements", f, x, None, post_rstd=rows32(5), **ok)
    refused("must be", f, x, None, rstd=b(4), out=b(4, 96), err=TypeError)


def test_residual_norm_backward_binding(no_device):
    f, d, r = loco.residual_norm_backward, b(4, 96), rows32(4)
    refused("device memory", f, d, b(4, 96), rstd=r, dresidual=b(4, 96))
    refused("needed", f, None, d, rstd=r)
    refused("shape", f, d, b(96, 4), rstd=r)
    refused("must be", f, d, d.float(), rstd=r, err=TypeError)
    refused("shape", f, d, d, rstd=r, dy=b(96, 4))
    refused("elements", f, d, d, rstd=r, dweight=b(95))
    refused("must be", f, d, d, rstd=r, dweight=b(96), dpost_weight=rows32(96), err=TypeError)
    refused("elements", f, d, d, rstd=r, gate=b(4, 96), y=d, dgate=b(96))
    refused("must be", f, d, d, rstd=r, gate=b(4, 96), y=d, dgate=rows32(4, 96), err=TypeError)
    refused("elements", f, d, d, rstd=r, gate=b(96), y=d, dgate=b(4, 96))


# -- log probabilities of tokens ---------------------------------------------------------------------

def logp(lib, **kw):
    a = dict(x=P[0], dtype=BF16, rows=4, vocab=100, ld=100, t=P[1], scale=1.0, lp=P[2], h=P[3], st=P[4], top=3, ids=P[5],
             tl=P[6], ws=P[7], nws=1 << 30)
    a.update(kw)
    return lib.loco_token_logprobs(a["x"], a["dtype"], a["rows"], a["vocab"], a["ld"], a["t"], a["scale"], a["lp"], a["h"],
                                   a["st"], a["top"], a["ids"], a["tl"], a["ws"], a["nws"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INV), (dict(vocab=0), INV), (dict(vocab=-1), INV), (dict(ld=99), INV), (dict(ld=-100), INV),
    (dict(rows=1 << 45), INV), (dict(vocab=(1 << 24) + 1, ld=1 << 25), UNSUP), (dict(dtype=I8), INV),
    (dict(scale=0.0), INV), (dict(scale=-1.0), INV), (dict(scale=NAN), INV), (dict(scale=INF), INV), (dict(scale=1e-7), INV),
    (dict(scale=1e7), INV), (dict(top=-1), INV), (dict(top=33), UNSUP), (dict(x=None), INV), (dict(t=None), INV),
    (dict(ids=None), INV), (dict(tl=None), INV), (dict(lp=None, h=None, st=None, top=0), INV),
    (dict(x=P[0] + 2), ALIGN), (dict(t=P[1] + 8), ALIGN), (dict(lp=P[2] + 4), ALIGN), (dict(h=P[3] + 4), ALIGN),
    (dict(st=P[4] + 8), ALIGN), (dict(ids=P[5] + 4), ALIGN), (dict(tl=P[6] + 4), ALIGN),
    (dict(lp=P[0] + 16), INV), (dict(lp=P[0] + 784), INV), (dict(h=P[2]), INV), (dict(st=P[3]), INV), (dict(ids=P[6]), INV),
    (dict(lp=P[1]), INV), (dict(ld=200, lp=P[0] + 1200), INV), (dict(rows=0), OK), (dict(rows=0, x=None, t=None), OK),
])
def test_token_logprobs(lib, kw, want):
    assert logp(lib, **kw) == want


def lback(lib, **kw):
    a = dict(x=P[0], dtype=F32, rows=4, vocab=100, ld=100, t=P[1], scale=1.0, st=P[2], h=P[3], dl=P[4], dh=P[5], dx=P[6],
             dld=100)
    a.update(kw)
    return lib.loco_token_logprobs_backward(a["x"], a["dtype"], a["rows"], a["vocab"], a["ld"], a["t"], a["scale"], a["st"],
                                            a["h"], a["dl"], a["dh"], a["dx"], a["dld"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(rows=-1), INV), (dict(vocab=0), INV), (dict(ld=99), INV), (dict(dld=99), INV), (dict(rows=1 << 45), INV),
    (dict(vocab=(1 << 24) + 1, ld=1 << 25, dld=1 << 25), UNSUP), (dict(dtype=I8), INV), (dict(scale=0.0), INV),
    (dict(x=None), INV), (dict(st=None), INV), (dict(dx=None), INV), (dict(dl=None, dh=None), INV), (dict(t=None), INV),
    (dict(h=None), INV), (dict(x=P[0] + 4), ALIGN), (dict(st=P[2] + 8), ALIGN), (dict(dl=P[4] + 4), ALIGN),
    (dict(dx=P[6] + 4), ALIGN), (dict(dx=P[0] + 16), INV), (dict(dx=P[0], dld=104), INV), (dict(dx=P[2]), INV),
    (dict(dx=P[4]), INV), (dict(dx=P[1]), INV), (dict(dx=P[0] + 1584), INV), (dict(rows=0), OK),
    (dict(rows=0, x=None, dx=None), OK),
])
def test_token_logprobs_backward(lib, kw, want):
    assert lback(lib, **kw) == want


def test_token_logprobs_workspace(lib):
    assert lib.loco_token_logprobs_workspace(0, 100, 0) == 0
    assert lib.loco_token_logprobs_workspace(-1, 100, 0) == 0


def test_token_logprobs_binding(no_device):
    f, x, t = loco.token_logprobs, b(4, 96), torch.zeros(4, dtype=torch.int64)
    r = rows32(4)
    refused("device memory", f, x, t, logprob=r)
    refused("elements", f, x, t[:3], logprob=r)
    refused("must be", f, x, t.int(), logprob=r, err=TypeError)
    refused("elements", f, x, t, logprob=rows32(5))
    refused("must be", f, x, t, logprob=b(4), err=TypeError)
    refused("shape", f, x, t, stats=rows32(2, 4))
    refused("go together", f, x, top_ids=torch.zeros(4, 2, dtype=torch.int32))
    refused("elements", f, x, top_ids=torch.zeros(4, 2, dtype=torch.int32), top_logprobs=rows32(4, 3))
    refused("must be", f, x, top_ids=torch.zeros(4, 2, dtype=torch.int64), top_logprobs=rows32(4, 2), err=TypeError)
    refused("must be", f, x.half(), t, logprob=r, err=TypeError)
    refused("apart", f, b(96, 4).t(), t, logprob=r)
    refused("apart", f, b(1, 96).expand(4, 96), t, logprob=r)
    refused("apart", f, b(4, 2, 96)[:, 0].unsqueeze(1).expand(4, 2, 96), torch.zeros(8, dtype=torch.int64), logprob=rows32(8))
    refused("row must be contiguous", f, b(192)[::2], t[:1], logprob=rows32(1))
    refused("device memory", f, b(4, 100)[:, :96], t, logprob=r)
    refused("device memory", f, b(2, 2, 100)[..., :96], t, logprob=r)
    refused("shape", f, b(2, 3, 96), torch.zeros(3, 2, dtype=torch.int64), logprob=rows32(6))
    g, s = loco.token_logprobs_backward, rows32(4, 2)
    refused("device memory", g, x, t, s, dlogprob=r, dlogits=b(4, 96))
    refused("shape", g, x, t, s, dlogprob=r, dlogits=b(96, 4))
    refused("must be", g, x, t, s, dlogprob=r, dlogits=rows32(4, 96), err=TypeError)
    refused("apart", g, x, t, s, dlogprob=r, dlogits=b(1, 96).expand(4, 96))
    refused("elements", g, x, t, rows32(4, 1), dlogprob=r, dlogits=b(4, 96))
    refused("elements", g, x, t, s, dlogprob=rows32(3), dlogits=b(4, 96))
