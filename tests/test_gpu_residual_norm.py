"""The norms around a block with gate and residual, forward and backward, against the 64-bit
oracle."""
import itertools

import numpy as np
import pytest
import torch

from layer_util import U, Guarded, assert_near, check_checkpoint, f64, guarded, new_checkpoint, randn, round_bound
from oracle import step_oracle as O

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32

SHAPES = [(1, 1), (3, 7), (5, 8), (5, 64), (6, 511), (4, 512), (7, 513), (9, 1000), (3, 1024), (5, 1025), (5, 2047),
          (2, 2048), (5, 4096), (2, 4097), (3, 8191), (2, 8192), (3, 9001), (3, 14336), (2, 16383), (2, 16384)]
GATES = [None, "column", "element"]


def seq(cols):
    """Additions a term of a row's sum passes through: a lane's own columns, then lanes and waves."""
    return cols / 256 + 24


class Case:
    def __init__(self, rows, cols, dtype=BF, param=BF, post=True, gate="column", scale=0.7, alone=False, residual=True,
                 affine=True, seed=0):
        s = rows * 131 + cols + 1000 * seed
        self.rows, self.cols, self.dtype, self.param, self.scale, self.eps = rows, cols, dtype, param, scale, 1e-5
        self.post, self.kind = post and not alone, None if alone else gate
        self.y = None if alone else randn(s, rows, cols, dtype=dtype, scale=2.0, shift=0.3)
        self.residual = randn(s + 1, rows, cols, dtype=dtype, scale=1.5) if residual or alone else None
        self.weight = randn(s + 2, cols, dtype=param, shift=1.0) if affine else None
        self.post_weight = randn(s + 3, cols, dtype=param, shift=1.0) if self.post and affine else None
        self.gate = None
        if self.kind == "column":
            self.gate = randn(s + 4, cols, dtype=param)
        elif self.kind == "element":
            self.gate = randn(s + 4, rows, cols, dtype=dtype)

    def f(self, name):
        t = getattr(self, name)
        return None if t is None else f64(t)

    def oracle(self):
        return O.residual_norm(self.f("y"), self.f("residual"), self.f("weight"), self.f("post_weight"), self.f("gate"),
                               self.scale, self.eps, self.post)

    def bounds(self, out, h, r, rp):
        """Errors of out, h, rstd and post_rstd.  A sum of squares has positive terms: its relative
        error, and so the factor's, is that of its additions and a few roundings.  h's error reaches
        rstd through the mean square."""
        k = 2 * (seq(self.cols) + 6) * U
        dh = np.zeros_like(h)
        if self.y is not None:
            u = np.abs(self.f("y") * self.scale * (1 if self.gate is None else self.f("gate")))
            if self.post:
                u = u * rp[:, None] * (1 if self.post_weight is None else np.abs(self.f("post_weight")))
            dh = u * (k + 6 * U) + 2 * U * (np.abs(h) + u)
        ms = np.maximum((h * h).mean(1) + self.eps, 1e-300)
        dr = k + (np.abs(h) * dh).mean(1) / ms
        w = 1 if self.weight is None else np.abs(self.f("weight"))
        dout = w * r[:, None] * (dh + np.abs(h) * (dr[:, None] + 4 * U))
        return dout, dh, r * dr, None if rp is None else rp * k

    def run(self, lib, block=0, h=True, out=True):
        shape = (self.rows, self.cols)
        g = {"h": guarded(shape, self.dtype) if h else None, "out": guarded(shape, self.dtype) if out else None,
             "rstd": guarded((self.rows,), F32) if out else None,
             "post_rstd": guarded((self.rows,), F32) if self.post else None}
        ck = new_checkpoint(*shape, block) if block else None
        t = {k: None if v is None else v.t for k, v in g.items()}
        lib.residual_norm(self.y, self.residual, weight=self.weight if out else None, post_weight=self.post_weight,
                          gate=self.gate, scale=self.scale, eps=self.eps, checkpoint=(ck[0].t, ck[1].t) if ck else None,
                          block=block or 64, **t)
        torch.cuda.synchronize()
        for x in [*g.values(), *(ck or ())]:
            if x is not None:
                x.check()
        return t, ck

    def check(self, lib, block=0, h=True, out=True):
        t, ck = self.run(lib, block, h, out)
        want = dict(zip(("out", "h", "rstd", "post_rstd"), self.oracle()))
        bound = dict(zip(("out", "h", "rstd", "post_rstd"), self.bounds(*want.values())))
        for k, v in t.items():
            if v is not None:
                assert_near(v, want[k], bound[k] + round_bound(want[k], v.dtype), k)
        if ck:
            check_checkpoint(ck[0].t, ck[1].t, block, want["out"], bound["out"] + U * np.abs(want["out"]))


@pytest.mark.parametrize("dtype,param", [(BF, BF), (F32, F32), (BF, F32), (F32, BF)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_forward(gpu_lib, rows, cols, dtype, param):
    for i, (post, gate) in enumerate(itertools.product((True, False), GATES)):
        Case(rows, cols, dtype, param, post, gate).check(gpu_lib, block=[0, 32, 64][(rows + cols + i) % 3])


@pytest.mark.parametrize("rows,cols", [(1, 5), (6, 511), (5, 1024), (3, 4096), (2, 9001)])
def test_forward_parts(gpu_lib, rows, cols):
    """The norm alone; no residual; no stored stream; no norm before the next block; no weights."""
    for dtype in (BF, F32):
        Case(rows, cols, dtype, alone=True).check(gpu_lib, block=64, h=False)
        Case(rows, cols, dtype, alone=True).check(gpu_lib, h=True)
        Case(rows, cols, dtype, residual=False).check(gpu_lib)
        Case(rows, cols, dtype, residual=False, gate=None, post=False).check(gpu_lib, h=False)
        Case(rows, cols, dtype).check(gpu_lib, h=False, block=32)
        Case(rows, cols, dtype).check(gpu_lib, out=False)
        Case(rows, cols, dtype, affine=False, gate=None).check(gpu_lib)
        Case(rows, cols, dtype, scale=0.0).check(gpu_lib)


def test_forward_hard_rows(gpu_lib):
    """Rows of zeros (with eps, and without: then NaN in that row only), tiny and huge values."""
    c = Case(6, 1003, F32, F32, gate=None)
    for t in (c.y, c.residual):
        t[0] = 0.0
        t[1] *= 1e-18
        t[2] *= 1e15
    c.y[3] = 0.0
    c.check(gpu_lib)
    z = Case(4, 515, F32, F32, alone=True)
    z.residual[1] = 0.0
    z.eps = 0.0
    t, _ = z.run(gpu_lib, h=False)
    good = torch.tensor([0, 2, 3], device="cuda")
    assert bool(torch.isnan(t["out"][1]).all()) and bool(torch.isfinite(t["out"][good]).all())
    assert bool(torch.isinf(t["rstd"][1]))


@pytest.mark.parametrize("cols", [300, 2000, 9000])
def test_non_finite_rows_stay_alone(gpu_lib, cols):
    c = Case(9, cols)
    clean, ck0 = c.run(gpu_lib, block=64)
    c.y[2, cols // 2] = float("nan")
    c.residual[5, 0] = float("inf")
    t, ck = c.run(gpu_lib, block=64)
    ok = torch.tensor([0, 1, 3, 4, 6, 7, 8], device="cuda")
    assert bool(torch.isnan(t["out"][2]).all()) and bool(torch.isnan(t["out"][5, 0]))
    assert float(t["rstd"][5]) == 0.0
    for k in t:
        assert torch.equal(t[k][ok], clean[k][ok]), k
    assert bool((ck[1].t[2] == 255).all()) and bool((ck[1].t[5, 0] == 255))
    assert torch.equal(ck[0].t[ok], ck0[0].t[ok]) and torch.equal(ck[1].t[ok], ck0[1].t[ok])


# -- backward ---------------------------------------------------------------------------

class Back(Case):
    """The backward pass of a case whose forward factors are the oracle's."""

    def __init__(self, *a, grad=F32, dout=True, dh=True, **kw):
        super().__init__(*a, **kw)
        s = self.rows * 17 + self.cols
        _, h, r, rp = self.oracle()
        self.h = torch.from_numpy(h).to(self.dtype).cuda()
        self.rstd = torch.from_numpy(r).float().cuda()
        self.post_rstd = None if rp is None else torch.from_numpy(rp).float().cuda()
        self.dout = randn(s, self.rows, self.cols, dtype=self.dtype, scale=1e-3) if dout else None
        self.dh = randn(s + 1, self.rows, self.cols, dtype=self.dtype, scale=1e-3) if dh else None
        self.grad = grad

    NAMES = ("dresidual", "dy", "dgate", "dweight", "dpost_weight")

    def outputs(self, names):
        shape, made = (self.rows, self.cols), {}
        for n in names:
            if n == "dgate" and self.gate is None or n == "dpost_weight" and not self.post or \
                    n == "dweight" and self.dout is None:
                continue
            matrix = n in ("dresidual", "dy") or (n == "dgate" and self.kind == "element")
            made[n] = guarded(shape, self.dtype) if matrix else guarded((self.cols,), self.grad)
        return made

    def run(self, lib, names=NAMES):
        g = self.outputs(names)
        ws = Guarded((lib.residual_norm_backward_workspace(self.rows, self.cols),), torch.uint8, 0xCC)
        lib.residual_norm_backward(self.dout, self.h if self.dout is not None else None, rstd=self.rstd, weight=self.weight,
                                   dh=self.dh, y=self.y, post_rstd=self.post_rstd, post_weight=self.post_weight,
                                   gate=self.gate, scale=self.scale, workspace=ws.t, **{k: v.t for k, v in g.items()})
        torch.cuda.synchronize()
        for x in [ws, *g.values()]:
            x.check()
        return {k: v.t for k, v in g.items()}

    def check(self, lib):
        got = self.run(lib)
        want = O.residual_norm_backward(self.f("dout"), self.f("dh"), self.f("h"), self.f("rstd"), self.f("weight"),
                                        self.f("y"), self.f("post_rstd"), self.f("post_weight"), self.f("gate"), self.scale)
        if self.kind == "column":
            want["dgate"] = want["dgate"].sum(0)
        bound = self.bounds()
        for k, v in got.items():
            assert_near(v, want[k], bound[k] + round_bound(want[k], v.dtype), k)

    def bounds(self):
        """Roundings of each product and the rows' sums (K), carried from the gradient of the stream
        to what follows from it; a sum over the rows passes each term through at most rows / 256
        (a group's own) + 64 (teams and the join) additions."""
        a = lambda n: None if getattr(self, n) is None else np.abs(self.f(n))
        one = lambda n: 1.0 if a(n) is None else a(n)
        K, per = 2 * (seq(self.cols) + 12) * U, self.rows / 256 + 64
        gh = db = np.zeros((self.rows, self.cols))
        out = {}
        if self.dout is not None:
            r = a("rstd")[:, None]
            xh, g = a("h") * r, a("dout") * one("weight")
            gh = r * (g + xh * (g * xh).mean(1, keepdims=True))
            db = K * gh
            out["dweight"] = 2 * (per + 4) * U * (a("dout") * xh).sum(0)
        if self.dh is not None:
            gh = gh + a("dh")
        db = db + 4 * U * gh
        out["dresidual"] = db
        s, gate = abs(self.scale), one("gate")
        yh = 0.0 if self.y is None else a("y") * (a("post_rstd")[:, None] if self.post else 1.0)
        e = lambda x: s * x * (db + 8 * U * gh)
        summed = lambda x: e(x).sum(0) + 2 * per * U * (s * x * gh).sum(0)
        if self.gate is not None:
            out["dgate"] = (summed if self.kind == "column" else e)(yh * one("post_weight"))
        t, dt = s * gate * one("post_weight") * gh, e(gate * one("post_weight"))
        out["dy"] = dt
        if self.post:
            out["dpost_weight"] = summed(gate * yh)
            rp = a("post_rstd")[:, None]
            out["dy"] = rp * (dt + yh * (dt * yh).mean(1, keepdims=True) + K * (t + yh * (t * yh).mean(1, keepdims=True)))
        return out


@pytest.mark.parametrize("dtype,param,grad", [(BF, BF, BF), (F32, F32, F32), (BF, F32, F32), (F32, BF, BF)])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_backward(gpu_lib, rows, cols, dtype, param, grad):
    for post, gate in itertools.product((True, False), GATES):
        Back(rows, cols, dtype, param, post, gate, grad=grad).check(gpu_lib)


@pytest.mark.parametrize("rows,cols", [(1, 4096), (4097, 64), (5000, 100), (3001, 520), (2500, 1500), (1500, 4097),
                                       (700, 8193), (523, 8008)])
def test_backward_many_rows(gpu_lib, rows, cols):
    Back(rows, cols, seed=1).check(gpu_lib)
    Back(rows, cols, post=False, gate=None, seed=1).check(gpu_lib)


@pytest.mark.parametrize("rows,cols", [(5, 9), (40, 300), (11, 3000), (3, 10001)])
def test_backward_parts(gpu_lib, rows, cols):
    """The norm alone; only one of the two incoming gradients; no weights; each output by itself has
    the bits that it has among the others."""
    for dtype in (BF, F32):
        Back(rows, cols, dtype, alone=True).check(gpu_lib)
        Back(rows, cols, dtype, alone=True, dh=False).check(gpu_lib)
        Back(rows, cols, dtype, dout=False).check(gpu_lib)
        Back(rows, cols, dtype, dh=False, gate="element").check(gpu_lib)
        Back(rows, cols, dtype, affine=False, gate=None).check(gpu_lib)
    b = Back(rows, cols)
    whole = b.run(gpu_lib)
    assert set(whole) == set(Back.NAMES)
    for n in Back.NAMES:
        assert torch.equal(b.run(gpu_lib, (n,))[n], whole[n]), n


def test_backward_without_rows(gpu_lib):
    e = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype, device="cuda")
    sums = [torch.full((96,), 7.0, device="cuda") for _ in range(3)]
    ws = e(gpu_lib.residual_norm_backward_workspace(0, 96), dtype=torch.uint8)
    gpu_lib.residual_norm_backward(e(0, 96), e(0, 96), rstd=e(0, dtype=F32), y=e(0, 96), post_rstd=e(0, dtype=F32),
                                   gate=e(96, dtype=F32), dresidual=e(0, 96), dy=e(0, 96), dgate=sums[0],
                                   dweight=sums[1], dpost_weight=sums[2], workspace=ws)
    assert all(bool((s == 0).all()) for s in sums)


@pytest.mark.parametrize("gate", [None, "column", "element"])
def test_backward_without_rows_or_statistics(gpu_lib, gate):
    """Without rows post_rstd is not needed, and the sums are 0, whatever the workspace held."""
    e = lambda *s, dtype=BF: torch.empty(*s, dtype=dtype, device="cuda")
    for cols in (96, 300, 1000, 4096, 9001):
        sums = [torch.full((cols,), 7.0, device="cuda") for _ in range(3)]
        ws = torch.full((gpu_lib.residual_norm_backward_workspace(0, cols),), 0x41, dtype=torch.uint8, device="cuda")
        g = {None: None, "column": torch.ones(cols, device="cuda"), "element": e(0, cols)}[gate]
        gpu_lib.residual_norm_backward(e(0, cols), gate=g, dgate=sums[0] if gate == "column" else None, dweight=sums[1],
                                       dpost_weight=sums[2], workspace=ws)
        assert all(bool((s == 0).all()) for s in sums[gate != "column":]), cols


def test_gradient_is_that_of_the_forward_pass(gpu_lib):
    """In fp32, the change of a random linear functional of h and out between two nearby inputs is what
    the gradients say.  Central differences: the step's square times third derivatives, and 2^-24 of the
    terms over the step; both far below the 1 % asked for here."""
    c = Back(7, 333, F32, F32)
    grads = c.run(gpu_lib)
    r = np.random.default_rng(0)
    for name in ("y", "residual", "weight", "post_weight", "gate"):
        t = getattr(c, name)
        d = torch.from_numpy(r.normal(size=tuple(t.shape))).float().cuda() * 0.02

        def loss(sign):
            keep = t.clone()
            t.add_(d, alpha=sign)
            o, _ = Case.run(c, gpu_lib)
            t.copy_(keep)
            return float((o["out"].double() * c.dout.double()).sum() + (o["h"].double() * c.dh.double()).sum())

        diff = (loss(1.0) - loss(-1.0)) / 2
        want = float((grads["d" + name].double() * d.double()).sum())
        size = float((grads["d" + name].double() * d.double()).abs().sum())
        assert abs(diff - want) <= 0.01 * size, (name, diff, want)


def test_offsets_past_32_bits(gpu_lib):
    """Matrices of more than 2^32 bytes: the last rows are those of a small call."""
    rows, cols = 70_001, 16384
    n = 5
    y = torch.zeros(rows, cols, dtype=F32, device="cuda")
    y[-n:] = randn(1, n, cols, dtype=F32)
    res = torch.zeros_like(y)
    res[-n:] = randn(2, n, cols, dtype=F32)
    h, out = torch.empty_like(y), torch.empty_like(y)
    rstd, rp = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    gpu_lib.residual_norm(y, res, h=h, out=out, rstd=rstd, post_rstd=rp, scale=0.5)
    small = [torch.empty(n, cols, device="cuda") for _ in range(2)] + [torch.empty(n, device="cuda") for _ in range(2)]
    gpu_lib.residual_norm(y[-n:], res[-n:], h=small[0], out=small[1], rstd=small[2], post_rstd=small[3], scale=0.5)
    for a, b in zip((h, out, rstd, rp), small):
        assert torch.equal(a[-n:], b)
    dy, dres = torch.empty_like(y), out  # out is not needed any more
    gpu_lib.residual_norm_backward(res, h, rstd=rstd, y=y, post_rstd=rp, scale=0.5, dresidual=dres, dy=dy)
    sdy, sdres = torch.empty_like(small[0]), torch.empty_like(small[0])
    gpu_lib.residual_norm_backward(res[-n:], small[0], rstd=small[2], y=y[-n:], post_rstd=small[3], scale=0.5,
                                   dresidual=sdres, dy=sdy)
    assert torch.equal(dy[-n:], sdy) and torch.equal(dres[-n:], sdres)


def test_streams_and_graphs(gpu_lib):
    """Another stream; a captured graph replayed with the program's own work between, and a second one
    that shares the workspace; the same call gives the same bits."""
    b = Back(500, 1040)
    want = b.run(gpu_lib)
    ws = torch.empty(gpu_lib.residual_norm_backward_workspace(b.rows, b.cols), dtype=torch.uint8, device="cuda")

    def call(out, stream=None):
        gpu_lib.residual_norm_backward(b.dout, b.h, rstd=b.rstd, weight=b.weight, dh=b.dh, y=b.y, post_rstd=b.post_rstd,
                                       post_weight=b.post_weight, gate=b.gate, scale=b.scale, workspace=ws, stream=stream,
                                       **out)

    new = lambda: {k: torch.full_like(v, float("nan")) for k, v in want.items()}
    side, out = torch.cuda.Stream(), new()
    side.wait_stream(torch.cuda.current_stream())
    call(out, side)
    side.synchronize()
    assert all(torch.equal(out[k], want[k]) for k in want)
    graphs, outs = [torch.cuda.CUDAGraph() for _ in range(2)], [new(), new()]
    for g, o in zip(graphs, outs):
        with torch.cuda.graph(g):
            call(o)
    for i in range(3):
        b.dout.mul_(0.5)
        want = b.run(gpu_lib)
        for g, o in zip(graphs, outs):
            for v in o.values():
                v.fill_(float("nan"))
            g.replay()
        torch.cuda.synchronize()
        for o in outs:
            assert all(torch.equal(o[k], want[k]) for k in want), i


@pytest.mark.parametrize("cols, rows", [(4096, 16500), (4095, 16500), (200, 340000)])
@pytest.mark.parametrize("post, gate", [(True, "column"), (True, None), (False, "column"), (True, "element"),
                                        (False, "element"), (False, None)])
def test_calls_past_the_caches(gpu_lib, cols, rows, post, gate):
    """Matrices that no cache holds are streamed: the rows of such a call have the bits that a call of
    few rows gives them, and its sums are those of the formula.  160 fp32 additions at most lie between a
    term and its sum over the rows (rows per team, 56 at most here, teams, groups per thread of the join, its 32
    threads), each off by half a step of at most the sum of the terms' sizes.  A term is a product of up to five
    roundings with dh', whose own are of its parts' sizes, at most 30 of them in the row's sum."""
    g = torch.Generator("cuda").manual_seed(7)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)
    y, res, dout, dh = (randn(rows, cols) for _ in range(4))
    w, wp = (1 + 0.1 * randn(cols) for _ in range(2))
    gt = None if gate is None else randn(cols) if gate == "column" else randn(rows, cols)
    rows_of = lambda t, s: t if s == slice(None) else t[s].clone()  # a buffer starts on 16 bytes

    def call(s, sums=True):
        e = lambda *shape, dtype=BF: torch.empty(*shape, dtype=dtype, device="cuda")
        ys, rs, ds, dhs = (rows_of(t, s) for t in (y, res, dout, dh))
        gs, n = rows_of(gt, s) if gate == "element" else gt, ys.shape[0]
        o = {"h": e(n, cols), "out": e(n, cols), "rstd": e(n, dtype=F32), "dres": e(n, cols), "dy": e(n, cols),
             "rp": e(n, dtype=F32) if post else None}
        gpu_lib.residual_norm(ys, rs, h=o["h"], out=o["out"], rstd=o["rstd"], weight=w, post_rstd=o["rp"],
                              post_weight=wp if post else None, gate=gs, scale=0.5)
        if gate == "element":
            o["dgate"] = e(n, cols)
        elif gate and sums:
            o["dgate"] = e(cols, dtype=F32)
        if sums:
            o["dw"] = e(cols, dtype=F32)
            o["dwp"] = e(cols, dtype=F32) if post else None
        ws = e(gpu_lib.residual_norm_backward_workspace(n, cols), dtype=torch.uint8)
        gpu_lib.residual_norm_backward(ds, o["h"], rstd=o["rstd"], weight=w, dh=dhs, y=ys, post_rstd=o["rp"],
                                       post_weight=wp if post else None, gate=gs, scale=0.5, dresidual=o["dres"],
                                       dy=o["dy"], dgate=o.get("dgate"), dweight=o.get("dw"), dpost_weight=o.get("dwp"),
                                       workspace=ws)
        return o

    whole = call(slice(None))
    for s in (slice(0, 300), slice(rows // 2, rows // 2 + 301), slice(rows - 77, rows)):
        few = call(s, sums=False)
        for k, t in few.items():
            assert t is None or torch.equal(whole[k][s], t), k
    d64 = lambda t: t.double()

    def near(got, term, size=None):
        return bool(((d64(got) - term.sum(0)).abs() <= 200 * 2.0 ** -24 * (term if size is None else size).abs().sum(0)).all())

    r = d64(whole["rstd"])[:, None]
    xh, gw = d64(whole["h"]) * r, d64(dout) * d64(w)
    assert near(whole["dw"], d64(dout) * xh)
    f = 0.5 * d64(y) * (d64(whole["rp"])[:, None] if post else 1.0)
    d = (d64(dh) + r * (gw - xh * (gw * xh).mean(1, keepdim=True))) * f
    size = (d64(dh).abs() + r * (gw.abs() + xh.abs() * (gw * xh).abs().mean(1, keepdim=True))) * f
    if post:
        k = 1.0 if gt is None else d64(gt)
        assert near(whole["dwp"], d * k, size * k)
    if gate == "column":
        assert near(whole["dgate"], d * (d64(wp) if post else 1.0), size * (d64(wp) if post else 1.0))
