"""AdamW over many tensors, bit for bit against its fp32 form, and its 8-bit states against
their definition."""
import numpy as np
import pytest
import torch

from layer_util import Guarded
from oracle import step_oracle as O

pytestmark = pytest.mark.gpu
BF, F32, F8, U8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn, torch.uint8
HP = dict(lr=3e-3, beta1=0.9, beta2=0.95, eps=1e-8, step=7)
SIZES = [1, 3, 4, 63, 64, 65, 255, 256, 257, 511, 512, 513, 1000, 4099, 20000]


def guarded(values, dtype):
    g = Guarded(values.shape, dtype)
    g.t.copy_(values)
    return g


def bits(t):
    t = t.detach().cpu().contiguous()
    return t.view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()]).numpy()


def same(got, want32, what):
    """got holds the float32 array want32, rounded to got's type; NaNs by place only."""
    want = torch.from_numpy(np.ascontiguousarray(want32)).to(got.dtype)
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got.cpu()), nan), what
    keep = ~nan.numpy()
    assert np.array_equal(bits(got)[keep], bits(want)[keep]), what


class Tensor:
    """One tensor with its states between guards, and the oracle's float32 copies."""

    def __init__(self, seed, n, param, grad, state_bits, block, copy, m=None, v=None, g=None):
        r = np.random.default_rng(seed)
        f = lambda x: torch.from_numpy(x.astype(np.float32))
        self.bits, self.block, self.n = state_bits, block, n
        self.p = guarded(f(r.normal(size=n)).to(param), param)
        self.g = guarded(f(r.normal(size=n) * np.exp(r.normal(size=n)) * 1e-2 if g is None else g).to(grad), grad)
        m = r.normal(size=n) * 1e-3 * np.exp(r.normal(size=n)) if m is None else m
        v = r.normal(size=n) ** 2 * 1e-4 * 10.0 ** r.uniform(-9, 0, size=n) if v is None else v
        self.copy = guarded(torch.zeros(n), BF) if copy else None
        if state_bits == 32:
            self.m, self.v = guarded(f(m), F32), guarded(f(v), F32)
        else:
            (mc, me), (vc, ve) = O.state_write(m, block, 1), O.state_write(v, block, 2)
            self.m, self.me = guarded(torch.from_numpy(mc).view(F8), F8), guarded(torch.from_numpy(me), U8)
            self.v, self.ve = guarded(torch.from_numpy(vc), U8), guarded(torch.from_numpy(ve), U8)

    def args(self, decay=None):
        m, v = (self.m.t, self.v.t) if self.bits == 32 else ((self.m.t, self.me.t), (self.v.t, self.ve.t))
        return self.p.t, self.g.t, m, v, None if self.copy is None else self.copy.t, decay

    def state(self):
        f = lambda t: t.detach().float().cpu().numpy()
        if self.bits == 32:
            return f(self.m.t), f(self.v.t)
        return tuple(O.state_read(bits(c.t), bits(e.t), self.block, k).astype(np.float32)
                     for c, e, k in ((self.m, self.me, 1), (self.v, self.ve, 2)))

    def expect(self, decay, grad_scale=None, **hp):
        f = lambda t: t.detach().float().cpu().numpy()
        m, v = self.state()
        self.want = O.adamw(f(self.p.t), f(self.g.t), m, v, weight_decay=decay, grad_scale=grad_scale, **{**HP, **hp})

    def check(self):
        p, m, v = self.want
        same(self.p.t, p, "param")
        if self.copy is not None:
            same(self.copy.t, p, "copy")
        if self.bits == 32:
            same(self.m.t, m, "m")
            same(self.v.t, v, "v")
        else:
            for c, e, x, k in ((self.m, self.me, m, 1), (self.v, self.ve, v, 2)):
                wc, we = O.state_write(x, self.block, k)
                assert np.array_equal(bits(e.t), we), ("exps", k)
                assert np.array_equal(bits(c.t), wc), ("codes", k)
        for x in vars(self).values():
            if isinstance(x, Guarded):
                x.check()


KINDS = [(p, g, s, b, c) for p, g in ((F32, BF), (F32, F32), (BF, BF), (BF, F32))
         for s, b in ((32, 256), (8, 64), (8, 128), (8, 256), (8, 512)) for c in ((False, True) if p == F32 else (False,))]


@pytest.mark.parametrize("param,grad,state_bits,block,copy", KINDS)
def test_adamw(gpu_lib, param, grad, state_bits, block, copy):
    """Every kind of tensor at sizes around the blocks and the tile, three steps."""
    ts = [Tensor(i, n, param, grad, state_bits, block, copy) for i, n in enumerate(SIZES)]
    scale = torch.tensor([0.37], device="cuda")
    tensors = gpu_lib.AdamwTensors([t.args(0.1 if i % 2 else 0.0) for i, t in enumerate(ts)], block=block)
    for step in (1, 2, 1000):
        for i, t in enumerate(ts):
            t.expect(0.1 if i % 2 else 0.0, np.float32(0.37) if step > 1 else None, step=step)
        gpu_lib.adamw(tensors, **{**HP, "step": step}, grad_scale=scale if step > 1 else None)
        torch.cuda.synchronize()
        for t in ts:
            t.check()


@pytest.mark.parametrize("state_bits", [32, 8])
def test_more_tensors_than_one_launch(gpu_lib, state_bits):
    """Past 48 tensors, empty ones among them, given as a plain list with one decay for all."""
    ts = [Tensor(i, (i * 37) % 700 if i % 9 else 0, BF, BF, state_bits, 128, False) for i in range(130)]
    for t in ts:
        t.expect(0.05)
    gpu_lib.adamw([t.args()[:4] for t in ts], weight_decay=0.05, block=128, **HP)
    torch.cuda.synchronize()
    for t in ts:
        t.check()


@pytest.mark.parametrize("state_bits", [32, 8])
def test_zero_and_tiny_states(gpu_lib, state_bits):
    """A first step from zero states; zero gradients; gradients whose squares are subnormal or 0;
    blocks of zeros beside others."""
    n = 1024
    g = np.zeros(n)
    g[:256] = np.random.default_rng(0).normal(size=256)
    g[256:300] = 1e-20
    g[300:310] = 1e-30
    g[768:] = np.random.default_rng(1).normal(size=256) * 1e-18
    t = Tensor(5, n, F32, F32, state_bits, 64, True, m=np.zeros(n), v=np.zeros(n), g=g)
    for step in (1, 2):
        t.expect(0.01, step=step)
        gpu_lib.adamw([t.args(0.01)], block=64, **{**HP, "step": step})
        torch.cuda.synchronize()
        t.check()
    if state_bits == 8:  # what is not 0 is not stored as 0
        v = t.want[2]
        assert np.array_equal(bits(t.v.t) > 0, v > 0)


@pytest.mark.parametrize("state_bits", [32, 8])
def test_infinities_and_nans(gpu_lib, state_bits):
    """They reach their own element; with 8-bit states their block's states, which then read as NaN."""
    n = 2000
    g = np.random.default_rng(2).normal(size=n)
    g[5], g[700], g[1999] = np.nan, np.inf, -np.inf
    g[1300] = 3e38  # its square overflows
    t = Tensor(6, n, F32, F32, state_bits, 64, False, g=g)
    t.expect(0.01)
    gpu_lib.adamw([t.args(0.01)], block=64, **HP)
    torch.cuda.synchronize()
    t.check()
    if state_bits == 8:
        assert set(np.flatnonzero(bits(t.ve.t) == 255)) == {5 // 64, 700 // 64, 1300 // 64, 1999 // 64}
        t.expect(0.01)  # the next step from such states
        assert np.isnan(t.want[1][:64]).all()
        gpu_lib.adamw([t.args(0.01)], block=64, **HP)
        torch.cuda.synchronize()
        t.check()


@pytest.mark.parametrize("scale", [0.0, 1.0, float("inf"), float("nan")])
def test_grad_scale_values(gpu_lib, scale):
    for state_bits in (32, 8):
        t = Tensor(8, 777, BF, BF, state_bits, 256, False)
        t.expect(0.0, np.float32(scale))
        gpu_lib.adamw([t.args(0.0)], grad_scale=torch.full((1,), scale, device="cuda"), **HP)
        torch.cuda.synchronize()
        t.check()


@pytest.mark.parametrize("hp", [dict(lr=0.0), dict(lr=-1e-3), dict(beta1=0.0), dict(beta2=0.0), dict(beta1=0.0, beta2=0.0),
                                dict(eps=1.0), dict(step=1), dict(step=10 ** 12), dict(beta1=0.99999, beta2=0.9999999)])
def test_hyper_parameters(gpu_lib, hp):
    for state_bits in (32, 8):
        t = Tensor(9, 1500, F32, BF, state_bits, 512, True)
        t.expect(0.3, **hp)
        gpu_lib.adamw([t.args(0.3)], block=512, **{**HP, **hp})
        torch.cuda.synchronize()
        t.check()


def test_offsets_past_32_bits(gpu_lib):
    """A tensor whose fp32 states pass 2^32 bytes: its ends and some of its middle."""
    n = (1 << 30) + 4097
    p = torch.zeros(n, dtype=BF, device="cuda")
    g = torch.ones(n, dtype=BF, device="cuda")
    m, v = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    g[-1], g[1 << 30], g[-600] = 3.0, -5.0, 0.0
    gpu_lib.adamw([(p, g, m, v)], **{**HP, "step": 1})
    at = torch.tensor([0, 1, 511, 512, 1 << 29, (1 << 30) - 1, 1 << 30, n - 600, n - 2, n - 1], device="cuda")
    z = np.zeros(at.numel(), np.float32)
    want = O.adamw(z, g[at].float().cpu().numpy(), z, z, weight_decay=0.0, **{**HP, "step": 1})
    for t, w in zip((p, m, v), want):
        same(t[at], w, "far element")
    assert bool((m[: 1 << 29] == m[0]).all()) and int((m != m[0]).sum()) == 3


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("block", [64, 128, 256, 512])
def test_state_read_and_write(gpu_lib, dtype, block):
    """Every code under steps over the whole range reads as its definition, and writing what was read
    gives codes that read as the same; random values are rounded as the definition says."""
    n = 3 * 512 + 300
    r = np.random.default_rng(block)
    nb = -(-n // block)
    for moment, ct in ((1, F8), (2, U8)):
        codes = np.arange(n).astype(np.uint8)
        exps = r.integers(10, 240, size=nb).astype(np.uint8) if moment == 1 else r.integers(0, 254, size=nb).astype(np.uint8)
        exps[1] = 255
        if moment == 1:
            codes[codes & 127 == 127] = 1
        c, e = guarded(torch.from_numpy(codes).view(ct), ct), guarded(torch.from_numpy(exps), U8)
        out = Guarded((n,), dtype, float("nan"))
        gpu_lib.adamw_state_read([((c.t, e.t), out.t)], block=block)
        want = O.state_read(codes, exps, block, moment)
        same(out.t, want.astype(np.float32), "read")
        c2, e2 = Guarded((n,), ct, None), Guarded((nb,), U8, 0xAA)
        back = Guarded((n,), dtype, float("nan"))
        gpu_lib.adamw_state_write([((c2.t, e2.t), out.t)], block=block)
        gpu_lib.adamw_state_read([((c2.t, e2.t), back.t)], block=block)
        torch.cuda.synchronize()
        nan = torch.isnan(out.t)
        lost = nan.view(-1)  # infinities of the lost block's other codes become NaN
        lost = lost | torch.isinf(out.t)
        assert torch.equal(back.t[~lost], out.t[~lost]) and bool(torch.isnan(back.t[lost]).all())
        x = torch.from_numpy((np.abs(r.normal(size=n)) * 10.0 ** r.uniform(-9, 2, size=n)).astype(np.float32)).to(dtype)
        if moment == 1:
            x = x * torch.from_numpy(np.where(r.random(n) < 0.5, 1.0, -1.0)).to(dtype)
        x[3 * 64:5 * 64] = 0
        values = guarded(x, dtype)
        gpu_lib.adamw_state_write([((c2.t, e2.t), values.t)], block=block)
        torch.cuda.synchronize()
        wc, we = O.state_write(x.float().numpy(), block, moment)
        assert np.array_equal(bits(e2.t), we) and np.array_equal(bits(c2.t), wc)
        for gd in (c, e, out, c2, e2, back, values):
            gd.check()


def test_states_of_many_tensors(gpu_lib):
    """Past one launch's 64 states, both moments mixed, empty ones among them."""
    r = np.random.default_rng(4)
    ss = []
    for i in range(150):
        n, moment = int(r.integers(0, 900)), 1 + i % 2
        x = np.abs(r.normal(size=n)).astype(np.float32)
        c, e = O.state_write(x, 256, moment)
        ct = F8 if moment == 1 else U8
        ss.append((torch.from_numpy(c).view(ct).cuda(), torch.from_numpy(e).cuda(), torch.zeros(n, device="cuda"), c, e, moment))
    gpu_lib.adamw_state_read([((c, e), x) for c, e, x, *_ in ss])
    torch.cuda.synchronize()
    for _, _, x, c, e, moment in ss:
        same(x, O.state_read(c, e, 256, moment).astype(np.float32), moment)


def test_streams_and_graphs(gpu_lib):
    """A step on another stream, and one captured and replayed with the program's own work between:
    each replay is one more step with the captured hyper-parameters and what the gradients hold then."""
    for state_bits in (32, 8):
        a, b = (Tensor(11, 5000, F32, BF, state_bits, 256, True) for _ in range(2))
        scale = torch.ones(1, device="cuda")
        ta, tb = (gpu_lib.AdamwTensors([t.args(0.1)]) for t in (a, b))
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        gpu_lib.adamw(ta, grad_scale=scale, stream=side, **HP)
        torch.cuda.current_stream().wait_stream(side)
        gpu_lib.adamw(tb, grad_scale=scale, **HP)
        torch.cuda.synchronize()
        assert np.array_equal(bits(a.p.t), bits(b.p.t))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            gpu_lib.adamw(ta, grad_scale=scale, **HP)
        for i in range(3):
            for t in (a, b):
                t.g.t.mul_(0.5).add_(0.01 * i)
            scale.fill_(1.0 / (i + 1))
            graph.replay()
            gpu_lib.adamw(tb, grad_scale=scale, **HP)
            torch.cuda.synchronize()
            for x, y in zip((a.p, a.m, a.v, a.copy), (b.p, b.m, b.v, b.copy)):
                assert np.array_equal(bits(x.t), bits(y.t)), i


def test_memory_is_kept_by_the_description(gpu_lib):
    """The description keeps the memory of a tensor whose last other name has gone."""
    p, g = torch.ones(4096, device="cuda"), torch.ones(4096, device="cuda")
    m, v = torch.zeros(4096, device="cuda"), torch.zeros(4096, device="cuda")
    kept = gpu_lib.AdamwTensors([(p, g, m, v)])
    where = g.data_ptr()
    del g
    other = torch.zeros(4096, device="cuda")
    assert other.data_ptr() != where
    gpu_lib.adamw(kept, **HP)
    assert bool((m != 0).all())


def test_description_and_streams(gpu_lib):
    """A description made on one stream is there for a step on another that waits for nothing else; it
    cannot be made while a graph is captured, but a plain list can be stepped there."""
    a, b = (Tensor(12, 3000, BF, BF, 8, 64, False) for _ in range(2))
    torch.cuda.synchronize()
    busy, side = torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.stream(busy):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(20):
            big = big @ big * 1e-2
        ta = gpu_lib.AdamwTensors([a.args(0.1)], block=64)
    gpu_lib.adamw(ta, stream=side, **HP)
    gpu_lib.adamw([b.args(0.1)], block=64, stream=side.cuda_stream, **HP)
    side.synchronize()
    for x, y in zip((a.p, a.m, a.v, a.me), (b.p, b.m, b.v, b.me)):
        assert np.array_equal(bits(x.t), bits(y.t))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gpu_lib.adamw([a.args(0.1)], block=64, **HP)
        with pytest.raises(RuntimeError, match="captured"):
            gpu_lib.AdamwTensors([b.args(0.1)], block=64)
    for _ in range(3):
        graph.replay()
        gpu_lib.adamw([b.args(0.1)], block=64, **HP)
        torch.cuda.synchronize()
        for x, y in zip((a.p, a.m, a.v), (b.p, b.m, b.v)):
            assert np.array_equal(bits(x.t), bits(y.t))


def test_a_list_on_a_stream_of_its_own(gpu_lib):
    """The table of a plain list is not memory that the current stream has freed and is still to write."""
    a, b = (Tensor(13, 5000, BF, BF, 8, 64, False) for _ in range(2))
    gpu_lib.adamw([b.args(0.1)], block=64, **HP)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    big = torch.randn(4096, 4096, device="cuda")
    for _ in range(20):
        big = big @ big * 1e-2
    for n in (256, 512, 1024):
        torch.empty(n, dtype=torch.uint8, device="cuda").fill_(255)
    gpu_lib.adamw([a.args(0.1)], block=64, stream=side, **HP)
    side.synchronize()
    torch.cuda.synchronize()
    for x, y in zip((a.p, a.m, a.v), (b.p, b.m, b.v)):
        assert np.array_equal(bits(x.t), bits(y.t))
