"""AdamW's 8-bit states rounded at random: bit for bit against the oracle with the same random bits."""
import numpy as np
import pytest
import torch

from oracle import step_oracle as O
from test_gpu_adamw import BF, F32, F8, HP, KINDS, SIZES, U8, Guarded, Tensor, bits, same

pytestmark = pytest.mark.gpu


class Random(Tensor):
    """A tensor whose first element is the step's element `place`."""

    def check(self, place, seed, step, counter=0):
        p, m, v = self.want
        same(self.p.t, p, "param")
        if self.copy is not None:
            same(self.copy.t, p, "copy")
        u = O.rounding_bits(seed, step, counter, place + np.arange(self.n))
        for c, e, x, k in ((self.m, self.me, m, 1), (self.v, self.ve, v, 2)):
            wc, we = O.state_write(x, self.block, k, u[k - 1])
            assert np.array_equal(bits(e.t), we), ("exps", k)
            assert np.array_equal(bits(c.t), wc), ("codes", k)
        for x in vars(self).values():
            if isinstance(x, Guarded):
                x.check()


def places(ts):
    at, out = 0, []
    for t in ts:
        out.append(at)
        at += -(-t.n // 512) * 512
    return out


@pytest.mark.parametrize("param,grad,state_bits,block,copy", [k for k in KINDS if k[2] == 8])
def test_random_steps(gpu_lib, param, grad, state_bits, block, copy):
    """Every kind of tensor at sizes around the blocks and the tile, an empty one among them; three steps."""
    ts = [Random(i, n, param, grad, 8, block, copy) for i, n in enumerate(SIZES[:7] + [0] + SIZES[7:])]
    scale = torch.tensor([0.37], device="cuda")
    tensors = gpu_lib.AdamwTensors([t.args(0.1 if i % 2 else 0.0) for i, t in enumerate(ts)], block=block)
    for step, seed in ((1, 0), (2, 12345), (1000, 2 ** 64 - 1)):
        for i, t in enumerate(ts):
            t.expect(0.1 if i % 2 else 0.0, np.float32(0.37) if step > 1 else None, step=step)
        gpu_lib.adamw(tensors, **{**HP, "step": step}, grad_scale=scale if step > 1 else None, seed=seed)
        torch.cuda.synchronize()
        for t, at in zip(ts, places(ts)):
            t.check(at, seed, step)


@pytest.mark.parametrize("hp", [dict(beta1=0.0), dict(beta2=0.0), dict(step=10 ** 12), dict(beta1=0.99999, beta2=0.9999999)])
def test_random_hyper_parameters(gpu_lib, hp):
    t = Random(9, 1500, F32, BF, 8, 512, True)
    t.expect(0.3, **hp)
    gpu_lib.adamw([t.args(0.3)], block=512, seed=3, **{**HP, **hp})
    torch.cuda.synchronize()
    t.check(0, 3, hp.get("step", HP["step"]))


def test_random_of_zero_tiny_large_and_lost(gpu_lib):
    """Zero states and gradients, subnormal ones, squares past the largest code and past fp32, infinities and NaN."""
    n = 1200
    r = np.random.default_rng(0)
    g = np.zeros(n)
    g[:256] = r.normal(size=256)
    g[256:300], g[300:310] = 1e-20, 1e-30
    g[320:384] = r.normal(size=64) * 1e-18
    g[384:448] = r.normal(size=64) * 1e-24
    g[448:512] = 1.0 - 2.0 ** -20  # squares between the largest code of a binade and the next
    g[512:576] = r.uniform(1.7e19, 1.85e19, size=64) * np.sqrt(20.0)  # around 15/8 2^127 of v
    g[640], g[704], g[770], g[1199] = 3e38, np.nan, np.inf, -np.inf
    t = Random(5, n, F32, F32, 8, 64, True, m=np.zeros(n), v=np.zeros(n), g=g)
    for step in (1, 2, 3):
        t.expect(0.01, step=step)
        gpu_lib.adamw([t.args(0.01)], block=64, seed=11, **{**HP, "step": step})
        torch.cuda.synchronize()
        t.check(0, 11, step)
        v = t.want[2]
        fine = np.isfinite(v) & (bits(t.ve.t) != 255)[np.arange(n) // 64]
        assert np.array_equal(bits(t.v.t)[fine] > 0, v[fine] > 0)  # what is not 0 is not stored as 0


def test_more_tensors_than_one_launch_fills(gpu_lib):
    """Past the descriptions that a launch carries, as a plain list: each has its own places."""
    ts = [Random(i, (i * 37) % 1500 if i % 9 else 0, BF, BF, 8, 128, False) for i in range(130)]
    for t in ts:
        t.expect(0.05)
    gpu_lib.adamw([t.args()[:4] for t in ts], weight_decay=0.05, block=128, seed=77, **HP)
    torch.cuda.synchronize()
    for t, at in zip(ts, places(ts)):
        t.check(at, 77, HP["step"])


def test_seed_without_eight_bits(gpu_lib):
    """States in fp32 do not take part."""
    a, b = (Tensor(3, 3000, F32, BF, 32, 256, True) for _ in range(2))
    gpu_lib.adamw([a.args(0.1)], seed=5, **HP)
    gpu_lib.adamw([b.args(0.1)], **HP)
    for x, y in ((a.p, b.p), (a.m, b.m), (a.v, b.v), (a.copy, b.copy)):
        assert np.array_equal(bits(x.t), bits(y.t))


@pytest.mark.parametrize("counter", [0, 1, -3, 2 ** 62])
def test_counter(gpu_lib, counter):
    """A seed in device memory is the counter of the seed 0."""
    t = Random(13, 2100, BF, BF, 8, 256, False)
    t.expect(0.0)
    gpu_lib.adamw([t.args(0.0)], seed=torch.tensor([counter], device="cuda"), **HP)
    torch.cuda.synchronize()
    t.check(0, 0, HP["step"], counter)


def test_captured_steps_with_a_counter(gpu_lib):
    """A captured step that raises its counter takes other bits at each replay: those of eager steps with the
    counters, on another stream."""
    a, b = (Random(11, 5000, F32, BF, 8, 256, True) for _ in range(2))
    ca, cb = (torch.zeros(1, dtype=torch.int64, device="cuda") for _ in range(2))
    ta, tb = (gpu_lib.AdamwTensors([t.args(0.1)]) for t in (a, b))
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ca.add_(1)
        gpu_lib.adamw(ta, seed=ca, **HP)
    before = None
    for i in range(3):
        a.expect(0.1)
        graph.replay()
        torch.cuda.synchronize()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            cb.add_(1)
            gpu_lib.adamw(tb, seed=cb, **HP)
        side.synchronize()
        for x, y in zip((a.p, a.m, a.v, a.me, a.ve, a.copy), (b.p, b.m, b.v, b.me, b.ve, b.copy)):
            assert np.array_equal(bits(x.t), bits(y.t)), i
        a.check(0, 0, HP["step"], i + 1)


def test_places_past_32_bits(gpu_lib):
    """A tensor of more than 2^32 elements: its first, some around 2^32 and its last blocks."""
    n = (1 << 32) + 1300
    p, g = (torch.empty(n, dtype=BF, device="cuda") for _ in range(2))
    p.zero_()
    g.fill_(0.013)
    m = torch.zeros(n, dtype=U8, device="cuda").view(F8), torch.zeros(-(-n // 64), dtype=U8, device="cuda")
    v = torch.zeros(n, dtype=U8, device="cuda"), torch.zeros(-(-n // 64), dtype=U8, device="cuda")
    gpu_lib.adamw([(p, g, m, v)], block=64, seed=21, **{**HP, "step": 1})
    for lo, hi in ((0, 1024), ((1 << 32) - 512, (1 << 32) + 512), (n - 1300, n)):
        k = hi - lo
        z = np.zeros(k, np.float32)
        _, wm, wv = O.adamw(z, g[lo:hi].float().cpu().numpy(), z, z, weight_decay=0.0, **{**HP, "step": 1})
        u = O.rounding_bits(21, 1, 0, lo + np.arange(k))
        for (c, e), x, moment in ((m, wm, 1), (v, wv, 2)):
            wc, we = O.state_write(x, 64, moment, u[moment - 1])
            assert np.array_equal(bits(c[lo:hi]), wc) and np.array_equal(bits(e[lo // 64:-(-hi // 64)]), we), (lo, moment)
            assert np.unique(wc).size == 2


@pytest.mark.parametrize("beta2", [0.95, 0.999])
def test_states_follow_fp32_states(gpu_lib, beta2):
    """400 steps with gradients that fall tenfold after 200: the means of a million elements within 1 % of fp32
    states' (a standard deviation of 0.4 of the value at most, 2^-10 of that for the mean)."""
    n = 1 << 20
    z = lambda k=n, dtype=U8: torch.zeros(k, dtype=dtype, device="cuda")
    p8, p32, g, m32, v32 = (z(n, F32) for _ in range(5))
    m, v = (z().view(F8), z(n // 256)), (z(), z(n // 256))
    rm, rv = z(n, F32), z(n, F32)
    gen = torch.Generator("cuda").manual_seed(1)
    t8, t32 = gpu_lib.AdamwTensors([(p8, g, m, v)]), gpu_lib.AdamwTensors([(p32, g, m32, v32)])
    states = gpu_lib.AdamwStates([(m, rm), (v, rv)])
    for t in range(1, 401):
        g.normal_(0.3, 1.0, generator=gen)
        if t > 200:
            g.mul_(0.1)
        gpu_lib.adamw(t8, step=t, lr=1e-3, beta2=beta2, seed=4)
        gpu_lib.adamw(t32, step=t, lr=1e-3, beta2=beta2)
    gpu_lib.adamw_state_read(states)
    near = lambda a, b: abs(float(a.double().mean() / b.double().mean()) - 1)
    assert near(rv, v32) <= 0.01 and near(rm, m32) <= 0.01
    # v's spread, 0.4 of the value at most, adds 3/8 of its square to the mean of its root's reciprocal: 2 to 6 %
    # over the steps, most of which are at half of that spread
    assert near(p8, p32) <= 0.05
