"""AdamW's 8-bit states over many steps: rounded at random, they are the averages that states in fp32
hold, in the mean, at any beta; and what the binding asks for them."""
import warnings

import numpy as np
import pytest
import torch

from oracle import step_oracle as O

N, BLOCK = 2048, 512


def run(beta1, beta2, grad, steps, seed=3, lr=1e-3, n=N, block=BLOCK):
    """Per step (t, param, stored m and v, param, m and v in fp32, the variances that the roundings can have added to
    each m and v)."""
    z = np.zeros(n, np.float32)
    p, p32, m32, v32 = z, z, z, z
    (mc, me), (vc, ve) = O.state_write(z, block, 1), O.state_write(z, block, 2)
    var_m = var_v = np.zeros(n)
    for t in range(1, steps + 1):
        g = grad(t).astype(np.float32)
        hp = dict(lr=lr, beta1=beta1, beta2=beta2, eps=1e-8, step=t, weight_decay=0.0)
        m, old = (O.state_read(*s, block, i + 1).astype(np.float32) for i, s in enumerate(((mc, me), (vc, ve))))
        p, m, v = O.adamw(p, g, m, old, **hp)
        p32, m32, v32 = O.adamw(p32, g, m32, v32, **hp)
        bits = O.rounding_bits(seed, t, 0, np.arange(n))
        (mc, me), (vc, ve) = O.state_write(m, block, 1, bits[0]), O.state_write(v, block, 2, bits[1])
        # A part f of a step d is rounded with the variance f (1 - f) d^2, at most d^2 / 4 and at most d times the
        # distance from a code, such as the old value.  d: an eighth of the value or less, with a first
        # moment's least 2^-9 of its block's power of two.
        least = np.repeat(2.0 ** (me.astype(float) - 136), block)[:n]
        var_m = beta1 ** 2 * var_m + np.maximum(np.abs(m) / 8, least) ** 2 / 4
        var_v = beta2 ** 2 * var_v + np.minimum((v / 8) ** 2 / 4, v / 8 * np.abs(v.astype(float) - old))
        yield t, p, O.state_read(mc, me, block, 1), O.state_read(vc, ve, block, 2), p32, m32, v32, var_m, var_v


def same_mean(got, want, var):
    """Means over the elements within five standard deviations of the roundings'."""
    assert abs(got.mean() - want.mean()) <= 5 * np.sqrt(var.mean() / got.size), (got.mean(), want.mean())


@pytest.mark.parametrize("beta2", [0.9, 0.95, 0.98, 0.999])
def test_averages_after_a_tenfold_fall(beta2):
    """Normal gradients, a tenth as large from step 300 on."""
    r = np.random.default_rng(0)
    for t, p, m, v, p32, m32, v32, var_m, var_v in run(0.9, beta2, lambda t: r.normal(size=N) * (1 if t <= 300 else 0.1), 1000):
        if t in (20, 300, 500, 1000):
            same_mean(v, v32, var_v)
            same_mean(m, m32, var_m)
    # the bound above is a few per cent of the value
    assert 5 * np.sqrt(var_v.mean() / N) <= 0.06 * v32.mean()


@pytest.mark.parametrize("beta1,beta2", [(0.9, 0.95), (0.95, 0.999), (0.99, 0.999)])
def test_averages_of_constant_and_of_no_gradients(beta1, beta2):
    """A constant gradient for 200 steps, whose average grows ever more slowly, then none."""
    g = np.random.default_rng(1).uniform(0.5, 1.0, size=N)
    for t, p, m, v, p32, m32, v32, var_m, var_v in run(beta1, beta2, lambda t: g * (t <= 200), 400):
        if t in (10, 200, 230, 400):
            same_mean(v, v32, var_v)
            same_mean(m, m32, var_m)
    assert v.mean() < 0.9 * v32.max()  # it does fall


@pytest.mark.parametrize("beta2", [0.9, 0.94, 0.999])
def test_a_parameter_without_a_gradient_comes_to_rest(beta2):
    """Beside one with a gradient of 1 in its block.  The mean movement is E[m] / sqrt(v): E[m] is the average, and v, whose
    roundings have a standard deviation of a fifth at most, brings the mean of its root's reciprocal some 2 % up;
    a factor of two is far outside.  (Rounded to nearest, such a parameter moved by nearly lr a step for good.)"""
    g = np.full(512, 0.1)
    g[::256] = 1.0
    late = np.arange(512) % 256 != 0
    for t, p, m, v, p32, m32, *_ in run(0.9, beta2, lambda t: np.where(late & (t > 20), 0.0, g), 1500, n=512, block=256):
        pass
    assert abs(p[late].mean()) <= 2 * abs(p32[late].mean())
    assert not m[late].any() or np.abs(m[late]).mean() < 1e-6


def test_random_bits():
    """Means, and products of neighbours (in place, in step, in seed, the two moments), as of independent uniform
    numbers: within five standard deviations."""
    n = 1 << 16
    u = lambda *a, at=0: [(x + 0.5) / 2 ** 20 - 0.5 for x in O.rounding_bits(*a, at + np.arange(n))]
    for seed, step, counter, at in ((0, 1, 0, 0), (1, 1, 0, 0), (2 ** 64 - 1, 10 ** 12, -5, 2 ** 33), (7, 2, 1, 2 ** 32 - 512)):
        m, v = u(seed, step, counter, at=at)
        other = [m[1:], m[512:], v, v[1:], u(seed, step + 1, counter, at=at)[0], u(seed, step, counter + 1, at=at)[0],
                 u((seed + 1) % 2 ** 64, step, counter, at=at)[0], u(seed, step, counter, at=at + 2 ** 32)[0]]
        for x in (m, v):
            assert abs(x.mean()) <= 5 / np.sqrt(12 * n) and abs((x * x).mean() - 1 / 12) <= 5 / np.sqrt(180 * n)
        for x in other:
            assert abs((m[:x.size] * x).mean()) <= 5 / 12 / np.sqrt(x.size)
        for i in range(20):
            for x in O.rounding_bits(seed, step, counter, at + np.arange(n)):
                assert abs((x >> i & 1).mean() - 0.5) <= 5 / 2 / np.sqrt(n)


@pytest.mark.parametrize("moment", [1, 2])
def test_random_rounding(moment):
    """Values of a code stay, others go to one of their two neighbours, up in proportion; the largest too."""
    values = np.zeros(512)
    values[:127 if moment == 1 else 256] = O.fp8_values()[:127] * 2.0 ** -20 if moment == 1 else O.second_values(100)
    bits = O.rounding_bits(5, 1, 0, np.arange(512))[moment - 1]
    assert np.array_equal(O.state_read(*O.state_write(values, 512, moment, bits), 512, moment), values)
    r = np.random.default_rng(2)
    x = (r.normal(size=256) ** 2 * 10.0 ** r.uniform(-6, 0, size=256)).astype(np.float32)
    x = np.maximum(x, x.max() * np.float32(2.0 ** -28))  # above what a second moment can hold
    x[0] = 1.9 * 2.0 ** np.ceil(np.log2(x.max()))  # between the largest code of its binade and the next
    got = np.stack([O.state_read(*O.state_write(x, 256, moment, O.rounding_bits(5, t, 0, np.arange(256))[moment - 1]), 256, moment)
                    for t in range(4000)])
    assert all(np.unique(c).size <= 2 for c in got.T) and np.unique(got[:, 0]).size == 2
    # a standard deviation of half a step at most; a step is an eighth of the value at most, or a first moment's
    # least, 2^-9 of a power of two below the largest value / 224
    step = np.maximum(x / 8, x.max() / 224 * 2.0 ** -9 if moment == 1 else 0.0)
    assert np.all(np.abs(got.mean(0) - x) <= 5 * step / 2 / np.sqrt(4000) + 1e-7 * x)


# -- the binding --------------------------------------------------------------------------------

if not torch.cuda.is_available():
    from bit_gradient_compression_amd import loco

    class Calls:
        """In the library's place: keeps the rounding of the last step."""

        def loco_adamw_ex(self, plan, options, scale, rounding, stream):
            self.rounding, self.options = rounding and rounding._obj, options._obj
            return 0

    @pytest.fixture
    def plan(monkeypatch):
        monkeypatch.setattr(loco, "_device", lambda: 0)
        monkeypatch.setattr(loco, "_stream", lambda stream, dev: 0)
        p = loco.AdamwTensors([])
        p.bits = 8
        monkeypatch.setattr(loco, "_lib", Calls())
        return p

    def test_eight_bits_without_a_seed(plan):
        """Refused with the default beta2; else a warning, once."""
        with pytest.raises(ValueError, match="seed"):
            loco.adamw(plan, step=1, lr=1e-3)
        with pytest.warns(RuntimeWarning, match="seed"):
            loco.adamw(plan, step=1, lr=1e-3, beta2=0.95)
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            loco.adamw(plan, step=2, lr=1e-3, beta2=0.95)
            plan.bits = 32
            loco.adamw(plan, step=1, lr=1e-3)
            assert loco._lib.options.beta2 == 0.999 and loco._lib.rounding is None

    def test_seeds(plan, monkeypatch):
        with warnings.catch_warnings():
            warnings.simplefilter("error")
            for seed, want in ((0, 0), (5, 5), (-1, 2 ** 64 - 1), (2 ** 70 + 3, 3)):
                loco.adamw(plan, step=1, lr=1e-3, seed=seed)
                assert (loco._lib.rounding.seed, loco._lib.rounding.counter) == (want, None)
            monkeypatch.setattr(loco, "_ptr", lambda t, dev: None if t is None else 4096)
            loco.adamw(plan, step=1, lr=1e-3, seed=torch.zeros(1, dtype=torch.int64))
            assert (loco._lib.rounding.seed, loco._lib.rounding.counter) == (0, 4096)
        for bad, err in ((torch.zeros(2, dtype=torch.int64), ValueError), (torch.zeros(1, dtype=torch.int32), TypeError),
                         (torch.zeros(1), TypeError), (1.5, TypeError), ("7", TypeError)):
            with pytest.raises(err):
                loco.adamw(plan, step=1, lr=1e-3, seed=bad)

    def test_rounding_of_the_c_call():
        """The counter is refused where the step writes, and off 16 bytes."""
        import ctypes
        lib = loco.load()
        tensor = loco.AdamwTensor(*(0x100000000 * (i + 1) for i in range(7)), 1000, 0.1)
        arr, p = (loco.AdamwTensor * 1)(tensor), loco.AdamwPlan()
        opt = loco.AdamwOptions(1e-3, 0.9, 0.99, 1e-8, 1)
        call = lambda c, s=None: lib.loco_adamw_ex(ctypes.byref(p), ctypes.byref(opt), s,
                                                   ctypes.byref(loco.AdamwRounding(1, c)), None)
        assert call(None) == loco.LOCO_ERR_INVALID  # a plan that is none
        assert lib.loco_adamw_plan(None, 0, loco.LOCO_F32, loco.LOCO_BF16, 8, 256, None, 0, ctypes.byref(p), None) == 0
        assert call(None) == call(0x900000000) == lib.loco_adamw_ex(ctypes.byref(p), ctypes.byref(opt), None, None, None) == 0
        p.ntensors, p.tensors = 1, arr
        for i in (0, 2, 3, 4, 5, 6):
            assert call(getattr(tensor, tensor._fields_[i][0])) == loco.LOCO_ERR_INVALID, i
        assert call(tensor.m - 4) == loco.LOCO_ERR_INVALID and call(0x900000008) == loco.LOCO_ERR_ALIGN
        assert call(0x900000000, 0xA00000004) == loco.LOCO_ERR_ALIGN
