"""Helpers of the layer operators' GPU tests: guarded buffers, inputs and error bounds.

Bounds count roundings.  U is fp32's unit roundoff, half a step relative to the value; the
result's own rounding to bf16 adds 2^-8 of the value.  A sum that a kernel forms in lanes,
waves and partial sums passes each term through `seq` additions; each additon is allowed two
units, since the matrix cores' internal additions may truncate where IEEE ones round."""
import numpy as np
import torch

U = 2.0 ** -24
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}
ACT = {"none": 0, "relu": 1, "gelu": 2, "silu": 3}


class Guarded:
    """A tensor between two 4 KiB stretches of a pattern that the call must leave alone."""

    def __init__(self, shape, dtype, fill=None):
        n = int(np.prod(shape))
        size = torch.empty(0, dtype=dtype).element_size()
        self.raw = torch.full((4096 + -(-n * size // 16) * 16 + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        self.n, self.used = n, n * size
        self.t = self.raw[4096:4096 + self.used].view(dtype).view(shape)
        if fill is not None:
            self.t.fill_(fill)

    def check(self):
        assert bool((self.raw[:4096] == 0xA5).all()) and bool((self.raw[4096 + self.used:] == 0xA5).all()), \
            "written outside the buffer"


def guarded(shape, dtype):
    """Outputs start as NaN (codes as -86), so that an element left out shows."""
    return Guarded(shape, dtype, float("nan") if dtype.is_floating_point else (0xAA if dtype == torch.uint8 else -86))


def new_checkpoint(rows, cols, block):
    return guarded((rows, cols), torch.int8), guarded((rows, -(-cols // block)), torch.uint8)


def f64(t):
    return t.detach().double().cpu().numpy()


def randn(seed, *shape, dtype=torch.bfloat16, scale=1.0, shift=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g, dtype=torch.float64) * scale + shift).to(dtype).cuda()


def random_checkpoint(seed, rows, cols, block):
    """Codes over their whole range, -128 too, and steps that put values around 1."""
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(-128, 128, (rows, cols), generator=g).to(torch.int8).cuda()
    exps = torch.randint(117, 123, (rows, -(-cols // block)), generator=g).to(torch.uint8).cuda()
    return codes, exps


def assert_near(got, want, bound, what=""):
    """|got - want| <= bound everywhere, NaNs in the same places."""
    got, want, bound = f64(got) if isinstance(got, torch.Tensor) else got, np.asarray(want), np.asarray(bound)
    assert got.shape == want.shape, (what, got.shape, want.shape)
    nan = np.isnan(want)
    assert np.array_equal(np.isnan(got), nan), (what, "NaNs in other places", int(np.isnan(got).sum()), int(nan.sum()))
    inf = np.isinf(want)
    assert np.array_equal(got[inf], want[inf]), what
    fine = ~nan & ~inf
    d = np.abs(got[fine] - want[fine])
    b = np.broadcast_to(bound, want.shape)[fine]
    bad = ~(d <= b)
    assert not bad.any(), (what, f"{int(bad.sum())} of {bad.size} outside", float(d[bad].max()),
                           float((d[bad] / np.maximum(b[bad], 1e-300)).max()))


def round_bound(want, dtype):
    """The rounding of a result to its type (and the smallest subnormal step, for results near 0)."""
    return HALF[dtype] * np.abs(want) + 2.0 ** -133


def act_bound(z, dz, name):
    """Error of act(z) in fp32, for an error dz of z: the derivative is at most 1.13, the
    sigmoid's argument x has a few roundings and enters an exponential (an error of |x| times
    theirs), exp and reciprocal have one unit each."""
    from oracle import layer_oracle as O
    x = np.abs(O.act_arg(z, name))
    with np.errstate(invalid="ignore", over="ignore"):
        return 1.13 * dz + (0 if name in ("none", "relu") else (8 * np.minimum(x, 200) + 16) * U) * np.abs(O.act(z, name))


def slope_bound(z, name):
    """Error of act'(z): s and q = 1 - s are each accurate to the argument's error, of which the
    second term has both; z s q p stays below 0.6."""
    from oracle import layer_oracle as O
    if name in ("none", "relu"):
        return 0.0
    x = np.abs(O.act_arg(z, name))
    q = 1.0 / (1.0 + np.exp(np.minimum(x, 200)))  # the smaller of s and 1 - s
    z = np.abs(O.f64(z))
    p = 2 * O.GELU_C * (1 + 3 * 0.044715 * z ** 2) if name == "gelu" else 1.0
    return 8 * U + (16 * np.minimum(x, 200) + 32) * U * q * (1 + z * p)


def check_checkpoint(codes, exps, block, z, dz):
    """A checkpoint written from values within dz of z: each value within half a step of z
    (plus dz), the step the oracle's wherever the block's largest value is not within dz of the
    border between two steps."""
    from oracle import layer_oracle as O
    codes, exps = codes.cpu().numpy(), exps.cpu().numpy()
    cols = z.shape[1]
    want_codes, want_exps = O.checkpoint_write(z, block)
    dz = np.broadcast_to(dz, z.shape)
    for b, (lo, hi) in enumerate(O.blocks_of(cols, block)):
        top, slack = np.abs(z[:, lo:hi]).max(1), dz[:, lo:hi].max(1)
        low = O.checkpoint_write(np.maximum(top - slack, 0)[:, None], block)[1][:, 0].astype(int)
        high = O.checkpoint_write((top + slack)[:, None], block)[1][:, 0].astype(int)
        assert np.all((exps[:, b] >= low) & (exps[:, b] <= high)), "another step than the values allow"
    step = O.checkpoint_steps(exps, cols, block)
    assert_near(O.checkpoint_read(codes, exps, block), z, step / 2 + dz, "checkpoint")
