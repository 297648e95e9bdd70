"""The rms bound of the product tests refuses what the worst case per element lets through: sums
that lose bits between the parts of a split contraction.  NumPy on the CPU; the losses are planted
here."""
import numpy as np
import pytest

from precision_util import U, product_rms_bound, rms


def bf16(x):
    """x in fp32, rounded to bf16 (ties to even), as float32."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    return (((u + 0x7FFF + (u >> 16 & 1)) >> 16 << 16).astype(np.uint32)).view(np.float32)


def operands(m, n, k, seed):
    r = np.random.default_rng(seed)
    return bf16(r.normal(size=(m, k))), bf16(r.normal(size=(k, n)) * k ** -0.5)


def split_product(a, b, splits, keep):
    """fp32 sums in order within each part, `keep` what happens to a part's sum, fp32 join."""
    out = np.zeros((a.shape[0], b.shape[1]), np.float32)
    for part in np.array_split(np.arange(a.shape[1]), splits):
        s = np.zeros_like(out)
        for i in part:
            s += a[:, i:i + 1] * b[i]
        out += keep(s)
    return out


@pytest.mark.parametrize("k,splits", [(520, 2), (2048, 8), (8192, 16)])
def test_bound_separates(k, splits):
    a, b = operands(24, 40, k, k)
    want = a.astype(np.float64) @ b.astype(np.float64)
    bound = product_rms_bound(a, b, want)
    worst = 2 * (k / 8 + 80) * U * (np.abs(a).astype(np.float64) @ np.abs(b))
    assert rms(split_product(a, b, splits, lambda s: s) - want) <= bound
    lossy = split_product(a, b, splits, bf16)
    assert rms(lossy - want) > 2 * bound
    if k == 8192:  # and the worst case of an element does not see it
        assert np.all(np.abs(lossy - want) <= worst)
    # a running sum that is cut to bf16 from part to part
    run = np.zeros_like(lossy)
    for part in np.array_split(np.arange(k), splits):
        run = bf16(run + a[:, part] @ b[part])
    assert rms(run - want) > 2 * bound
