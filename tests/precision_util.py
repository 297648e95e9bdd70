"""A root-mean-square bound of fp32 products, far below the worst case of each element."""
import numpy as np

U = 2.0 ** -24


def rms(x):
    return float(np.sqrt(np.mean(np.square(np.asarray(x, np.float64)))))


def product_rms_bound(a, b, want):
    """Bound of rms(error) over a whole fp32 product a @ b with k = a.shape[1], for operands whose
    elements are independent and centred.  A partial sum of any of the products has then an rms of at
    most sqrt(k) rms(a) rms(b); an element passes through k / 8 additions of the matrix cores, 16
    inside one instruction and 64 of partial sums, each of which is off by at most 2 U of the partial
    sum it forms; and the rms of a sum of errors is at most the sum of their rms.  A tenth is left
    for the operands being a sample, U rms(want) for the result's own rounding.  The worst case of a
    single element is larger by rms's factor sqrt(k)."""
    k = a.shape[1]
    return 1.1 * 2 * (k / 8 + 80) * U * np.sqrt(k) * rms(a) * rms(b) + U * rms(want)
