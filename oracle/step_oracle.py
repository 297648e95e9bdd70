"""AdamW with its 8-bit states, the norms around a block and log probabilities of tokens, from
the formulas.  Plain NumPy; test infrastructure only.  AdamW is defined in IEEE fp32 operations
in order, so it is computed in float32 and compared in bits; the others in 64 bits."""

from __future__ import annotations

import functools

import numpy as np

from .layer_oracle import f64

# -- 8-bit states -------------------------------------------------------------------------


@functools.lru_cache
def fp8_values():
    """The 256 values of a float8 with 4 exponent bits (bias 7) and 3 mantissa bits, no infinities."""
    out = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        out[c] = np.nan if c & 127 == 127 else (-x if c & 128 else x)
    return out


def second_values(exp):
    """The 256 values of a second moment's codes under the block's byte exp."""
    if exp == 255:
        return np.full(256, np.nan)
    c = np.arange(256)
    x = (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 31.0 + max(int(exp), 32) - 127)
    x[0] = 0.0
    return x


def _nearest(x, values):
    """The index of the nearest of the ascending values, ties to the even index."""
    hi = np.searchsorted(values, x).clip(1, len(values) - 1)
    lo = hi - 1
    d = (x - values[lo]) - (values[hi] - x)
    return np.where((d > 0) | ((d == 0) & (hi % 2 == 0)), hi, lo)


def _mix(x):
    x = ((x ^ (x >> 32)) * 0x9E3779B97F4A7C15) % 2 ** 64
    x = ((x ^ (x >> 29)) * 0xB504F333F9DE6485) % 2 ** 64
    return x ^ (x >> 32)


def rounding_bits(seed, step, counter, places):
    """(first moment's, second moment's) 20 bits for random rounding of the elements at these places among
    the step's."""
    places = np.asarray(places, np.uint64)
    key = _mix((_mix((seed + step * 0x9E3779B97F4A7C15) % 2 ** 64) + counter) % 2 ** 64)
    low = lambda x: (x & 0xFFFFFFFF).astype(np.uint32)
    x = low(places) ^ np.uint32(key % 2 ** 32) ^ (low(places >> 32) * np.uint32(0x9E3779B9))
    x = (x ^ (x >> 16)) * np.uint32(0x9E3779B9)
    x = x ^ np.uint32(key >> 32)
    x = (x ^ (x >> 15)) * np.uint32(0xB504F335)
    x = x ^ (x >> 16)
    back = np.zeros_like(x)
    for i in range(20):
        back |= (x >> i & 1) << (19 - i)
    return x >> 12, back


def _random(x, values, bits):
    """The index of one of the two of the ascending values around x: the upper one if the part of their
    distance that x has over the lower one, in 2^-20 of it, and the bits come to 2^20."""
    hi = np.searchsorted(values, x, side="right").clip(1, len(values) - 1)
    lo = hi - 1
    part = np.rint((x - values[lo]) / (values[hi] - values[lo]) * 2.0 ** 20)
    return np.where(part + bits >= 2 ** 20, hi, lo)


def state_write(x, block, moment, bits=None):
    """(codes, exps) of values x, block by block from the definition: rounded to nearest, or at random by 20
    bits for each."""
    x = f64(x)
    codes, exps = np.zeros(x.size, np.uint8), np.zeros(-(-x.size // block), np.uint8)
    fp8 = fp8_values()[:127]
    for b in range(exps.size):
        v = x[b * block:(b + 1) * block]
        top = np.abs(v).max() if np.isfinite(v).all() else np.inf
        if moment == 1:
            s = -117
            while np.isfinite(top) and top > 448.0 * 2.0 ** s:
                s += 1
            if not np.isfinite(top):
                exps[b] = 255
                continue
            exps[b] = s + 127
            y = np.abs(v) * 2.0 ** -s
            code = _nearest(y, fp8) if bits is None else _random(y, fp8, bits[b * block:(b + 1) * block])
            codes[b * block:(b + 1) * block] = code | np.where(np.signbit(v), 128, 0)
        else:
            # the exponent of the largest value once it has four significant bits
            # to nearest from halfway between 15/8 and 2 on, at random from 15/8
            most = 2.0 - 2.0 ** -4 if bits is None else np.nextafter(2.0 - 2.0 ** -3, 2.0)
            if not np.isfinite(top) or top >= most * 2.0 ** 127:
                exps[b] = 255
                continue
            e = 32
            while top >= most * 2.0 ** (e - 127):
                e += 1
            exps[b] = e
            values = second_values(e)
            # between 0 and the code 1 (and at the bottom of the lowest exponent, which 0 takes): 1
            values[0] = values[1] / 1.125
            code = _nearest(v, values) if bits is None else _random(v, values, bits[b * block:(b + 1) * block])
            codes[b * block:(b + 1) * block] = np.where(v > 0, np.maximum(code, 1), 0)
    return codes, exps


def state_read(codes, exps, block, moment):
    out = np.zeros(codes.size)
    fp8 = fp8_values()
    for b, e in enumerate(exps):
        c = codes[b * block:(b + 1) * block]
        if moment == 1:
            step = np.inf if e == 255 else 0.0 if e == 0 else 2.0 ** (int(e) - 127)
            with np.errstate(invalid="ignore"):
                out[b * block:(b + 1) * block] = fp8[c] * step
        else:
            out[b * block:(b + 1) * block] = second_values(e)[c]
    return out


# -- AdamW ----------------------------------------------------------------------------------


def adamw(param, grad, m, v, *, lr, beta1, beta2, eps, step, weight_decay, grad_scale=None):
    """(param, m, v) after the step, all float32 arrays, one rounding an operation in the order that
    the header states."""
    f = np.float32
    b1, o1, b2, o2 = f(beta1), f(1.0 - beta1), f(beta2), f(1.0 - beta2)
    size, root = f(lr / (1.0 - beta1 ** step)), f(1.0 / np.sqrt(1.0 - beta2 ** step))
    with np.errstate(all="ignore"):
        g = grad.astype(f) if grad_scale is None else grad.astype(f) * f(grad_scale)
        m = b1 * m.astype(f) + o1 * g
        v = b2 * v.astype(f) + o2 * (g * g)
        u = m / (np.sqrt(v) * root + f(eps))
        param = param.astype(f) * f(1.0 - lr * weight_decay) - size * u
    assert param.dtype == m.dtype == v.dtype == f
    return param, m, v


def adamw64(param, grad, m, v, *, lr, beta1, beta2, eps, step, weight_decay):
    """The textbook form in 64 bits."""
    g = f64(grad)
    m, v = beta1 * f64(m) + (1 - beta1) * g, beta2 * f64(v) + (1 - beta2) * g * g
    mh, vh = m / (1 - beta1 ** step), v / (1 - beta2 ** step)
    return f64(param) - lr * (mh / (np.sqrt(vh) + eps) + weight_decay * f64(param)), m, v


# -- the norms around a block -----------------------------------------------------------------


def residual_norm(y, residual, weight, post_weight, gate, scale, eps, post):
    """(out, h, rstd, post_rstd); y, residual, gate and the weights may be None."""
    rp, h = None, 0.0
    if y is not None:
        u = f64(y)
        if post:
            rp = 1.0 / np.sqrt((u * u).mean(1) + eps)
            u = u * rp[:, None] * (1.0 if post_weight is None else f64(post_weight))
        h = scale * u * (1.0 if gate is None else f64(gate))
    if residual is not None:
        h = h + f64(residual)
    r = 1.0 / np.sqrt((h * h).mean(1) + eps)
    return h * r[:, None] * (1.0 if weight is None else f64(weight)), h, r, rp


def _rms_backward(g, x, r):
    return r[:, None] * (g - x * r[:, None] * (g * x * r[:, None]).mean(1, keepdims=True))


def residual_norm_backward(dout, dh, h, rstd, weight, y, post_rstd, post_weight, gate, scale):
    """dict of dresidual, dweight, dy, dgate (of each element), dpost_weight from the gradients of out
    and h (either may be None) and what the forward pass left."""
    gh, out = 0.0, {}
    if dout is not None:
        r = f64(rstd)
        gh = _rms_backward(f64(dout) * (1.0 if weight is None else f64(weight)), f64(h), r)
        out["dweight"] = (f64(dout) * f64(h) * r[:, None]).sum(0)
    if dh is not None:
        gh = gh + f64(dh)
    out["dresidual"] = gh
    du = scale * gh
    g = 1.0 if gate is None else f64(gate)
    if y is not None:
        y = f64(y)
        yh = y if post_rstd is None else y * f64(post_rstd)[:, None]
        u = yh if post_rstd is None or post_weight is None else yh * f64(post_weight)
        out["dgate"] = du * u
        if post_rstd is not None:
            out["dpost_weight"] = (du * g * yh).sum(0)
            dn = du * g * (1.0 if post_weight is None else f64(post_weight))
            out["dy"] = _rms_backward(dn, y, f64(post_rstd))
            return out
    out["dy"] = du * g
    return out


# -- log probabilities of tokens ---------------------------------------------------------------


def token_logprobs(x, targets, scale, top):
    """dict of stats (largest logit, sum of exp(scale (x - it))), logprob, entropy, top_ids and
    top_logprobs.  Rows of minus infinities only have the sum 0, log probability minus infinity and
    entropy 0; rows with a NaN or plus infinity have NaN in every number and the ids -1."""
    x = f64(x)
    rows, vocab = x.shape
    big = np.where(np.isnan(x).any(1), np.nan, x.max(1))
    lost, empty = ~(big < np.inf), big == -np.inf
    m = np.where(lost | empty, 0.0, big)
    with np.errstate(all="ignore"):
        d = x - m[:, None]
        e = np.exp(scale * d)
        s = e.sum(1)
        ls = np.log(s)
        h = np.where(empty, 0.0, ls - scale * np.where(e > 0, e * d, 0.0).sum(1) / s)
        own = x[np.arange(rows), np.clip(targets, 0, vocab - 1)]
        lp = np.where(empty, -np.inf, scale * (own - m) - ls)
    lp[lost] = h[lost] = np.nan
    lp = np.where(targets < 0, 0.0, np.where(targets >= vocab, np.nan, lp))
    ids, tops = np.full((rows, top), -1), np.full((rows, top), -np.inf)
    k = min(top, vocab)
    for r in range(rows):
        order = np.argsort(-x[r], kind="stable")[:k]
        if lost[r]:
            tops[r] = np.nan
        else:
            ids[r, :k] = order
            tops[r, :k] = -np.inf if empty[r] else scale * (x[r, order] - m[r]) - ls[r]
    stats = np.stack([np.where(lost, np.nan, big), np.where(lost, np.nan, s)], 1)
    return dict(stats=stats, logprob=lp, entropy=h, top_ids=ids, top_logprobs=tops, lost=lost, empty=empty)


def token_logprobs_backward(x, targets, scale, dlogprob, dentropy):
    """The gradient of sum(dlogprob logprob + dentropy entropy) with respect to x."""
    o = token_logprobs(x, targets, scale, 0)
    x = f64(x)
    rows, vocab = x.shape
    with np.errstate(all="ignore"):
        z = scale * (x - o["stats"][:, :1]) - np.log(o["stats"][:, 1:])
        p = np.exp(z)
    lp = np.zeros(rows) if dlogprob is None else np.where(targets < 0, 0.0, f64(dlogprob))
    dz = -lp[:, None] * p
    good = (targets >= 0) & (targets < vocab)
    dz[np.arange(rows)[good], targets[good]] += lp[good]
    if dentropy is not None:
        with np.errstate(all="ignore"):
            dz = dz - f64(dentropy)[:, None] * np.where(p > 0, p * (z + o["entropy"][:, None]), 0.0)
    dz = scale * dz
    dz[o["empty"]] = 0.0
    if dlogprob is not None:
        dz[targets >= vocab] = np.nan
    dz[o["lost"]] = np.nan
    if dentropy is None:
        dz[(targets < 0) | (dlogprob is None)] = 0.0
    return dz
