"""The layer operators in 64 bits: layer norm, activations, 8-bit activation checkpoints and
the products of a linear layer.  Plain NumPy, straight from the formulas; test
infrastructure only."""

from __future__ import annotations

import numpy as np

ACTS = ("none", "relu", "gelu", "silu")
GELU_C = np.sqrt(2.0 / np.pi)


def f64(x):
    return np.asarray(x, np.float64)


def act(z, name):
    z = f64(z)
    if name == "relu":
        return np.where(z < 0, 0.0, z)
    if name in ("gelu", "silu"):
        # the quotient keeps its relative accuracy where z is far below 0; 1 + tanh would cancel there
        with np.errstate(over="ignore"):
            return z / (1.0 + np.exp(-act_arg(z, name)))
    return z.copy()


def act_slope(z, name):
    z = f64(z)
    if name == "relu":
        return np.where(z > 0, 1.0, np.where(z <= 0, 0.0, z))
    if name == "gelu":
        u = GELU_C * (z + 0.044715 * z ** 3)
        return 0.5 * (1.0 + np.tanh(u)) + 0.5 * z / np.cosh(np.clip(u, -300, 300)) ** 2 * GELU_C * (
            1.0 + 3 * 0.044715 * z ** 2)
    if name == "silu":
        s = 1.0 / (1.0 + np.exp(-z))
        return s * (1.0 + z * (1.0 - s))
    return np.ones_like(z)


def act_arg(z, name):
    """The argument x of the sigmoid in act(z) = z sigmoid(x), for error bounds."""
    z = f64(z)
    return 2 * GELU_C * (z + 0.044715 * z ** 3) if name == "gelu" else z if name == "silu" else np.zeros_like(z)


# -- 8-bit checkpoints ------------------------------------------------------------------

def blocks_of(cols, block):
    return [(lo, min(lo + block, cols)) for lo in range(0, cols, block)]


def checkpoint_write(x, block):
    """codes int8 and exps uint8 of a float matrix, block by block, from the definition."""
    x = f64(x)
    rows, cols = x.shape
    codes = np.zeros((rows, cols), np.int8)
    spans = blocks_of(cols, block)
    exps = np.zeros((rows, len(spans)), np.uint8)
    for b, (lo, hi) in enumerate(spans):
        v = x[:, lo:hi]
        fine = np.isfinite(v).all(1)
        top = np.where(fine, np.abs(np.where(np.isfinite(v), v, 0.0)).max(1), 0.0)
        s = np.full(rows, -126)
        while True:
            small = top >= 127.5 * 2.0 ** s.astype(np.float64)
            if not small.any():
                break
            s += small
        exps[:, b] = np.where(fine, s + 127, 255)
        q = np.rint(np.where(np.isfinite(v), v, 0.0) * 2.0 ** (-s[:, None].astype(np.float64)))
        codes[:, lo:hi] = np.where(fine[:, None], q, 0)
    return codes, exps


def checkpoint_steps(exps, cols, block):
    """One step per element: 2^(byte - 127), 0 for the byte 0 and inf for 255."""
    e = np.repeat(np.asarray(exps).astype(np.int64), block, axis=1)[:, :cols]
    return np.where(e == 0, 0.0, np.where(e == 255, np.inf, 2.0 ** (e - 127.0)))


def checkpoint_read(codes, exps, block):
    with np.errstate(invalid="ignore"):
        return f64(codes) * checkpoint_steps(exps, codes.shape[1], block)


# -- layer norm -----------------------------------------------------------------------

def layer_norm(x, w, b, eps):
    x = f64(x)
    mean = x.mean(1)
    rstd = 1.0 / np.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    y = (x - mean[:, None]) * rstd[:, None]
    return (y * (1.0 if w is None else f64(w)) + (0.0 if b is None else f64(b))), mean, rstd


def layer_norm_backward(dy, x, w, mean, rstd, residual=None):
    dy, mean, rstd = f64(dy), f64(mean)[:, None], f64(rstd)[:, None]
    xh = (f64(x) - mean) * rstd
    g = dy * (1.0 if w is None else f64(w))
    dx = rstd * (g - g.mean(1, keepdims=True) - xh * (g * xh).mean(1, keepdims=True))
    if residual is not None:
        dx = dx + f64(residual)
    return dx, (dy * xh).sum(0), dy.sum(0)


# -- products -------------------------------------------------------------------------

def linear(x, w, bias, act_name, residual):
    """(out, z)"""
    z = f64(x) @ f64(w).T + (0.0 if bias is None else f64(bias))
    return act(z, act_name) + (0.0 if residual is None else f64(residual)), z


def linear_input_grad(dy, w, z, act_name, residual):
    dx = f64(dy) @ f64(w)
    if act_name != "none":
        dx = dx * act_slope(z, act_name)
    return dx + (0.0 if residual is None else f64(residual))


def linear_weight_grad(dy, z, act_name):
    return f64(dy).T @ act(z, act_name), f64(dy).sum(0)
