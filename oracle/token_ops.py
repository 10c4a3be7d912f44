"""Token-wise operators in 64 bits (numpy), the reference the tests compare with: the norms,
their gradients, rows quantised to 8-bit integers, and the linear layer over them.  Inputs are
arrays of any float type, widened to float64; nothing here is shared with the CUDA path."""
from __future__ import annotations

import numpy as np

TINIEST = 2.0 ** -100  # smallest magnitude that a row's scale is taken from


def moments(x, eps):
    x = np.asarray(x, np.float64)
    mean = x.mean(axis=1)
    var = ((x - mean[:, None]) ** 2).mean(axis=1)
    return mean, 1.0 / np.sqrt(var + eps)


def layer_norm(x, gamma=None, beta=None, eps=1e-5):
    """(y, mean, rstd)."""
    x = np.asarray(x, np.float64)
    mean, rstd = moments(x, eps)
    y = (x - mean[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * np.asarray(gamma, np.float64)
    if beta is not None:
        y = y + np.asarray(beta, np.float64)
    return y, mean, rstd


def layer_norm_backward(dy, x, gamma, mean, rstd):
    """(dx, dgamma, dbeta)."""
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    mean, rstd = np.asarray(mean, np.float64)[:, None], np.asarray(rstd, np.float64)[:, None]
    h = (x - mean) * rstd
    g = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    c = x.shape[1]
    dx = rstd * (g - g.sum(1, keepdims=True) / c - h * ((g * h).sum(1, keepdims=True) / c))
    return dx, (dy * h).sum(0), dy.sum(0)


def row_scales(v):
    v = np.asarray(v, np.float64)
    return np.maximum(np.abs(v).max(axis=1), TINIEST) / 127.0


def quantize_rows_f32(x):
    """The definition in its own arithmetic (one float32 division, product and rounding per
    step), which the kernels follow bit for bit: (q, scale)."""
    x = np.asarray(x, np.float32)
    most = np.maximum(np.abs(x).max(axis=1), np.float32(TINIEST))
    inv = np.float32(127.0) / most
    return np.rint(x * inv[:, None]).astype(np.int8), most / np.float32(127.0)


def activate(z, activation):
    if activation == "silu":
        with np.errstate(over="ignore"):
            return z / (1.0 + np.exp(-z))
    return np.maximum(z, 0.0) if activation == "relu" else z


def linear_int8(a, w, a_scale, w_scale, bias=None, activation="identity", residual=None):
    """(y, z, total): the layer, its value before the activation, and sum_k |a w| for error bounds.
    Integer sums stay below 2**53, so they are exact."""
    a, w = np.asarray(a, np.float64), np.asarray(w, np.float64)
    z = (a @ w.T) * np.asarray(a_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)[None, :]
    if bias is not None:
        z = z + np.asarray(bias, np.float64)
    y = activate(z, activation)
    if residual is not None:
        y = y + np.asarray(residual, np.float64)
    return y, z, np.abs(a) @ np.abs(w).T


def rms_norm(x, gamma=None, eps=1e-6):
    """(y, rstd)."""
    x = np.asarray(x, np.float64)
    rstd = 1.0 / np.sqrt((x ** 2).mean(axis=1) + eps)
    y = x * rstd[:, None]
    return (y if gamma is None else y * np.asarray(gamma, np.float64)), rstd


def rms_norm_backward(dy, x, gamma, rstd, residual=None):
    """(dx, dgamma)."""
    dy, x, rstd = np.asarray(dy, np.float64), np.asarray(x, np.float64), np.asarray(rstd, np.float64)[:, None]
    h = x * rstd
    g = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    dx = rstd * (g - h * (g * h).mean(axis=1, keepdims=True))
    return (dx if residual is None else dx + np.asarray(residual, np.float64)), (dy * h).sum(0)


def adamw(p, g, m, v, step, lr, beta1, beta2, eps, decay, grad_scale=1.0):
    """(p, m, v) after the step."""
    p, g, m, v = (np.asarray(t, np.float64) for t in (p, g, m, v))
    g = g * grad_scale
    m, v = beta1 * m + (1 - beta1) * g, beta2 * v + (1 - beta2) * g * g
    u = m / (1 - beta1 ** step) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p * (1 - lr * decay) - lr * u, m, v


def dither(n, step):
    """The two numbers in [0, 1) of each place of a tensor in a step with 8-bit moments."""
    with np.errstate(over="ignore"):
        z = np.arange(n, dtype=np.uint32) + np.uint32(step * 0x9E3779B9 % 2 ** 32)
        z = (z ^ (z >> np.uint32(16))) * np.uint32(0x85EBCA6B)
        z = (z ^ (z >> np.uint32(13))) * np.uint32(0xC2B2AE35)
        z = z ^ (z >> np.uint32(16))
    return (z >> np.uint32(16)) / 65536.0, (z & np.uint32(0xFFFF)) / 65536.0


def e4m3_distance(x):
    """Between the 8-bit floats around magnitudes x."""
    with np.errstate(divide="ignore"):
        return 2.0 ** (np.maximum(np.floor(np.log2(np.maximum(x, 2.0 ** -60))), -6) - 3)


def linear_adapters(x, index, a, b, scale=None, base=None):
    """(y, hidden, total): the adapters' output, their hidden rows, and sum |terms| of y for error bounds."""
    x, a, b = (np.asarray(t, np.float64) for t in (x, a, b))
    hidden, y = np.zeros((len(x), a.shape[1])), np.zeros((len(x), b.shape[1]))
    total = np.zeros_like(y)
    for i, g in enumerate(index):
        if 0 <= g < len(a):
            s = 1.0 if scale is None else float(scale[g])
            hidden[i] = a[g] @ x[i]
            y[i] = s * (b[g] @ hidden[i])
            total[i] = abs(s) * (np.abs(b[g]) @ (np.abs(a[g]) @ np.abs(x[i])))
    if base is not None:
        y, total = y + np.asarray(base, np.float64), total + np.abs(np.asarray(base, np.float64))
    return y, hidden, total


def linear_adapters_backward(dy, x, index, a, b, scale, hidden, base=None):
    """((dx, da, db), (sum |terms| of each))."""
    dy, x, a, b, hidden = (np.asarray(t, np.float64) for t in (dy, x, a, b, hidden))
    out, terms = (np.zeros_like(x), np.zeros_like(a), np.zeros_like(b)), (np.zeros_like(x), np.zeros_like(a), np.zeros_like(b))
    for i, g in enumerate(index):
        if 0 <= g < len(a):
            s = 1.0 if scale is None else float(scale[g])
            for to, f in ((out, lambda v: v), (terms, np.abs)):
                dh = f(b[g]).T @ f(dy[i])
                to[0][i] = f(np.float64(s)) * (f(a[g]).T @ dh)
                to[1][g] += f(np.float64(s)) * np.outer(dh, f(x[i]))
                to[2][g] += f(np.float64(s)) * np.outer(f(dy[i]), f(hidden[i]))
    if base is not None:
        out[0][:] += np.asarray(base, np.float64)
        terms[0][:] += np.abs(np.asarray(base, np.float64))
    return out, terms
