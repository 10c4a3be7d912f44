"""Token-wise operators in 64 bits (numpy), the reference the tests compare with: layer norm,
its gradient, rows quantised to 8-bit integers, and the linear layer over them.  Inputs are
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
