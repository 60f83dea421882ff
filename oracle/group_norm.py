"""fp64 restatement of group norm with an activation, channels last, and its
gradients (the chain rule through the mean and the variance). x [N,S,C]."""
import numpy as np

from .linear_attention import _f64


def _act(z, act):
    """act(z) and its derivative."""
    if act == "none":
        return z, np.ones_like(z)
    p = 0.5 * (1 + np.tanh(0.5 * z))
    return z * p, p + z * p * (1 - p)


def forward(x, weight, bias, groups, eps, act):
    """(y, mean, rstd)"""
    x = _f64(x)
    N, S, C = x.shape
    xg = x.reshape(N, S, groups, C // groups)
    mean = xg.mean((1, 3))
    var = ((xg - mean[:, None, :, None]) ** 2).mean((1, 3))
    rstd = 1 / np.sqrt(var + eps)
    z = ((xg - mean[:, None, :, None]) * rstd[:, None, :, None]).reshape(N, S, C)
    if weight is not None:
        z = z * _f64(weight)
    if bias is not None:
        z = z + _f64(bias)
    return _act(z, act)[0], mean, rstd


def backward(dy, x, weight, bias, mean, rstd, groups, act):
    """(dx, dweight, dbias) with the given statistics."""
    x, dy, mean, rstd = (_f64(t) for t in (x, dy, mean, rstd))
    N, S, C = x.shape
    w = np.ones(C) if weight is None else _f64(weight)
    b = np.zeros(C) if bias is None else _f64(bias)
    xg = x.reshape(N, S, groups, C // groups)
    h = (xg - mean[:, None, :, None]) * rstd[:, None, :, None]
    d = dy * _act(h.reshape(N, S, C) * w + b, act)[1]
    u = (d * w).reshape(h.shape)
    dx = rstd[:, None, :, None] * (u - u.mean((1, 3), keepdims=True) - h * (u * h).mean((1, 3), keepdims=True))
    return dx.reshape(N, S, C), (d * h.reshape(N, S, C)).sum((0, 1)), d.sum((0, 1))
