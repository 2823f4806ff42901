"""Layer norm, forward and backward, in float64 (oracle side).

Test infrastructure only (see ``oracle/__init__.py``).

    mean = sum x / n,  rstd = 1 / sqrt(sum (x - mean)^2 / n + eps)
    y    = (x - mean) rstd w + b
and for an output gradient dy, with xh = (x - mean) rstd and g = dy w,
    dx = rstd (g - sum(g) / n - xh sum(g xh) / n)
    dw = sum_rows dy xh,  db = sum_rows dy.
mean and rstd are those of the exact x; the backward pass may be given another
x (the one 8 bits hold), which enters xh alone.
"""
import numpy as np


def forward(x, w=None, b=None, eps=1e-5):
    x = np.asarray(x, np.float64)
    n = x.shape[1]
    mean = x.sum(1) / n
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).sum(1) / n + eps)
    y = d * rstd[:, None]
    if w is not None:
        y = y * np.asarray(w, np.float64)
    if b is not None:
        y = y + np.asarray(b, np.float64)
    return y, mean, rstd


def backward(dy, x, mean, rstd, w=None):
    dy, x = np.asarray(dy, np.float64), np.asarray(x, np.float64)
    mean, rstd = np.asarray(mean, np.float64)[:, None], np.asarray(rstd, np.float64)[:, None]
    n = x.shape[1]
    xh = (x - mean) * rstd
    g = dy if w is None else dy * np.asarray(w, np.float64)
    c1 = (g * xh).sum(1, keepdims=True) / n
    c2 = g.sum(1, keepdims=True) / n
    return rstd * (g - c2 - xh * c1), (dy * xh).sum(0), dy.sum(0)
