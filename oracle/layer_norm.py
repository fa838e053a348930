"""fp64 oracle of layer norm over the last dimension (test infrastructure only).

h = x + residual rounded to the I/O type (the tensor that is normalised), and with
mu and the biased var of a row, rstd = 1 / sqrt(var + eps), x_hat = (h - mu) rstd:
    y = gamma x_hat + beta
    dx = rstd (g - mean(g) - x_hat mean(g x_hat)) + dh,  g = gamma dy
    dgamma = sum over rows of dy x_hat,  dbeta = sum over rows of dy
dh is the gradient that reaches h past the norm. Library primitives used as steps:
numpy mean, sum, sqrt.
"""

from __future__ import annotations

import numpy as np

from .numerics import round_to_dtype


def layer_norm_fwd(x, gamma, beta, eps: float, residual=None, dtype: str = "f64"):
    """(y, mean, rstd, h) for x [M, N]; gamma, beta None mean 1 and 0; h is rounded to `dtype`."""
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = round_to_dtype(h + np.asarray(residual, np.float64), dtype)
    mu = h.mean(axis=1)
    rstd = 1.0 / np.sqrt(((h - mu[:, None]) ** 2).mean(axis=1) + eps)
    y = (h - mu[:, None]) * rstd[:, None]
    if gamma is not None:
        y = y * np.asarray(gamma, np.float64)
    if beta is not None:
        y = y + np.asarray(beta, np.float64)
    return y, mu, rstd, h


def layer_norm_bwd(dy, h, mean, rstd, gamma, dh=None):
    """(dx, dgamma, dbeta) from the forward's mean and rstd."""
    dy = np.asarray(dy, np.float64)
    xhat = (np.asarray(h, np.float64) - np.asarray(mean, np.float64)[:, None]) * np.asarray(rstd, np.float64)[:, None]
    g = dy if gamma is None else dy * np.asarray(gamma, np.float64)
    dx = np.asarray(rstd, np.float64)[:, None] * (
        g - g.mean(axis=1)[:, None] - xhat * (g * xhat).mean(axis=1)[:, None])
    if dh is not None:
        dx = dx + np.asarray(dh, np.float64)
    return dx, (dy * xhat).sum(axis=0), dy.sum(axis=0)
