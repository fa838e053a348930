"""fp64 oracle of the linear layer with its epilogue (test infrastructure only).

    z = x w + b,  y = f(z) + residual
    dz = dy f'(z), rounded to the I/O type as the products take it;  dx = dz w^T,  dw = x^T dz,
    db = sum over rows of the unrounded dz
f is the identity (None), SiLU, GELU (exact) or HardSwish; f' is act_grad's. Library primitives used as steps:
numpy matmul and sum, scipy.special.ndtr.
"""

from __future__ import annotations

import numpy as np
from scipy.special import ndtr

from .activations import act_grad
from .numerics import round_to_dtype
from .swiglu import sigmoid


def act_fwd(z, act):
    z = np.asarray(z, np.float64)
    if act is None:
        return z
    if act == "silu":
        return z * sigmoid(z)
    if act == "gelu":
        return z * ndtr(z)
    if act == "hardswish":
        return z * np.minimum(np.maximum(z + 3.0, 0.0), 6.0) / 6.0
    raise ValueError(act)


def linear_fwd(x, w, b=None, act=None, residual=None):
    """(y, z)"""
    z = np.asarray(x, np.float64) @ np.asarray(w, np.float64)
    if b is not None:
        z = z + np.asarray(b, np.float64)
    y = act_fwd(z, act)
    return (y if residual is None else y + np.asarray(residual, np.float64)), z


def linear_bwd(dy, x, w, z=None, act=None, dtype: str = "f64"):
    """(dx, dw, db, dz): dz rounded to `dtype`, db of the unrounded one."""
    dz = np.asarray(dy, np.float64)
    if act is not None:
        dz = act_grad(dz, z, act)
    db = dz.sum(axis=0)
    dz = round_to_dtype(dz, dtype)
    return dz @ np.asarray(w, np.float64).T, np.asarray(x, np.float64).T @ dz, db, dz
