"""fp64 oracle of the norms between two blocks (test infrastructure only).

    rstd(t) = 1 / sqrt(mean(t^2) + eps)
    v = u rstd(u) gamma_post (v = u without post);  h = alpha residual + gate v, rounded to the I/O type
    y = h rstd(h) gamma_pre (with pre)
gate [G, N] serves M / G rows with each of its rows. Backward, written out by the chain rule, from dy, dh, u, h
and the two rstd. Library primitives used as steps: numpy mean, sum, sqrt, repeat.
"""

from __future__ import annotations

import numpy as np

from .numerics import round_to_dtype


def _a(t):
    return None if t is None else np.asarray(t, np.float64)


def _rows(gate, M):
    return 1.0 if gate is None else np.repeat(gate, M // gate.shape[0], axis=0)


def block_norm_fwd(u, residual=None, gamma_post=None, gamma_pre=None, gate=None, alpha=1.0, eps=1e-6, post=True,
                   pre=True, dtype: str = "f64"):
    """(h, y, rstd_u, rstd_h); y is None without pre, the rstd of a norm that is not there 0."""
    u, residual, gamma_post, gamma_pre, gate = (_a(t) for t in (u, residual, gamma_post, gamma_pre, gate))
    M, N = u.shape
    v, ru = u, np.zeros(M)
    if post:
        ru = 1.0 / np.sqrt((u * u).mean(axis=1) + eps)
        v = u * ru[:, None] * (1.0 if gamma_post is None else gamma_post)
    h = v * _rows(gate, M)
    if residual is not None:
        h = h + alpha * residual
    h = round_to_dtype(h, dtype)
    if not pre:
        return h, None, ru, np.zeros(M)
    rh = 1.0 / np.sqrt((h * h).mean(axis=1) + eps)
    return h, h * rh[:, None] * (1.0 if gamma_pre is None else gamma_pre), ru, rh


def block_norm_bwd(dy, dh, u, h, rstd_u, rstd_h, gamma_post=None, gamma_pre=None, gate=None, alpha=1.0, post=True,
                   pre=True):
    """A dict of du, dresidual, dgamma_post, dgamma_pre and dgate (None where there is none)."""
    dy, dh, u, h, gamma_post, gamma_pre, gate = (_a(t) for t in (dy, dh, u, h, gamma_post, gamma_pre, gate))
    M, N = u.shape
    d = np.zeros((M, N)) if dh is None else dh
    out = dict(dgamma_post=None, dgamma_pre=None, dgate=None)
    if pre:
        hh = h * _a(rstd_h)[:, None]
        a = dy * (1.0 if gamma_pre is None else gamma_pre)
        d = d + _a(rstd_h)[:, None] * (a - hh * (a * hh).mean(axis=1, keepdims=True))
        out["dgamma_pre"] = (dy * hh).sum(axis=0)
    out["dresidual"] = alpha * d
    uh = u * _a(rstd_u)[:, None] if post else u
    gp = 1.0 if gamma_post is None else gamma_post
    dv = d * _rows(gate, M)
    if gate is not None:
        out["dgate"] = (d * uh * gp).reshape(gate.shape[0], -1, N).sum(axis=1)
    if not post:
        out["du"] = dv
        return out
    out["dgamma_post"] = (dv * uh).sum(axis=0)
    q = dv * gp
    out["du"] = _a(rstd_u)[:, None] * (q - uh * (q * uh).mean(axis=1, keepdims=True))
    return out
