"""fp64 oracle of the operators on rows of logits (test infrastructure only):
log probabilities of given tokens and distillation from a teacher's top logits.

With d_j = (z_j - max z) / tau and s = sum exp(d_j) of a row: ln p_j = d_j - ln s.
A logit of -inf has p = 0 and ln p = -inf; a row of nothing else has max -inf, s = 0,
entropy 0 and no gradient. Library primitives used as steps: numpy max, exp, log, sum,
lexsort.
"""

from __future__ import annotations

import numpy as np


def row_softmax(z, temperature: float):
    """(max, s, ln p, p) of rows z [T, V]."""
    z = np.asarray(z, np.float64)
    m = z.max(axis=1)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        d = (z - np.where(np.isneginf(m), 0.0, m)[:, None]) / temperature
        s = np.exp(d).sum(axis=1)
        lp = np.where(np.isneginf(z) & ~np.isnan(s)[:, None], -np.inf, d - np.log(s)[:, None])
    return m, s, lp, np.exp(lp)


def token_logprobs_fwd(z, targets, top_k: int, temperature: float, ignore_index: int = -100) -> dict:
    z = np.asarray(z, np.float64)
    T, V = z.shape
    m, s, lp, p = row_softmax(z, temperature)
    with np.errstate(invalid="ignore"):
        entropy = -np.where(p == 0, 0.0, p * lp).sum(axis=1)
    out = dict(stats=np.stack([m, s], axis=1), entropy=entropy)
    if targets is not None:
        logp = np.full(T, np.nan)
        for r, t in enumerate(np.asarray(targets)):
            if t == ignore_index:
                logp[r] = 0.0
            elif 0 <= t < V:
                logp[r] = lp[r, t]
        out["logp"] = logp
    if top_k:
        order = np.where(np.isnan(z), -np.inf, z)
        idx = np.stack([np.lexsort((np.arange(V), -order[r]))[:top_k] for r in range(T)])
        out["top_idx"] = idx
        out["top_logp"] = np.take_along_axis(np.where(np.isnan(z) & ~np.isnan(s)[:, None], -np.inf, lp), idx, axis=1)
    return out


def token_logprobs_bwd(z, targets, temperature: float, dlogp=None, dentropy=None, ignore_index: int = -100):
    """The gradient of sum(dlogp * logp) + sum(dentropy * entropy)."""
    z = np.asarray(z, np.float64)
    T, V = z.shape
    _, s, lp, p = row_softmax(z, temperature)
    g = np.zeros((T, V))
    for r in range(T):
        if s[r] == 0:
            continue
        if targets is not None and targets[r] != ignore_index:
            g[r] -= dlogp[r] * p[r]
            g[r, targets[r]] += dlogp[r]
        if dentropy is not None:
            l0 = np.where(p[r] == 0, 0.0, lp[r])
            g[r] -= dentropy[r] * p[r] * (l0 - (p[r] * l0).sum())
    return g / temperature


def teacher_probs(ids, teacher, V: int, temperature: float):
    """(q, ln q) of the entries; q = 0 for absent ones and for rows without entries."""
    ids, t = np.asarray(ids), np.asarray(teacher, np.float64)
    t = np.where((ids >= 0) & (ids < V), t, -np.inf) / temperature
    m = t.max(axis=1, keepdims=True)
    with np.errstate(divide="ignore", invalid="ignore"):
        d = t - np.where(np.isneginf(m), 0.0, m)
        s = np.exp(d).sum(axis=1, keepdims=True)
        return np.where(s > 0, np.exp(d) / s, 0.0), np.where(s > 0, d - np.log(s), -np.inf)


def distill_fwd(z, ids, teacher, temperature: float):
    """(loss [T], max, s): loss = sum over the entries of q (ln q - ln p)."""
    z, ids = np.asarray(z, np.float64), np.asarray(ids)
    m, s, lp, _ = row_softmax(z, temperature)
    q, lq = teacher_probs(ids, teacher, z.shape[1], temperature)
    lpk = np.take_along_axis(lp, np.clip(ids, 0, z.shape[1] - 1), axis=1)
    with np.errstate(invalid="ignore"):
        loss = np.where(q > 0, q * (lq - lpk), 0.0).sum(axis=1)
    return loss, m, s


def distill_bwd(weight, z, ids, teacher, temperature: float):
    """The gradient of sum(weight * loss): (weight / tau) (Q p - q)."""
    z, ids = np.asarray(z, np.float64), np.asarray(ids)
    T, V = z.shape
    p = row_softmax(z, temperature)[3]
    q, _ = teacher_probs(ids, teacher, V, temperature)
    g = np.zeros((T, V))
    for r in range(T):
        if weight[r] == 0 or not (q[r] > 0).any():
            continue
        g[r] = p[r]
        for i, x in zip(ids[r], q[r]):
            if x > 0:
                g[r, i] -= x
        g[r] *= weight[r] / temperature
    return g
