"""Inputs and error bounds shared by the tests of the linear layer and of the norms between blocks.

Element bounds are those of _row_ops.check: one rounding of the output, and an fp32 part from the arithmetic.

Products: bf16 or fp16 factors are exact in fp32, and every one of the K additions may be truncated, 2^-23 of the sum of
the magnitudes: (K + 8) 2^-23 |x| |w|. In the norm the rounding errors are far smaller: U + 2^-16 of a rounded
output, twice U where a rounded dz enters it.
Activations (relative to the value): 2^-20 and the exponent's rounding, |z| 2^-22 for SiLU; for GELU the fit's 1.3e-6 <
2^-19 and z^2 2^-22. Their gradients, absolute: 2^-19 (1 + |z|), as the values themselves are below 1.2.
Sums of the norms: 64 terms in sequence in a thread, a tree, or 128 rows of a chunk and 64 chunks: (128 + 64 + 10) 2^-24
< 2^-16 of the sum of the magnitudes.
"""

import numpy as np
import torch

import oracle

from ._row_ops import NAME, SUM, U, check, f64

ACTS = (None, "silu", "gelu", "hardswish")
NORM_SUM = 2.0 ** -16


def rel(got, ref):
    g = f64(got).reshape(np.shape(ref))
    n = np.linalg.norm(ref)
    return float(np.linalg.norm(g - ref) / n) if n else float(np.linalg.norm(g))


def linear_inputs(M, K, N, dtype, seed=3):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return dict(x=rn(M, K).to(dtype), w=(rn(K, N) * (1.5 / K ** 0.5)).to(dtype), b=(0.5 * rn(N)).to(dtype),
                residual=rn(M, N).to(dtype), dy=rn(M, N).to(dtype), z=(1.5 * rn(M, N)).to(dtype))


def products(a, b):
    """a b in fp64 and the bound of its fp32 sum."""
    return a @ b, (a.shape[1] + 8) * 2.0 ** -23 * (np.abs(a) @ np.abs(b))


def act_part(z, y, act):
    if act is None:
        return 0.0
    if act == "hardswish":
        return 2.0 ** -20 * np.abs(y)
    return np.abs(y) * (2.0 ** -19 + (np.abs(z) if act == "silu" else z * z) * 2.0 ** -22) + 1e-36


def check_linear_fwd(t, out, dtype, act, b=None, residual=None):
    x, w = f64(t["x"]), f64(t["w"])
    x = x.reshape(-1, x.shape[-1])
    y, z = oracle.linear_fwd(x, w, None if b is None else f64(b), act,
                             None if residual is None else f64(residual).reshape(x.shape[0], -1))
    part = products(x, w)[1] + 2.0 ** -23 * np.abs(z)
    if "z" in out:
        check("z", out["z"], z, dtype, part)
    f = y if residual is None else y - f64(residual).reshape(y.shape)
    check("y", out["y"], y, dtype, 1.2 * part + act_part(z, f, act) + 2.0 ** -23 * (np.abs(f) + np.abs(y)))
    assert y.size < 64 or rel(out["y"], y) <= U[dtype] + 2.0 ** -16


def check_linear_bwd(t, out, dtype, act, old=None, db_dtype=None):
    """old: dw and db that the call added to."""
    dy, x, w = (f64(t[k]).reshape(-1, t[k].shape[-1]) for k in ("dy", "x", "w"))
    z = f64(t["z"]).reshape(dy.shape)
    dx, dw, db, dz = oracle.linear_bwd(dy, x, w, z, act)
    # dz: a rounding, and the activation's own error
    grad = np.zeros_like(dy) if act is None else np.abs(dy) * 2.0 ** -19 * (1 + np.abs(z))
    edz = grad + (0.0 if act is None else U[dtype] * np.abs(dz) + 2.0 ** -25)
    near = U[dtype] * (1 if act is None else 2) + 2.0 ** -16
    for name, ref, part in (("dx", dx, products(dz, w.T)[1] + edz @ np.abs(w).T),
                            ("dw", dw, products(x.T, dz)[1] + np.abs(x).T @ edz)):
        if name in out:
            if old is not None and name in old:
                ref = ref + old[name]
                part = part + 2.0 ** -23 * np.abs(ref)
            check(name, out[name], ref, dtype, part)
            assert ref.size < 64 or rel(out[name], ref) <= near, name
    if "db" in out:
        if old is not None:
            db = db + old["db"]
        check("db", out["db"], db, db_dtype or dtype, SUM * np.abs(dz).sum(axis=0) + grad.sum(axis=0)
              + 2.0 ** -23 * np.abs(db))


def norm_inputs(M, N, dtype, wdtype, gates, gdtype=None, seed=5):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    t = dict(u=(rn(M, N) * (0.3 + torch.rand((M, 1), generator=g, device="cuda"))).to(dtype),
             residual=(2 * rn(M, N)).to(dtype), dy=rn(M, N).to(dtype), dh=rn(M, N).to(dtype),
             gamma_post=(1 + 0.3 * rn(N)).to(wdtype), gamma_pre=(1 + 0.3 * rn(N)).to(wdtype))
    t["gate"] = rn(gates, N).to(gdtype or dtype) if gates else None
    return t


def _of(t, post, pre):
    n = lambda v: None if v is None else f64(v)  # noqa: E731
    return dict(gamma_post=n(t["gamma_post"]) if post else None, gamma_pre=n(t["gamma_pre"]) if pre else None,
                gate=n(t["gate"]), post=post, pre=pre)


def check_norm_fwd(t, out, dtype, residual=True, alpha=1.0, eps=1e-6, post=True, pre=True):
    u, a = f64(t["u"]), _of(t, post, pre)
    u = u.reshape(-1, u.shape[-1])
    res = f64(t["residual"]).reshape(u.shape) if residual else None
    if a["gate"] is not None:
        a["gate"] = a["gate"].reshape(-1, u.shape[1])
    h, _, ru, _ = oracle.block_norm_fwd(u, res, alpha=alpha, eps=eps, **a)  # not rounded
    joined = h if res is None else h - alpha * res
    err = NORM_SUM + 2.0 ** -21  # of a rstd and the products with it, relative
    stats = out["stats"].view(-1, 2)
    check("rstd(u)", stats[:, 0], ru, torch.float32, ru * err)
    if "h" in out:
        check("h", out["h"], h, dtype, np.abs(joined) * (err if post else 2.0 ** -22) + 2.0 ** -23 * np.abs(h))
        h = f64(out["h"]).reshape(h.shape)
    _, y, _, rh = oracle.block_norm_fwd(h, None, gamma_pre=a["gamma_pre"], eps=eps, post=False, pre=True)
    check("rstd(h)", stats[:, 1], rh if pre else 0 * rh, torch.float32, rh * err if pre else 0.0)
    assert ("y" in out) == pre
    if pre:
        check("y", out["y"], y, dtype, np.abs(y) * err)


def check_norm_bwd(t, h, stats, out, dtype, wdtype, gdtype, residual=True, alpha=1.0, post=True, pre=True, dh=True,
                   params=True):
    a = _of(t, post, pre)
    u, hh = f64(t["u"]), f64(h)
    M, N = int(np.prod(u.shape[:-1])), u.shape[-1]
    u, hh, dy = u.reshape(M, N), hh.reshape(M, N), f64(t["dy"]).reshape(M, N)
    g_h = f64(t["dh"]).reshape(M, N) if dh else np.zeros((M, N))
    st = f64(stats).reshape(M, 2)
    if a["gate"] is not None:
        a["gate"] = a["gate"].reshape(-1, N)
    ref = oracle.block_norm_bwd(dy if pre else None, g_h, u, hh, st[:, 0], st[:, 1], alpha=alpha, **a)
    e = 2.0 ** -21
    gate = 1.0 if a["gate"] is None else np.repeat(np.abs(a["gate"]), M // a["gate"].shape[0], axis=0)
    gp = 1.0 if a["gamma_post"] is None else np.abs(a["gamma_post"])
    mean = lambda v: v.mean(axis=1, keepdims=True)  # noqa: E731
    # the gradient D of h, and its error
    if pre:
        rh = st[:, 1:]
        xh, av = np.abs(hh) * rh, np.abs(dy) * (1.0 if a["gamma_pre"] is None else np.abs(a["gamma_pre"]))
        c1 = rh * mean(av * xh)
        ed = e * (np.abs(g_h) + rh * av) + (NORM_SUM + e) * xh * c1
        size = np.abs(g_h) + rh * av + xh * c1
    else:
        ed, size = e * np.abs(g_h), np.abs(g_h)
    d = np.abs(ref["dresidual"]) / abs(alpha) if alpha else np.zeros_like(size)
    if residual:
        check("dresidual", out["dresidual"], ref["dresidual"], dtype, abs(alpha) * (ed + e * d))
    q = gate * gp
    if post:
        uh = np.abs(u) * st[:, :1]
        edu = st[:, :1] * (q * ed + e * q * size + uh * (NORM_SUM + e) * 2 * mean(q * uh * size))
    else:
        uh, edu = np.abs(u), q * (ed + e * size)
    check("du", out["du"], ref["du"], dtype, edu + e * np.abs(ref["du"]))
    names = [k for k, there in (("dgamma_post", post), ("dgamma_pre", pre), ("dgate", a["gate"] is not None)) if there]
    assert all((k in out) == params for k in names)
    if not params:
        return
    if post:
        check("dgamma_post", out["dgamma_post"], ref["dgamma_post"], wdtype,
              (gate * uh * (ed + (NORM_SUM + e) * size)).sum(axis=0))
    if pre:
        check("dgamma_pre", out["dgamma_pre"], ref["dgamma_pre"], wdtype, (NORM_SUM + e) * (np.abs(dy) * xh).sum(axis=0))
    if a["gate"] is not None:
        G = a["gate"].shape[0]
        check("dgate", out["dgate"], ref["dgate"], gdtype,
              (gp * uh * (ed + (NORM_SUM + e) * size)).reshape(G, M // G, N).sum(axis=1))


__all__ = ["ACTS", "NAME", "check_linear_bwd", "check_linear_fwd", "check_norm_bwd", "check_norm_fwd", "f64",
           "linear_inputs", "norm_inputs", "rel"]
