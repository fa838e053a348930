"""Pins of the fp64 oracle of the linear layer and of the norms between blocks: torch's fp64 autograd of forwards
written out here, and differences of the oracle's own forwards."""

import itertools

import numpy as np
import pytest
import torch

import oracle


def _rng(seed):
    return np.random.default_rng(seed)


def _torch_act(z, act):
    f = torch.nn.functional
    return {None: lambda v: v, "silu": f.silu, "gelu": f.gelu, "hardswish": f.hardswish}[act](z)


@pytest.mark.parametrize("act", [None, "silu", "gelu", "hardswish"])
def test_linear_matches_autograd(act):
    r = _rng(1)
    x, w, b, res, dy = (r.standard_normal(s) for s in ((6, 5), (5, 7), (7,), (6, 7), (6, 7)))
    x = x * 2
    tx, tw, tb, tr = (torch.tensor(v, requires_grad=True) for v in (x, w, b, res))
    z = tx @ tw + tb
    y = _torch_act(z, act) + tr
    (y * torch.tensor(dy)).sum().backward()
    oy, oz = oracle.linear_fwd(x, w, b, act, res)
    np.testing.assert_allclose(oz, z.detach().numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(oy, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    dx, dw, db, _ = oracle.linear_bwd(dy, x, w, oz, act)
    for got, want in ((dx, tx), (dw, tw), (db, tb)):
        np.testing.assert_allclose(got, want.grad.numpy(), rtol=1e-11, atol=1e-11)


@pytest.mark.parametrize("act", [None, "silu", "gelu", "hardswish"])
def test_linear_gradient_by_differences(act):
    r = _rng(2)
    x, w, dy = r.standard_normal((2, 3)), r.standard_normal((3, 4)), r.standard_normal((2, 4))
    f = lambda x, w: (oracle.linear_fwd(x, w, None, act)[0] * dy).sum()  # noqa: E731
    dx, dw, _, _ = oracle.linear_bwd(dy, x, w, oracle.linear_fwd(x, w, None, act)[1], act)
    e = 1e-6
    for t, d, at in ((x, dx, 0), (w, dw, 1)):
        for i in np.ndindex(*t.shape):
            p, m = t.copy(), t.copy()
            p[i] += e
            m[i] -= e
            num = (f(p, w) - f(m, w)) if at == 0 else (f(x, p) - f(x, m))
            assert abs(num / (2 * e) - d[i]) < 1e-7


def test_linear_rounds_dz():
    r = _rng(3)
    dy, x, w, z = (r.standard_normal(s) for s in ((4, 8), (4, 8), (8, 8), (4, 8)))
    dx, dw, db, dz = oracle.linear_bwd(dy, x, w, z, "silu", "bf16")
    exact = oracle.act_grad(dy, z, "silu")
    np.testing.assert_array_equal(dz, oracle.f64_to_bf16_value(exact))
    np.testing.assert_allclose(db, exact.sum(axis=0), rtol=1e-14)
    np.testing.assert_allclose(dw, x.T @ dz, rtol=1e-14)


CASES = [(g, res, post, pre, alpha) for g, res, post, pre, alpha in itertools.product(
    (0, 1, 3, 6), (True, False), (True, False), (True, False), (1.0, 0.7)) if post or pre]


@pytest.mark.parametrize("gates,res,post,pre,alpha", CASES)
def test_block_norm_matches_autograd(gates, res, post, pre, alpha):
    r = _rng(4)
    M, N, eps = 6, 9, 1e-3
    t = {k: torch.tensor(r.standard_normal(s), requires_grad=True)
         for k, s in (("u", (M, N)), ("r", (M, N)), ("gp", (N,)), ("gn", (N,)), ("g", (max(gates, 1), N)))}
    dy, dh = r.standard_normal((M, N)), r.standard_normal((M, N))
    norm = lambda v, g: v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps) * g  # noqa: E731
    v = norm(t["u"], t["gp"]) if post else t["u"]
    if gates:
        v = torch.cat([v[i * (M // gates):(i + 1) * (M // gates)] * t["g"][i] for i in range(gates)])
    h = v + alpha * t["r"] if res else v
    loss = (h * torch.tensor(dh)).sum()
    if pre:
        y = norm(h, t["gn"])
        loss = loss + (y * torch.tensor(dy)).sum()
    loss.backward()
    n = {k: v.detach().numpy() for k, v in t.items()}
    args = dict(gamma_post=n["gp"] if post else None, gamma_pre=n["gn"] if pre else None,
                gate=n["g"] if gates else None, alpha=alpha, post=post, pre=pre)
    oh, oy, ru, rh = oracle.block_norm_fwd(n["u"], n["r"] if res else None, eps=eps, **args)
    np.testing.assert_allclose(oh, h.detach().numpy(), rtol=1e-12, atol=1e-12)
    if pre:
        np.testing.assert_allclose(oy, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    got = oracle.block_norm_bwd(dy if pre else None, dh, n["u"], oh, ru, rh, **args)
    for k, leaf, there in (("du", "u", True), ("dresidual", "r", res), ("dgamma_post", "gp", post),
                           ("dgamma_pre", "gn", pre), ("dgate", "g", gates > 0)):
        if there:
            np.testing.assert_allclose(got[k], t[leaf].grad.numpy(), rtol=1e-9, atol=1e-11, err_msg=k)
        elif k not in ("dresidual",):
            assert got[k] is None


def test_block_norm_gradient_by_differences():
    r = _rng(5)
    u, res, gate = r.standard_normal((4, 5)), r.standard_normal((4, 5)), r.standard_normal((2, 5))
    gp, gn, dy, dh = r.standard_normal(5), r.standard_normal(5), r.standard_normal((4, 5)), r.standard_normal((4, 5))

    def loss(**change):
        a = {**dict(u=u, residual=res, gate=gate, gamma_post=gp, gamma_pre=gn), **change}
        h, y, _, _ = oracle.block_norm_fwd(alpha=0.5, **a)
        return (h * dh + y * dy).sum()

    h, _, ru, rh = oracle.block_norm_fwd(u, res, gp, gn, gate, alpha=0.5)
    got = oracle.block_norm_bwd(dy, dh, u, h, ru, rh, gp, gn, gate, alpha=0.5)
    e = 1e-6
    for name, t in (("u", u), ("residual", res), ("gate", gate), ("gamma_post", gp), ("gamma_pre", gn)):
        for i in np.ndindex(*t.shape):
            p, m = t.copy(), t.copy()
            p[i] += e
            m[i] -= e
            assert abs((loss(**{name: p}) - loss(**{name: m})) / (2 * e) - got["d" + name][i]) < 1e-7
