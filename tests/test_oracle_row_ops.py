"""Pins of the fp64 oracle of layer norm, token log probabilities and top-logit
distillation: torch's fp64 autograd of forwards written out here, differences of
the oracle's own forwards, and brute-force rankings."""

import numpy as np
import pytest
import torch

import oracle


def _rng(seed=7):
    return np.random.default_rng(seed)


def test_layer_norm_matches_autograd():
    r = _rng()
    x, res, dy, dh = (r.standard_normal((5, 9)) * 2 + 1 for _ in range(4))
    gamma, beta = r.standard_normal(9), r.standard_normal(9)
    h = torch.tensor(x + res, requires_grad=True)
    g, b = (torch.tensor(v, requires_grad=True) for v in (gamma, beta))
    y = torch.nn.functional.layer_norm(h, (9,), g, b, 1e-3)
    (torch.tensor(dy) * y).sum().backward()
    oy, mu, rstd, oh = oracle.layer_norm_fwd(x, gamma, beta, 1e-3, residual=res)
    np.testing.assert_allclose(oy, y.detach().numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_array_equal(oh, x + res)
    dx, dg, db = oracle.layer_norm_bwd(dy, oh, mu, rstd, gamma, dh=dh)
    np.testing.assert_allclose(dx - dh, h.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(dg, g.grad.numpy(), rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(db, b.grad.numpy(), rtol=1e-12, atol=1e-12)


def test_layer_norm_gradient_by_differences():
    r = _rng(8)
    x, dy, gamma = r.standard_normal((3, 7)), r.standard_normal((3, 7)), r.standard_normal(7)
    f = lambda v: (oracle.layer_norm_fwd(v, gamma, None, 1e-5)[0] * dy).sum()  # noqa: E731
    _, mu, rstd, _ = oracle.layer_norm_fwd(x, gamma, None, 1e-5)
    dx = oracle.layer_norm_bwd(dy, x, mu, rstd, gamma)[0]
    e = 1e-6
    for i in range(3):
        for j in range(7):
            p, m = x.copy(), x.copy()
            p[i, j] += e
            m[i, j] -= e
            assert abs((f(p) - f(m)) / (2 * e) - dx[i, j]) < 1e-7


@pytest.mark.parametrize("tau", [0.5, 1.0, 2.0])
def test_token_logprobs_match_autograd(tau):
    r = _rng(9)
    z = torch.tensor(r.standard_normal((6, 11)) * 3, requires_grad=True)
    t = np.array([0, 10, 5, -100, 3, 3])
    dl, de = r.standard_normal(6), r.standard_normal(6)
    lp = torch.log_softmax(z / tau, dim=1)
    ent = -(lp.exp() * lp).sum(dim=1)
    keep = torch.tensor(t >= 0)
    sel = torch.where(keep, lp[torch.arange(6), torch.tensor(np.maximum(t, 0))], torch.zeros(6, dtype=torch.float64))
    ((torch.tensor(dl) * sel).sum() + (torch.tensor(de) * ent).sum()).backward()
    out = oracle.token_logprobs_fwd(z.detach().numpy(), t, 4, tau)
    np.testing.assert_allclose(out["logp"], sel.detach().numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(out["entropy"], ent.detach().numpy(), rtol=1e-12)
    g = oracle.token_logprobs_bwd(z.detach().numpy(), t, tau, dlogp=dl, dentropy=de)
    np.testing.assert_allclose(g, z.grad.numpy(), rtol=1e-10, atol=1e-13)


def test_token_logprobs_ranking_and_empty_rows():
    z = np.array([[1.0, 3.0, 3.0, -np.inf, 2.0], [-np.inf] * 5, [0.0, -0.0, 0.0, -1.0, 0.0]])
    out = oracle.token_logprobs_fwd(z, np.array([3, 0, 9]), 5, 1.0)
    assert out["top_idx"].tolist() == [[1, 2, 4, 0, 3], [0, 1, 2, 3, 4], [0, 1, 2, 4, 3]]
    assert np.isneginf(out["logp"][0]) and np.isneginf(out["logp"][1]) and np.isnan(out["logp"][2])
    assert out["entropy"][1] == 0 and np.isneginf(out["top_logp"][1]).all()
    assert out["stats"][1].tolist() == [-np.inf, 0.0]
    p = np.exp(z[0] - 3.0) / np.exp(z[0] - 3.0).sum()
    assert abs(out["entropy"][0] + sum(v * np.log(v) for v in p if v > 0)) < 1e-15
    assert not oracle.token_logprobs_bwd(z, np.array([3, 0, 1]), 1.0, dlogp=np.ones(3), dentropy=np.ones(3))[1].any()


@pytest.mark.parametrize("tau", [0.7, 1.0, 3.0])
def test_distillation_matches_autograd(tau):
    r = _rng(10)
    z = torch.tensor(r.standard_normal((4, 13)) * 2, requires_grad=True)
    ids = np.stack([r.permutation(13)[:5] for _ in range(4)])
    ids[1, 3:] = (-1, 13)
    ids[2, 1] = ids[2, 0]  # the same token twice
    tl = r.standard_normal((4, 5)) * 2
    w = r.standard_normal(4)
    lp = torch.log_softmax(z / tau, dim=1)
    total = torch.zeros((), dtype=torch.float64)
    losses = []
    for i in range(4):
        there = [k for k in range(5) if 0 <= ids[i, k] < 13]
        lq = torch.log_softmax(torch.tensor(tl[i, there]) / tau, dim=0)
        loss = (lq.exp() * (lq - lp[i, ids[i, there]])).sum()
        losses.append(float(loss.detach()))
        total = total + w[i] * loss
    total.backward()
    loss, _, _ = oracle.distill_fwd(z.detach().numpy(), ids, tl, tau)
    np.testing.assert_allclose(loss, losses, rtol=1e-12)
    np.testing.assert_allclose(oracle.distill_bwd(w, z.detach().numpy(), ids, tl, tau), z.grad.numpy(),
                               rtol=1e-10, atol=1e-13)


def test_distillation_edges():
    z = np.array([[0.0, 1.0, -np.inf], [0.0, 1.0, 2.0], [-np.inf] * 3])
    ids = np.array([[2, 1], [-1, 7], [0, 1]])
    tl = np.array([[0.0, 0.0], [1.0, 1.0], [0.0, 0.0]])
    loss, _, _ = oracle.distill_fwd(z, ids, tl, 1.0)
    assert np.isposinf(loss[0]) and loss[1] == 0 and np.isposinf(loss[2])
    g = oracle.distill_bwd(np.array([1.0, 1.0, 0.0]), z, ids, tl, 1.0)
    assert g[0, 2] == -0.5 and not g[1].any() and not g[2].any()
    # equal distributions: loss 0, gradient 0
    z = np.array([[0.3, -1.0, 2.0]])
    loss, _, _ = oracle.distill_fwd(z, np.array([[0, 1, 2]]), z, 0.5)
    assert abs(loss[0]) < 1e-15
    assert np.abs(oracle.distill_bwd(np.ones(1), z, np.array([[0, 1, 2]]), z, 0.5)).max() < 1e-15
