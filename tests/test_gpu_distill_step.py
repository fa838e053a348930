"""The example that runs the row-wise operators around the SwiGLU block: its gradients against autograd on
the same formulas in fp64, and its training (GPU)."""

import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


def _example():
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "distill_step.py")
    spec = importlib.util.spec_from_file_location("distill_step", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def _inputs(ex, T, cols, hidden, vocab, entries):
    g = torch.Generator(device="cuda")
    g.manual_seed(5)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    p = ex.make_params(cols, hidden, vocab)
    u, r = rn(T, cols).bfloat16(), rn(T, cols).bfloat16()
    ids = torch.rand((T, vocab), generator=g, device="cuda").topk(entries, dim=1).indices
    return p, u, r, ids, rn(T, entries) * 2, torch.rand(T, generator=g, device="cuda") / T


def _norm(h, gamma, beta):
    return torch.nn.functional.layer_norm(h, h.shape[-1:], gamma, beta, eps=1e-5)


def _reference(p, u, r, ids, teacher, weight, tau):
    q = {k: v.double().requires_grad_() for k, v in {**p, "u": u}.items()}
    h = q["u"] + r.double()
    x = _norm(h, q["gamma1"], q["beta1"])
    a = torch.nn.functional.silu(x @ q["w_g"]) * (x @ q["w_fc"])
    z = _norm(h + a @ q["w_out"], q["gamma2"], q["beta2"]) @ q["embed"].t()
    lq = torch.log_softmax(teacher.double() / tau, dim=1)
    loss = (lq.exp() * (lq - torch.log_softmax(z / tau, dim=1).gather(1, ids))).sum(dim=1)
    (loss * weight.double()).sum().backward()
    return z.detach(), loss.detach(), {k: v.grad for k, v in q.items()}


@pytest.mark.parametrize("T,cols,hidden,vocab", [(256, 64, 128, 1000), (384, 128, 256, 8008)])
def test_gradients(T, cols, hidden, vocab):
    ex = _example()
    p, u, r, ids, teacher, weight = _inputs(ex, T, cols, hidden, vocab, 20)
    z, want, grads = _reference(p, u, r, ids, teacher, weight, 2.0)
    loss, got = ex.distill_step(p, u, r, ids, teacher, weight, 2.0)
    # some ten tensors on the way are rounded to bf16, 2^-9 relative each: in the norm 10 2^-9 < 2^-5, of the
    # gradients, and of the logits, which enter the loss over tau
    rel = lambda a, b: float((a.double() - b).norm() / b.norm())  # noqa: E731
    assert float((loss.double() - want).abs().max()) <= 2.0 ** -5 * float(z.abs().max())
    assert set(got) == set(grads)
    for k, v in grads.items():
        assert rel(got[k], v) <= 2.0 ** -5, k


def test_scores():
    ex = _example()
    p, u, r, ids, _, _ = _inputs(ex, 256, 64, 128, 1000, 20)
    z = ex.forward(p, u, r)[0].double()
    lp = torch.log_softmax(z, dim=1)
    out = ex.score(p, u, r, ids[:, 0], top_k=5)
    # the library's own logits, summed in fp32: 2^-17 relative of the sum, 2^-22 of the logits' size
    bound = 2.0 ** -16 + 2.0 ** -21 * float(z.abs().max())
    assert float((out["logp"].double() - lp.gather(1, ids[:, :1])[:, 0]).abs().max()) <= bound
    assert torch.equal(z.gather(1, out["top_idx"]), z.topk(5, dim=1).values)


def test_training_lowers_the_loss():
    losses = _example().main("--tokens 256 --cols 64 --hidden 128 --vocab 1000 --entries 20 --steps 8".split())
    assert all(b < a for a, b in zip(losses, losses[1:]))
