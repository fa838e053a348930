"""Training steps of one transformer block's feed-forward half and its head, distilled from a teacher's top
logits, and scoring of given tokens with the result:

    h  = u + r                            layer_norm_fwd (adds the residual)
    x  = LN(h)
    a  = SiLU(x W_g) (x W_fc)             swiglu_fwd
    h' = h + a W_out                      layer_norm_fwd
    z  = LN(h') E^T                       the logits
    loss, dz                              distill_fwd_bwd (dz over z)
    ... back through layer_norm_bwd, swiglu_bwd, layer_norm_bwd

    python examples/distill_step.py [--tokens 2048 --cols 512 --hidden 1024 --vocab 32000 --steps 20]

u and r stand for what attention and the residual stream bring. The matrix products by W_out and E are
plain library ones.
"""

import argparse
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import swiglu_ffn_backward_gb300 as swg  # noqa: E402


def make_params(cols, hidden, vocab, seed=0, device="cuda"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    rn = lambda *s, scale: (torch.randn(s, generator=g, device=device) * scale).bfloat16()  # noqa: E731
    return {"gamma1": torch.ones(cols, device=device), "beta1": torch.zeros(cols, device=device),
            "w_g": rn(cols, hidden, scale=cols ** -0.5), "w_fc": rn(cols, hidden, scale=cols ** -0.5),
            "w_out": rn(hidden, cols, scale=hidden ** -0.5),
            "gamma2": torch.ones(cols, device=device), "beta2": torch.zeros(cols, device=device),
            "embed": rn(vocab, cols, scale=cols ** -0.5)}


def forward(p, u, r):
    """The logits, and what the backward needs."""
    n1 = swg.layer_norm_fwd(u, p["gamma1"], p["beta1"], residual=r)
    f = swg.swiglu_fwd(n1["y"], p["w_g"], p["w_fc"])
    n2 = swg.layer_norm_fwd(f["y"] @ p["w_out"], p["gamma2"], p["beta2"], residual=n1["h"])
    return n2["y"] @ p["embed"].t(), (n1, f, n2)


def backward(p, saved, dz):
    """Gradients of the parameters and of u (which is also that of r)."""
    n1, f, n2 = saved
    grads = {"embed": dz.t() @ n2["y"]}
    dh2, grads["gamma2"], grads["beta2"] = swg.layer_norm_bwd(dz @ p["embed"], n2["h"], n2["stats"], gamma=p["gamma2"])
    grads["w_out"] = f["y"].t() @ dh2
    ffn = swg.swiglu_bwd(n1["y"], p["w_g"], p["w_fc"], dh2 @ p["w_out"].t(), f["g"], f["fc"], return_dg=False)
    grads["w_g"], grads["w_fc"] = ffn["dw_g"], ffn["dw_fc"]
    # dh2 also reaches h past the block: it is added inside the kernel
    grads["u"], grads["gamma1"], grads["beta1"] = swg.layer_norm_bwd(ffn["dx"], n1["h"], n1["stats"],
                                                                     gamma=p["gamma1"], dh=dh2)
    return grads


def distill_step(p, u, r, ids, teacher, weight, temperature):
    """Loss of each token and the gradients of sum(weight loss)."""
    z, saved = forward(p, u, r)
    out = swg.distill_fwd_bwd(z, ids, teacher, weight, temperature=temperature, out={"dlogits": z})
    return out["loss"], backward(p, saved, out["dlogits"])


def score(p, u, r, tokens, top_k=5):
    """Log probabilities of the given tokens, entropies, and the best alternatives."""
    return swg.token_logprobs_fwd(forward(p, u, r)[0], tokens, top_k=top_k)


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("tokens", 2048), ("cols", 512), ("hidden", 1024), ("vocab", 32000), ("entries", 64),
                          ("steps", 20)):
        ap.add_argument(f"--{name}", type=int, default=default)
    ap.add_argument("--lr", type=float, default=1.0)
    ap.add_argument("--temperature", type=float, default=1.0)
    args = ap.parse_args(argv)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    rn = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    p = make_params(args.cols, args.hidden, args.vocab)
    u, r = rn(args.tokens, args.cols).bfloat16(), rn(args.tokens, args.cols).bfloat16()
    # the teacher is another block, of which only the largest logits are kept
    teacher, ids = forward(make_params(args.cols, args.hidden, args.vocab, seed=7), u, r)[0].float().mul_(3) \
        .topk(args.entries, dim=1)
    weight = torch.full((args.tokens,), 1.0 / args.tokens, device="cuda")
    losses = []
    for step in range(args.steps):
        loss, grads = distill_step(p, u, r, ids, teacher, weight, args.temperature)
        for k, v in p.items():
            v.sub_(grads[k].to(v.dtype), alpha=args.lr)
        losses.append(float(loss.mean()))
        print(f"step {step}: loss {losses[-1]:.4f}")
    out = score(p, u, r, ids[:, 0])
    print(f"the teacher's first token: log probability {float(out['logp'].mean()):.4f}, "
          f"among the five best in {float((out['top_idx'] == ids[:, :1]).any(1).float().mean()):.1%} of the rows, "
          f"entropy {float(out['entropy'].mean()):.3f}")
    swg.swg_check()
    return losses


if __name__ == "__main__":
    main()
