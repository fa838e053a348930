"""Timed cases of what stands around a SwiGLU layer in a transformer block: the matrix product with
bias, activation and residual (forward, backward), and the junction of two blocks, which is the norm
after a block, its gate, the scaled residual and the norm before the next block (forward, backward).

`run` makes one pass of a case on the state that `prepare` built: in plain torch operations in fp32
when `own` is false, through the library's entry points when it is true. `exact` restates the
definitions in fp64. `work` counts the bytes and operations a pass cannot do without: each input read
once, each output written once.

Conventions (those of the library):
  linear      z = x w + b, y = f(z) + residual, f one of none, silu, gelu (x Phi(x)), hardswish; x [M, K],
              w [K, N]. Backward from dy and the saved z: dz = dy f'(z), dx = dz w^T, dw = x^T dz,
              db = the sum of dz over the rows.
  block norm  v = u rstd(u) gamma_post (v = u without the norm after the block), h = alpha residual +
              gate v rounded to the I/O type, y = h rstd(h) gamma_pre, rstd(t) = 1 / sqrt(mean(t^2) + eps);
              stats = (rstd(u), rstd(h)) of a row, 0 for a norm that is not there. A gate has one row for
              every M / G rows. The backward takes dy and dh, the gradient that reaches h past the
              second norm.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-6


# ------------------------------------------------------------------------------------ cases
def _lin(op, name, rows, k, n, dtype, act, bias, residual):
    # k, n: the weight's input and output width; residual: (forward) there is one to add
    return {"name": name, "op": op, "rows": rows, "k": k, "n": n, "dtype": dtype, "act": act, "bias": bias,
            "residual": residual}


def _bn(op, name, rows, cols, dtype, weights, gates, post, alpha):
    # weights: type of the gammas; gates: rows of the gate (0: no gate, 1: one for all rows, rows: one for
    # each); post: whether there is a norm after the block; alpha: the residual's scale
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "weights": weights, "gates": gates,
            "post": post, "alpha": alpha}


def listed():
    return [
        # a decoding step of one sequence: the down projection after the LLM-scale SwiGLU layer
        _lin("lin_fwd", "lin_fwd 1x14336x4096 bf16 residual", 1, 14336, 4096, "bf16", "none", False, True),
        # the up projection of some drafted or batched tokens, nothing kept for a backward
        _lin("lin_fwd", "lin_fwd 77x4096x14336 bf16 gelu bias", 77, 4096, 14336, "bf16", "gelu", True, False),
        # an odd batch of short sequences in fp16
        _lin("lin_fwd", "lin_fwd 4097x512x1024 f16 silu bias residual", 4097, 512, 1024, "f16", "silu", True, True),
        # the down projection of a training or prefill batch, with the residual stream
        _lin("lin_fwd", "lin_fwd 16384x14336x4096 bf16 residual", 16384, 14336, 4096, "bf16", "none", False, True),
        # a small odd micro-batch with an activation: two products, the activation's gradient, the bias
        _lin("lin_bwd", "lin_bwd 257x512x1024 f16 gelu bias", 257, 512, 1024, "f16", "gelu", True, False),
        # the many-row FFN workload of this repository: the down projection's gradients, a long reduction
        _lin("lin_bwd", "lin_bwd 220000x1024x512 bf16 bias", 220000, 1024, 512, "bf16", "none", True, False),
        # the LLM-scale down projection's gradients
        _lin("lin_bwd", "lin_bwd 16384x14336x4096 bf16", 16384, 14336, 4096, "bf16", "none", False, False),
        # a decoding step of one sequence between two blocks
        _bn("bn_fwd", "bn_fwd 1x4096 bf16", 1, 4096, "bf16", "bf16", 1, True, 1.0),
        # a training batch of eight sequences, each with its own gate
        _bn("bn_fwd", "bn_fwd 16384x4096 bf16 8 gates", 16384, 4096, "bf16", "bf16", 8, True, 1.0),
        # a small odd batch in full precision, a gate for each token and a scaled residual
        _bn("bn_bwd", "bn_bwd 257x1001 f32 row gates", 257, 1001, "f32", "f32", 257, True, 0.8),
        # the same training batch backward: five gradients
        _bn("bn_bwd", "bn_bwd 16384x4096 bf16 8 gates", 16384, 4096, "bf16", "bf16", 8, True, 1.0),
        # the many-row workload, fp32 master weights, no gate
        _bn("bn_bwd", "bn_bwd 220000x512 bf16", 220000, 512, "bf16", "f32", 0, True, 1.0),
    ]


def _log_int(rng, lo, hi):
    return min(max(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))), lo), hi)


def draw(rng):
    op = rng.choice(["lin_fwd", "lin_fwd", "lin_bwd", "bn_fwd", "bn_bwd"])
    if op.startswith("lin"):
        k, n = (8 * _log_int(rng, 8, 2048) for _ in range(2))
        if rng.random() < 0.5:  # half of the widths are multiples of 64, the others of 8
            k, n = max(64, k // 64 * 64), max(64, n // 64 * 64)
        rows = _log_int(rng, 1, max(1, min(262144, 10 ** 12 // (2 * k * n), 3 * 10 ** 8 // (k + n))))
        act = rng.choice(["none", "none", "silu", "gelu", "hardswish"])
        c = _lin(op, "", rows, k, n, rng.choice(["bf16", "bf16", "f16"]), act, rng.random() < 0.5,
                 op == "lin_fwd" and rng.random() < 0.5)
    else:
        cols = _log_int(rng, 64, 16384)
        if rng.random() < 0.5:
            cols = max(64, cols // 64 * 64)
        most = max(1, min(220000, 40_000_000 // cols))
        rows = _log_int(rng, 1, most)
        kind = rng.choice(["none", "one", "sequences", "rows"])
        gates = {"none": 0, "one": 1, "rows": rows}.get(kind)
        if kind == "sequences":
            gates = rng.randint(1, min(16, rows))
            rows = rows // gates * gates
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        c = _bn(op, "", rows, cols, dtype, rng.choice([dtype, "f32"]), gates, rng.random() < 0.75,
                rng.choice([1.0, 1.0, 0.8]))
    del c["name"]
    return c


# ----------------------------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    dtype, rows, s = DTYPES[case["dtype"]], case["rows"], {"op": case["op"], "case": case}
    if case["op"].startswith("lin"):
        k, n = case["k"], case["n"]
        s["x"] = randn(rows, k).to(dtype)
        s["w"] = (randn(k, n) / math.sqrt(k)).to(dtype)
        s["b"] = (0.2 * randn(n)).to(dtype) if case["bias"] else None
        if case["op"] == "lin_fwd":
            s["residual"] = randn(rows, n).to(dtype) if case["residual"] else None
        else:
            s["dy"] = randn(rows, n).to(dtype)
            s["z"] = randn(rows, n).to(dtype) if case["act"] != "none" else None  # what the forward kept
        return s
    cols, w = case["cols"], DTYPES[case["weights"]]
    # a block's output with a spread of each row's own, and the residual stream, which is wider
    s["u"] = randn(rows, cols).mul_(0.25 + torch.rand((rows, 1), generator=g, device="cuda")).to(dtype)
    r = randn(rows, cols).mul_(2.0).to(dtype)
    s["gamma_post"] = (1 + 0.2 * randn(cols)).to(w) if case["post"] else None
    s["gamma_pre"] = (1 + 0.2 * randn(cols)).to(w)
    s["gate"] = randn(case["gates"], cols).to(dtype) if case["gates"] else None
    if case["op"] == "bn_fwd":
        s["residual"] = r
        return s
    s["dy"], s["dh"] = randn(rows, cols).to(dtype), randn(rows, cols).to(dtype)
    s["h"] = r  # the stream behind the junction, as the forward returned it
    s["stats"] = torch.stack([torch.rsqrt(s[t].float().square().mean(dim=1) + EPS) for t in ("u", "h")], dim=1)
    if not case["post"]:
        s["stats"][:, 0] = 0.0
    return s


# ------------------------------------------------------------------------------ plain forms
def _plain_act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "hardswish":
        return z * (z + 3).clamp(0, 6) / 6
    return z


def _plain_act_grad(z, act):
    if act == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    return torch.where(z <= -3, 0.0, torch.where(z < 3, z / 3 + 0.5, 1.0))  # hardswish


def _plain_lin_fwd(s):
    case, dtype = s["case"], s["x"].dtype
    z = s["x"].float() @ s["w"].float()
    if s["b"] is not None:
        z = z + s["b"].float()
    y = _plain_act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"y": y.to(dtype)}
    if _keeps_z(case):
        out["z"] = z.to(dtype)
    return out


def _keeps_z(case):
    # a training step keeps z for the backward; a few tokens are those of a step that only answers
    return case["act"] != "none" and case["rows"] > 256


def _plain_lin_bwd(s):
    case, dtype = s["case"], s["x"].dtype
    dz = s["dy"].float()
    if case["act"] != "none":
        dz = dz * _plain_act_grad(s["z"].float(), case["act"])
    out = {"dx": (dz @ s["w"].float().t()).to(dtype), "dw": (s["x"].float().t() @ dz).to(dtype)}
    if case["bias"]:
        out["db"] = dz.sum(dim=0).to(dtype)
    return out


def _per_row(gate, rows):
    """A gate's rows for every row: [rows, N], in fp32; 1 without a gate."""
    return 1.0 if gate is None else gate.float().repeat_interleave(rows // gate.shape[0], dim=0)


def _plain_bn_fwd(s):
    case, dtype = s["case"], s["u"].dtype
    f = s["u"].float()
    rstd_u = torch.zeros(f.shape[0], 1, device=f.device)
    if case["post"]:
        rstd_u = 1 / torch.sqrt((f * f).sum(dim=1, keepdim=True) / f.shape[1] + EPS)
        f = f * rstd_u * s["gamma_post"].float()
    h = (case["alpha"] * s["residual"].float() + _per_row(s["gate"], f.shape[0]) * f).to(dtype)
    f = h.float()
    rstd_h = 1 / torch.sqrt((f * f).sum(dim=1, keepdim=True) / f.shape[1] + EPS)
    return {"h": h, "y": (f * rstd_h * s["gamma_pre"].float()).to(dtype), "stats": torch.cat([rstd_u, rstd_h], dim=1)}


def _plain_bn_bwd(s):
    case, dtype = s["case"], s["u"].dtype
    rstd_u, rstd_h = s["stats"][:, :1], s["stats"][:, 1:]
    rows, n = s["u"].shape
    hh, dy = s["h"].float() * rstd_h, s["dy"].float()
    out = {"dgamma_pre": (dy * hh).sum(dim=0).to(s["gamma_pre"].dtype)}
    a = dy * s["gamma_pre"].float()
    d = s["dh"].float() + rstd_h * (a - hh * ((a * hh).sum(dim=1, keepdim=True) / n))
    out["dresidual"] = (case["alpha"] * d).to(dtype)
    v = s["u"].float()
    g = _per_row(s["gate"], rows)
    if case["post"]:
        uh = v * rstd_u
        v = uh * s["gamma_post"].float()
        out["dgamma_post"] = (d * g * uh).sum(dim=0).to(s["gamma_post"].dtype)
    if s["gate"] is not None:
        gates = s["gate"].shape[0]
        out["dgate"] = (d * v).view(gates, rows // gates, n).sum(dim=1).to(s["gate"].dtype)
    d = d * g
    if case["post"]:
        d = d * s["gamma_post"].float()
        d = rstd_u * (d - uh * ((d * uh).sum(dim=1, keepdim=True) / n))
    out["du"] = d.to(dtype)
    return out


PLAIN = {"lin_fwd": _plain_lin_fwd, "lin_bwd": _plain_lin_bwd, "bn_fwd": _plain_bn_fwd, "bn_bwd": _plain_bn_bwd}


# ---------------------------------------------------------------------- the library's calls
def _own(s):
    import swiglu_ffn_backward_gb300 as swg

    case = s["case"]
    act = None if case.get("act") == "none" else case.get("act")
    if s["op"] == "lin_fwd":
        return swg.linear_fwd(s["x"], s["w"], s["b"], act=act, residual=s["residual"], save_z=_keeps_z(case))
    if s["op"] == "lin_bwd":
        return swg.linear_bwd(s["dy"], s["x"], s["w"], z=s["z"], act=act, bias=case["bias"])
    if s["op"] == "bn_fwd":
        return swg.block_norm_fwd(s["u"], s["residual"], gamma_post=s["gamma_post"], gamma_pre=s["gamma_pre"],
                                  gate=s["gate"], alpha=case["alpha"], eps=EPS, post=case["post"])
    return swg.block_norm_bwd(s["dy"], s["dh"], s["u"], s["h"], s["stats"], gamma_post=s["gamma_post"],
                              gamma_pre=s["gamma_pre"], gate=s["gate"], alpha=case["alpha"], post=case["post"])


def _in_order(case, out):
    """The outputs of a pass under one set of names, in one order."""
    if case["op"] == "lin_fwd":
        names = ["y", "z"] if _keeps_z(case) else ["y"]
    elif case["op"] == "lin_bwd":
        names = ["dx", "dw", "db"] if case["bias"] else ["dx", "dw"]
    elif case["op"] == "bn_fwd":
        names = ["h", "y", "stats"]
    else:
        names = ["du", "dresidual", "dgamma_pre"]
        names += ["dgamma_post"] if case["post"] else []
        names += ["dgate"] if case["gates"] else []
    return {k: out[k] for k in names}


def run(state):
    return _in_order(state["case"], _own(state) if own else PLAIN[state["op"]](state))


# ------------------------------------------------------------------------------ work, exact
def work(case):
    rows, es = case["rows"], 4 if case["dtype"] == "f32" else 2
    if case["op"].startswith("lin"):
        k, n = case["k"], case["n"]
        if case["op"] == "lin_fwd":
            count = rows * k + k * n + n * case["bias"] + rows * n * (1 + case["residual"] + _keeps_z(case))
            return {"bytes": es * count, "flops": 2 * rows * k * n}
        count = rows * n * (1 + (case["act"] != "none")) + 2 * rows * k + 2 * k * n + n * case["bias"]
        return {"bytes": es * count, "flops": 4 * rows * k * n}
    cols, ws = case["cols"], 4 if case["weights"] == "f32" else 2
    n = rows * cols
    if case["op"] == "bn_fwd":
        return {"bytes": es * (4 * n + case["gates"] * cols) + ws * cols * (1 + case["post"]) + 8 * rows,
                "flops": 9 * n}
    return {"bytes": es * (6 * n + 2 * case["gates"] * cols) + 2 * ws * cols * (1 + case["post"]) + 8 * rows,
            "flops": 24 * n}


def _exact_act(z, act):
    if act == "silu":
        return z * torch.sigmoid(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    if act == "hardswish":
        return torch.where(z <= -3, torch.zeros_like(z), torch.where(z >= 3, z, z * (z + 3) / 6))
    return z


def _exact_norm(t, gamma):
    rstd = (t.pow(2).mean(dim=1) + EPS) ** -0.5
    return torch.einsum("ij,i,j->ij", t, rstd, gamma), rstd


def _exact_gated(v, gate):
    return v if gate is None else (v.view(gate.shape[0], -1, v.shape[1]) * gate.unsqueeze(1)).view_as(v)


def _leaf(t):
    return None if t is None else t.double().requires_grad_()


def exact(case, seed):
    s, act = prepare(case, seed), case.get("act")
    if case["op"] == "lin_fwd":
        z = torch.einsum("ik,kj->ij", s["x"].double(), s["w"].double())
        z = z if s["b"] is None else z + s["b"].double()
        y = _exact_act(z, act)
        return _in_order(case, {"y": y if s["residual"] is None else y + s["residual"].double(), "z": z})
    if case["op"] == "lin_bwd":
        dz = s["dy"].double()
        if act != "none":  # the activation's gradient by differentiating its definition
            z = _leaf(s["z"])
            dz, = torch.autograd.grad(_exact_act(z, act), z, dz)
        return _in_order(case, {"dx": torch.einsum("ij,kj->ik", dz, s["w"].double()),
                                "dw": torch.einsum("ik,ij->kj", s["x"].double(), dz), "db": dz.sum(dim=0)})
    if case["op"] == "bn_fwd":
        v, rstd_u = s["u"].double(), torch.zeros(case["rows"], dtype=torch.float64, device="cuda")
        if case["post"]:
            v, rstd_u = _exact_norm(v, s["gamma_post"].double())
        gate = None if s["gate"] is None else s["gate"].double()
        h = (case["alpha"] * s["residual"].double() + _exact_gated(v, gate)).to(s["u"].dtype).double()
        y, rstd_h = _exact_norm(h, s["gamma_pre"].double())
        return _in_order(case, {"h": h, "y": y, "stats": torch.stack([rstd_u, rstd_h], dim=1)})
    # the gradients by differentiating the two halves of the forward in fp64
    h, gamma_pre = _leaf(s["h"]), _leaf(s["gamma_pre"])
    d, dgamma_pre = torch.autograd.grad(_exact_norm(h, gamma_pre)[0], (h, gamma_pre), s["dy"].double())
    d = d + s["dh"].double()
    u, gamma_post, gate = _leaf(s["u"]), _leaf(s["gamma_post"]), _leaf(s["gate"])
    v = _exact_norm(u, gamma_post)[0] if case["post"] else u
    leaves = {k: t for k, t in (("du", u), ("dgamma_post", gamma_post), ("dgate", gate)) if t is not None}
    grads = torch.autograd.grad(_exact_gated(v, gate), tuple(leaves.values()), d)
    return _in_order(case, {"dresidual": case["alpha"] * d, "dgamma_pre": dgamma_pre, **dict(zip(leaves, grads))})
