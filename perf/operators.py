"""Timed cases of the operators around a SwiGLU block: layer norm (forward, backward with the
weight gradients), log probabilities of given tokens with entropy and top alternatives (forward,
backward), and distillation from a teacher's top logits (forward, backward, and both in one call).

`run` makes one pass of a case on the state that `prepare` built: in plain torch operations in
fp32 when `own` is false, through the library's entry points when it is true. `exact` restates the
definitions in fp64. `work` counts the bytes and operations a pass cannot do without: each input
read once, each output written once.

Conventions (those of the library):
  layer norm   h = x + residual rounded to the I/O type (h = x without one); mean, biased variance,
               rstd = 1 / sqrt(var + eps); y = (h - mean) rstd gamma + beta; stats = (mean, rstd).
  row softmax  stats = (max, sum exp((z - max) / temperature)); a row with no logit above -inf has
               stats (-inf, 0), probability 0 everywhere, entropy 0 and log probabilities -inf.
  tokens       a target equal to -100 is ignored: log probability 0, no gradient.
  distillation q = softmax of the teacher's entries over temperature (ids outside the vocabulary are
               absent entries), loss = sum q (ln q - ln p), p the student's full softmax; a row
               without entries has loss 0 and no gradient.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
IGNORE = -100
EPS = 1e-5
NEG_INF = float("-inf")


# ------------------------------------------------------------------------------------ cases
def _ln(op, name, rows, cols, dtype, weights, add):
    # weights: type of gamma and beta; add: a residual to add first (forward), the residual path's
    # gradient to add to dx (backward)
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "weights": weights, "add": add}


def _lp(op, name, rows, cols, dtype, top, temperature, masked, pad):
    # masked: part of the vocabulary is -inf or the type's lowest value, some rows wholly, and some
    # targets are ignored; pad: columns between the end of a row and the next row's start
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "top": top,
            "temperature": temperature, "masked": masked, "pad": pad}


def _kd(op, name, rows, cols, dtype, entries, temperature, masked):
    # masked: rows of weight 0, absent entries, rows without entries
    return {"name": name, "op": op, "rows": rows, "cols": cols, "dtype": dtype, "entries": entries,
            "temperature": temperature, "masked": masked}


def listed():
    return [
        # a decoding step of one sequence: the add-and-norm before its FFN
        _ln("ln_fwd", "ln_fwd 1x4096 bf16 add", 1, 4096, "bf16", "bf16", True),
        # the norm before the LLM-scale FFN, with the residual add
        _ln("ln_fwd", "ln_fwd 16384x4096 bf16 add", 16384, 4096, "bf16", "bf16", True),
        # a small odd batch in full precision: latency counts, nothing is a multiple of a vector
        _ln("ln_bwd", "ln_bwd 257x1001 f32", 257, 1001, "f32", "f32", False),
        # the many-row FFN workload of this repository, fp32 master weights, residual gradient
        _ln("ln_bwd", "ln_bwd 220000x512 bf16 add", 220000, 512, "bf16", "f32", True),
        # sampling one token: its log probability and the 20 best alternatives
        _lp("logp_fwd", "logp_fwd 1x131072 f32 top20", 1, 131072, "f32", 20, 1.0, False, 0),
        # scoring a prompt batch
        _lp("logp_fwd", "logp_fwd 4096x131072 bf16 top20", 4096, 131072, "bf16", 20, 1.0, False, 0),
        # constrained decoding scores: masked vocabulary, rows padded in memory, odd vocabulary
        _lp("logp_fwd", "logp_fwd 515x50001 f16 top5 masked", 515, 50001, "f16", 5, 0.7, True, 47),
        # a policy-gradient step with an entropy bonus
        _lp("logp_bwd", "logp_bwd 4096x65536 bf16", 4096, 65536, "bf16", 0, 1.0, False, 0),
        # a distillation step over one large micro-batch: loss and gradient at once
        _kd("kd_step", "kd_step 4096x131072 bf16 k64", 4096, 131072, "bf16", 64, 2.0, False),
        # a tiny odd micro-batch in full precision, with padding tokens
        _kd("kd_step", "kd_step 16x50001 f32 k32 masked", 16, 50001, "f32", 32, 1.0, True),
        # the loss on held-out text
        _kd("kd_fwd", "kd_fwd 2048x32768 bf16 k128", 2048, 32768, "bf16", 128, 1.0, False),
        # the gradient alone (the loss enters a larger graph), odd vocabulary
        _kd("kd_bwd", "kd_bwd 2048x65537 f16 k20 masked", 2048, 65537, "f16", 20, 2.0, True),
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(max(n, lo), hi)
    if rng.random() < 0.5:  # half of the sizes land on a multiple of 64, the others where they fall
        n = max(lo, n // 64 * 64)
    return n + 1 if n == 3 * 1024 else n


def draw(rng):
    op = rng.choice(["ln_fwd", "ln_bwd", "logp_fwd", "logp_bwd", "kd_step", "kd_fwd", "kd_bwd"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op.startswith("ln"):
        cols = _log_int(rng, 64, 16384)
        rows = _log_int(rng, 1, max(1, min(220000, 48_000_000 // cols)))
        c = _ln(op, "", rows, cols, dtype, rng.choice([dtype, "f32"]), rng.random() < 0.5)
    else:
        cols = _log_int(rng, 1000, 160000)
        rows = _log_int(rng, 1, max(1, min(16384, 160_000_000 // cols)))
        temperature = rng.choice([0.7, 1.0, 1.0, 2.0])
        masked = rng.random() < 0.4
        if op.startswith("logp"):
            c = _lp(op, "", rows, cols, dtype, rng.randint(0, 32) if op == "logp_fwd" else 0, temperature, masked,
                    rng.choice([0, 0, 1, 64]))
        else:
            c = _kd(op, "", rows, cols, dtype, rng.choice([8, 20, 50, 64, 128]), temperature, masked)
    del c["name"]
    return c


# ----------------------------------------------------------------------------------- inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _logits(g, rows, cols, dtype, pad):
    z = _randn(g, rows, cols + pad).mul_(2.5).to(dtype)
    return z[:, :cols]


def _mask_vocabulary(g, z):
    """Every fourth row keeps about 1 token in 50 (the others -inf), one of eight has its second half
    at the type's lowest value; the second row, and every 64th after it, keeps no token at all."""
    rows, cols = z.shape
    r = torch.arange(rows, device="cuda")
    drop = torch.rand((rows, cols), generator=g, device="cuda") > 0.02
    z.masked_fill_(drop & (r % 4 == 0).unsqueeze(1), NEG_INF)
    z[r % 8 == 3, cols // 2:] = torch.finfo(z.dtype).min
    z[r % 64 == 1] = NEG_INF


def _row_stats64(z, temperature):
    """(max, sum, ln sum, (z - max) / temperature) of rows in fp64, the definitions of `exact`."""
    f = z.double()
    m = f.max(dim=1, keepdim=True).values
    d = (f - torch.where(torch.isinf(m), torch.zeros_like(m), m)) / temperature
    s = torch.exp(d).sum(dim=1, keepdim=True)
    return m, s, torch.log(s), d


def _entropy64(d, s, log_s):
    p = torch.exp(d) / s
    h = -torch.where(p > 0, p * (d - log_s), torch.zeros_like(p)).sum(dim=1, keepdim=True)
    return torch.where(s > 0, h, torch.zeros_like(h))


def _chunks(rows, cols):
    step = max(1, 32_000_000 // cols)
    return [(i, min(rows, i + step)) for i in range(0, rows, step)]


def prepare(case, seed):
    g = _gen(seed)
    rows, cols, dtype, op = case["rows"], case["cols"], DTYPES[case["dtype"]], case["op"]
    s = {"op": op, "case": case}
    if op.startswith("ln"):
        w = DTYPES[case["weights"]]
        # activations of a residual stream: a mean and a spread of each row's own
        x = _randn(g, rows, cols).mul_(0.5 + torch.rand((rows, 1), generator=g, device="cuda")).add_(_randn(g, rows, 1))
        s["x"] = x.to(dtype)
        del x
        s["gamma"] = (1 + 0.2 * _randn(g, cols)).to(w)
        s["beta"] = (0.1 * _randn(g, cols)).to(w)
        if op == "ln_fwd":
            s["residual"] = _randn(g, rows, cols).to(dtype) if case["add"] else None
        else:
            s["dy"] = _randn(g, rows, cols).to(dtype)
            s["dh"] = _randn(g, rows, cols).to(dtype) if case["add"] else None
            f = s["x"].float()
            mean = f.mean(dim=1)
            var = f.sub_(mean.unsqueeze(1)).square_().mean(dim=1)
            s["stats"] = torch.stack([mean, torch.rsqrt(var + EPS)], dim=1)
        return s
    temperature = case["temperature"]
    z = _logits(g, rows, cols, dtype, case.get("pad", 0))
    target = torch.randint(0, cols, (rows,), generator=g, device="cuda")
    # a trained model favours the given token in most places
    boost = (torch.rand((rows, 1), generator=g, device="cuda") < 0.8) * 9.0
    r = torch.arange(rows, device="cuda")
    z[r, target] = (z[r, target].float() + boost[:, 0]).to(dtype)
    if op.startswith("logp"):
        if case["masked"]:
            _mask_vocabulary(g, z)
            target = torch.where(torch.rand(rows, generator=g, device="cuda") < 0.1, IGNORE, target)
        s["logits"], s["target"] = z, target
        if op == "logp_bwd":
            s["dlogp"] = _randn(g, rows)
            s["dentropy"] = 0.1 * _randn(g, rows)
    else:
        k = min(case["entries"], cols)
        # the teacher: the student's logits with noise, of which the k largest are kept
        ids, vals = [], []
        for i, j in _chunks(rows, cols):
            t = z[i:j].float() + 1.5 * _randn(g, j - i, cols)
            v, n = t.topk(k, dim=1)
            ids.append(n)
            vals.append(v)
        ids, vals = torch.cat(ids), torch.cat(vals)
        w = torch.rand(rows, generator=g, device="cuda") + 0.5
        if case["masked"]:
            ids[:, k - k // 4:] = torch.where(r.unsqueeze(1) % 3 == 0, -1, ids[:, k - k // 4:])  # fewer entries
            ids[r % 16 == 5] = -1                                                                # none
            w = torch.where(r % 8 == 2, 0.0, w)                                                  # padding tokens
        w = w * ((1024.0 if case["dtype"] == "f16" else 1.0) / rows)  # a mean over the tokens; fp16 with its loss scale
        s["logits"], s["ids"], s["teacher"], s["weight"] = z, ids, vals.to(dtype), w
    if op in ("logp_bwd", "kd_bwd"):
        stats, ent = [], []
        for i, j in _chunks(rows, cols):
            m, t, log_s, d = _row_stats64(z[i:j], temperature)
            stats.append(torch.cat([m, t], dim=1).float())
            ent.append(_entropy64(d, t, log_s)[:, 0].float())
        s["stats"], s["entropy"] = torch.cat(stats), torch.cat(ent)
    return s


# ------------------------------------------------------------------------------ plain forms
def _plain_ln_fwd(s):
    x, res = s["x"], s["residual"]
    h = x if res is None else (x.float() + res.float()).to(x.dtype)
    f = h.float()
    n = f.shape[1]
    mean = f.sum(dim=1, keepdim=True) / n
    d = f - mean
    rstd = 1.0 / torch.sqrt((d * d).sum(dim=1, keepdim=True) / n + EPS)
    y = (d * rstd * s["gamma"].float() + s["beta"].float()).to(x.dtype)
    out = {"y": y, "stats": torch.cat([mean, rstd], dim=1)}
    if res is not None:
        out["h"] = h
    return out


def _plain_ln_bwd(s):
    x, dy, dh = s["x"], s["dy"], s["dh"]
    mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    n = x.shape[1]
    g = dy.float()
    xh = (x.float() - mean) * rstd
    dgamma = (g * xh).sum(dim=0).to(s["gamma"].dtype)
    dbeta = g.sum(dim=0).to(s["gamma"].dtype)
    g = g * s["gamma"].float()
    a = g.sum(dim=1, keepdim=True) / n
    b = (g * xh).sum(dim=1, keepdim=True) / n
    dx = rstd * (g - a - xh * b)
    if dh is not None:
        dx = dx + dh.float()
    return {"dx": dx.to(x.dtype), "dgamma": dgamma, "dbeta": dbeta}


def _plain_rows(z, temperature):
    f = z.float()
    m = f.amax(dim=1, keepdim=True)
    d = (f - torch.where(m == NEG_INF, 0.0, m)) / temperature
    e = torch.exp(d)
    return f, m, d, e, e.sum(dim=1, keepdim=True)


def _plain_top(f, k):
    """The k largest of each row, ties to the lowest index: one unique 64-bit key for each element, the
    value's order in the high half, the index counted down in the low half."""
    bits = (f + 0.0).view(torch.int32)
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
    n = f.shape[1]
    key = (order << 32) + (n - 1 - torch.arange(n, device=f.device))
    return n - 1 - (key.topk(k, dim=1).values & 0xFFFFFFFF)


def _plain_logp_fwd(s):
    case = s["case"]
    f, m, d, e, t = _plain_rows(s["logits"], case["temperature"])
    log_s = torch.log(t)
    ent = torch.where(t > 0, log_s - torch.where(e > 0, e * d, 0.0).sum(dim=1, keepdim=True) / t, 0.0)
    target = s["target"].unsqueeze(1)
    at = target.clamp(min=0)
    lp = torch.where(f.gather(1, at) == NEG_INF, NEG_INF, d.gather(1, at) - log_s)
    out = {"logp": torch.where(target == IGNORE, 0.0, lp)[:, 0], "entropy": ent[:, 0],
           "stats": torch.cat([m, t], dim=1)}
    if case["top"]:
        idx = _plain_top(f, case["top"])
        out["top_logp"] = torch.where(f.gather(1, idx) == NEG_INF, NEG_INF, d.gather(1, idx) - log_s)
        out["top_idx"] = idx
    return out


def _plain_probs(s):
    m, t = s["stats"][:, :1], s["stats"][:, 1:]
    d = (s["logits"].float() - torch.where(m == NEG_INF, 0.0, m)) / s["case"]["temperature"]
    return d, torch.exp(d) * torch.where(t == 0, 0.0, 1.0 / t), t


def _plain_logp_bwd(s):
    d, p, t = _plain_probs(s)
    keep = s["target"] != IGNORE
    dlogp = torch.where(keep, s["dlogp"], 0.0).unsqueeze(1)
    lp = torch.where(p > 0, d - torch.log(t), 0.0)
    g = -p * (dlogp + s["dentropy"].unsqueeze(1) * (lp + s["entropy"].unsqueeze(1)))
    some = (t > 0).float()  # a row without a token has no gradient
    g = g.scatter_add(1, s["target"].clamp(min=0).unsqueeze(1), dlogp * some)
    return {"dlogits": (g / s["case"]["temperature"]).to(s["logits"].dtype)}


def _plain_teacher(s):
    n = s["logits"].shape[1]
    ids = s["ids"]
    there = (ids >= 0) & (ids < n)
    t = torch.where(there, s["teacher"].float(), NEG_INF)
    m = t.amax(dim=1, keepdim=True)
    d = (t - torch.where(m == NEG_INF, 0.0, m)) / s["case"]["temperature"]
    e = torch.exp(d)
    total = e.sum(dim=1, keepdim=True)
    q = torch.where(total > 0, e / total, 0.0)
    return ids.clamp(0, n - 1), q, d - torch.log(total)


def _plain_kd_loss(s, d, log_s):
    at, q, lq = _plain_teacher(s)
    lp = torch.where(s["logits"].gather(1, at) == NEG_INF, NEG_INF, d.gather(1, at) - log_s)
    return torch.where(q > 0, q * (lq - lp), 0.0).sum(dim=1)


def _plain_kd_grad(s, p):
    at, q, _ = _plain_teacher(s)
    w = s["weight"].unsqueeze(1) / s["case"]["temperature"]
    g = (p * q.sum(dim=1, keepdim=True).gt(0).float()).scatter_add(1, at, -q)
    return (g * w).to(s["logits"].dtype)


def _plain_kd_fwd(s):
    _, m, d, _, t = _plain_rows(s["logits"], s["case"]["temperature"])
    return {"loss": _plain_kd_loss(s, d, torch.log(t)), "stats": torch.cat([m, t], dim=1)}


def _plain_kd_bwd(s):
    _, p, _ = _plain_probs(s)
    return {"dlogits": _plain_kd_grad(s, p)}


def _plain_kd_step(s):
    _, m, d, e, t = _plain_rows(s["logits"], s["case"]["temperature"])
    return {"loss": _plain_kd_loss(s, d, torch.log(t)), "stats": torch.cat([m, t], dim=1),
            "dlogits": _plain_kd_grad(s, e * torch.where(t == 0, 0.0, 1.0 / t))}


PLAIN = {"ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd, "logp_fwd": _plain_logp_fwd,
         "logp_bwd": _plain_logp_bwd, "kd_fwd": _plain_kd_fwd, "kd_bwd": _plain_kd_bwd, "kd_step": _plain_kd_step}


# ---------------------------------------------------------------------- the library's calls
def _own(s):
    import swiglu_ffn_backward_gb300 as swg

    op, case = s["op"], s["case"]
    if op == "ln_fwd":
        return swg.layer_norm_fwd(s["x"], s["gamma"], s["beta"], eps=EPS, residual=s["residual"])
    if op == "ln_bwd":
        dx, dgamma, dbeta = swg.layer_norm_bwd(s["dy"], s["x"], s["stats"], gamma=s["gamma"], dh=s["dh"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    t = case["temperature"]
    if op == "logp_fwd":
        return swg.token_logprobs_fwd(s["logits"], s["target"], top_k=case["top"], temperature=t)
    if op == "logp_bwd":
        return {"dlogits": swg.token_logprobs_bwd(s["dlogp"], s["logits"], s["target"], s["stats"],
                                                  dentropy=s["dentropy"], entropy=s["entropy"], temperature=t)}
    if op == "kd_fwd":
        return swg.distill_fwd(s["logits"], s["ids"], s["teacher"], temperature=t)
    if op == "kd_bwd":
        return {"dlogits": swg.distill_bwd(s["weight"], s["logits"], s["ids"], s["teacher"], s["stats"],
                                           temperature=t)}
    return swg.distill_fwd_bwd(s["logits"], s["ids"], s["teacher"], s["weight"], temperature=t)


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# ------------------------------------------------------------------------------ work, exact
def work(case):
    rows, cols = case["rows"], case["cols"]
    es = 4 if case["dtype"] == "f32" else 2
    n = rows * cols
    op = case["op"]
    if op.startswith("ln"):
        ws = 4 if case["weights"] == "f32" else 2
        # fwd: x (and the residual) in, y (and h) out; bwd: dy, x (and dh) in, dx out
        streams = (2 + 2 * case["add"]) if op == "ln_fwd" else (3 + case["add"])
        params = (2 if op == "ln_fwd" else 3) * cols * ws
        return {"bytes": streams * n * es + params + 8 * rows, "flops": (8 if op == "ln_fwd" else 14) * n}
    if op == "logp_fwd":
        return {"bytes": n * es + rows * (8 + 16 + 12 * case["top"]), "flops": 6 * n}
    if op == "logp_bwd":
        return {"bytes": 2 * n * es + rows * 28, "flops": 9 * n}
    k = min(case["entries"], cols)
    teacher = rows * k * (8 + es)
    if op == "kd_fwd":
        return {"bytes": n * es + teacher + rows * 12, "flops": 4 * n + 8 * rows * k}
    if op == "kd_bwd":
        return {"bytes": 2 * n * es + teacher + rows * 12, "flops": 5 * n + 8 * rows * k}
    return {"bytes": 2 * n * es + teacher + rows * 16, "flops": 7 * n + 16 * rows * k}


def _exact_ln(s):
    case = s["case"]
    x = s["x"].double()
    n = x.shape[1]
    gamma = s["gamma"].double()
    if case["op"] == "ln_fwd":
        out = {}
        if s["residual"] is not None:
            out["h"] = (x + s["residual"].double()).to(s["x"].dtype).double()
            x = out["h"]
        mean = x.mean(dim=1, keepdim=True)
        var = ((x - mean) ** 2).mean(dim=1, keepdim=True)
        rstd = (var + EPS) ** -0.5
        out["y"] = (x - mean) * rstd * gamma + s["beta"].double()
        out["stats"] = torch.cat([mean, rstd], dim=1)
        return out
    mean, rstd = s["stats"].double().unbind(dim=1)
    xh = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1)
    dy = s["dy"].double()
    gdy = dy * gamma
    dx = (gdy - gdy.mean(dim=1, keepdim=True) - xh * (gdy * xh).mean(dim=1, keepdim=True)) * rstd.unsqueeze(1)
    if s["dh"] is not None:
        dx += s["dh"].double()
    return {"dx": dx, "dgamma": torch.einsum("ij,ij->j", dy, xh), "dbeta": dy.sum(dim=0)}


def _exact_rows(s, i, j):
    """The outputs for rows i to j - 1."""
    case, op = s["case"], s["op"]
    T = case["temperature"]
    z = s["logits"][i:j]
    if op in ("logp_bwd", "kd_bwd"):  # the saved statistics are inputs
        m, t = s["stats"][i:j].double().split(1, dim=1)
        d = (z.double() - torch.where(torch.isinf(m), torch.zeros_like(m), m)) / T
        log_s = torch.log(t)
    else:
        m, t, log_s, d = _row_stats64(z, T)
    lp = torch.where(torch.isinf(d), d, d - log_s)
    p = torch.exp(lp)
    out = {} if op in ("logp_bwd", "kd_bwd") else {"stats": torch.cat([m, t], dim=1)}
    row = torch.arange(j - i, device=z.device)
    if op.startswith("logp"):
        target = s["target"][i:j]
        given = target >= 0
        at = target.clamp(min=0)
        if op == "logp_fwd":
            out["logp"] = torch.where(given, lp[row, at], 0.0)
            out["entropy"] = _entropy64(d, t, log_s)[:, 0]
            if case["top"]:
                out["top_logp"] = lp.topk(case["top"], dim=1).values
                out["top_idx"] = None
            return out
        dl = torch.where(given, s["dlogp"][i:j].double(), 0.0)
        g = -dl.unsqueeze(1) * p
        g[row, at] += torch.where(t[:, 0] > 0, dl, 0.0)
        shape = torch.where(p > 0, p * (lp + s["entropy"][i:j].double().unsqueeze(1)), torch.zeros_like(p))
        return {"dlogits": (g - s["dentropy"][i:j].double().unsqueeze(1) * shape) / T}
    ids = s["ids"][i:j]
    there = (ids >= 0) & (ids < z.shape[1])
    tl = torch.where(there, s["teacher"][i:j].double() / T, NEG_INF)
    some = there.any(dim=1, keepdim=True)
    lq = torch.where(some, torch.log_softmax(tl, dim=1), NEG_INF)
    q = torch.exp(lq)
    at = ids.clamp(0, z.shape[1] - 1)
    if op != "kd_bwd":
        out["loss"] = torch.where(q > 0, q * (lq - lp.gather(1, at)), torch.zeros_like(q)).sum(dim=1)
    if op != "kd_fwd":
        g = torch.where(some, p, torch.zeros_like(p))
        g.scatter_add_(1, at, -q)
        out["dlogits"] = g * (s["weight"][i:j].double().unsqueeze(1) / T)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"].startswith("ln"):
        return _exact_ln(s)
    parts = [_exact_rows(s, i, j) for i, j in _chunks(case["rows"], case["cols"])]
    return {k: None if parts[0][k] is None else torch.cat([p[k] for p in parts]) for k in parts[0]}
