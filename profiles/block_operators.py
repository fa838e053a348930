"""The calls whose counters block_operators_bf16.md lists: the linear layer and the norms between blocks in bf16, one operator a
run, called twice. From the repository's root: python profiles/block_operators.py NAME."""

import sys

import torch

sys.path.insert(0, ".")
import swiglu_ffn_backward_gb300 as swg  # noqa: E402

g = torch.Generator("cuda")
g.manual_seed(1)


def rn(*shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()


def one_token():
    x, w, r = rn(1, 14336), rn(14336, 4096, scale=14336 ** -0.5), rn(1, 4096)
    return lambda: swg.linear_fwd(x, w, residual=r)


def some_tokens():
    x, w = rn(77, 4096), rn(4096, 14336, scale=4096 ** -0.5)
    return lambda: swg.linear_fwd(x, w, act="gelu")


def large():
    x, w, r = rn(2048, 14336), rn(14336, 4096, scale=14336 ** -0.5), rn(2048, 4096)
    return lambda: swg.linear_fwd(x, w, residual=r)


def large_dw():
    x, dy = rn(2048, 14336), rn(2048, 4096)
    return lambda: swg.linear_bwd(dy, x, None, bias=False, need_dx=False)


def large_dx():
    w, dy = rn(14336, 4096, scale=14336 ** -0.5), rn(2048, 4096)
    return lambda: swg.linear_bwd(dy, None, w, bias=False, need_dw=False)


def short():
    x, w = rn(65536, 512), rn(512, 1024, scale=512 ** -0.5)
    return lambda: swg.linear_fwd(x, w, act="gelu", save_z=True)


def short_backward():
    x, w, z, dy = rn(65536, 512), rn(512, 1024, scale=512 ** -0.5), rn(65536, 1024), rn(65536, 1024)
    return lambda: swg.linear_bwd(dy, x, w, z=z, act="gelu")


def norms(backward, rows, cols, gates):
    u, r, dy, dh = (rn(rows, cols) for _ in range(4))
    kw = dict(gamma_post=1 + rn(cols, scale=0.2).float(), gamma_pre=1 + rn(cols, scale=0.2).float(),
              gate=rn(gates, cols) if gates else None)
    if not backward:
        return lambda: swg.block_norm_fwd(u, r, **kw)
    o = swg.block_norm_fwd(u, r, **kw)
    return lambda: swg.block_norm_bwd(dy, dh, u, o["h"], o["stats"], **kw)


CALLS = {"one_token": one_token, "some_tokens": some_tokens, "large": large, "large_dw": large_dw, "large_dx": large_dx,
         "short": short, "short_backward": short_backward,
         "norms": lambda: norms(False, 16384, 4096, 8), "norms_backward": lambda: norms(True, 16384, 4096, 8),
         "ragged": lambda: norms(False, 4000, 4001, 0), "ragged_backward": lambda: norms(True, 4000, 4001, 0)}

call = CALLS[sys.argv[1]]()
for _ in range(2):
    call()
torch.cuda.synchronize()
swg.swg_check()
print("ok")
