"""The calls whose counters block_operators_bf16.md lists: the linear layer and the norms between blocks, each twice, in
bf16. Run from the repository's root."""

import sys

import torch

sys.path.insert(0, ".")
import swiglu_ffn_backward_gb300 as swg  # noqa: E402

g = torch.Generator("cuda")
g.manual_seed(1)


def rn(*shape, scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).bfloat16()


K, N = 14336, 4096
w, wu, ws = rn(K, N, scale=K ** -0.5), rn(N, K, scale=N ** -0.5), rn(512, 1024, scale=512 ** -0.5)
x1, r1 = rn(1, K), rn(1, N)
xl, rl, dyl = rn(2048, K), rn(2048, N), rn(2048, N)
xs, zs, dys = rn(65536, 512), rn(65536, 1024), rn(65536, 1024)
u, r, dy, dh = (rn(16384, 4096) for _ in range(4))
gate = rn(8, 4096)
gp, gn = (1 + rn(4096, scale=0.2).float() for _ in range(2))
uo, ro = rn(4000, 4001), rn(4000, 4001)
go = 1 + rn(4001, scale=0.2).float()
for _ in range(2):
    swg.linear_fwd(x1, w, residual=r1)
    swg.linear_fwd(rn(77, N), wu, act="gelu")
    swg.linear_fwd(xl, w, residual=rl)
    swg.linear_bwd(dyl, xl, w, bias=False)
    swg.linear_fwd(xs, ws, act="gelu", save_z=True)
    swg.linear_bwd(dys, xs, ws, z=zs, act="gelu")
    o = swg.block_norm_fwd(u, r, gamma_post=gp, gamma_pre=gn, gate=gate)
    swg.block_norm_bwd(dy, dh, u, o["h"], o["stats"], gamma_post=gp, gamma_pre=gn, gate=gate)
    o = swg.block_norm_fwd(uo, ro, gamma_post=go, gamma_pre=go)
    swg.block_norm_bwd(uo, ro, uo, o["h"], o["stats"], gamma_post=go, gamma_pre=go)
torch.cuda.synchronize()
swg.swg_check()
print("ok")
