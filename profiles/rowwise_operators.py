"""The calls whose counters rowwise_operators_bf16.md lists: each row-wise operator twice, weights bf16, logits N(0, 2.5),
random ids. Run from the repository's root."""

import sys

import torch

sys.path.insert(0, ".")
import swiglu_ffn_backward_gb300 as swg  # noqa: E402

g = torch.Generator("cuda")
g.manual_seed(1)


def rn(*shape):
    return torch.randn(shape, generator=g, device="cuda")


M, N = 16384, 4096
x, r, dy = rn(M, N).bfloat16(), rn(M, N).bfloat16(), rn(M, N).bfloat16()
gamma = (1 + 0.1 * rn(N)).bfloat16()
beta = gamma.clone()
xr, dyr = rn(4000, 4001).bfloat16(), rn(4000, 4001).bfloat16()
T, V, K = 1024, 131072, 64
z = (rn(T, V) * 2.5).bfloat16()
t = torch.randint(0, V, (T,), generator=g, device="cuda")
ids = torch.randint(0, V, (T, K), generator=g, device="cuda")
tl, w, dz = rn(T, K), torch.rand(T, generator=g, device="cuda"), torch.empty_like(z)
T2, V2 = 4096, 32768
z2 = (rn(T2, V2) * 2.5).bfloat16()
t2 = torch.randint(0, V2, (T2,), generator=g, device="cuda")
ids2, tl2, w2 = ids.remainder(V2).repeat(4, 1), tl.repeat(4, 1), w.repeat(4)
for _ in range(2):
    o = swg.layer_norm_fwd(x, gamma, beta, residual=r)
    swg.layer_norm_bwd(dy, o["h"], o["stats"], gamma=gamma, dh=r)
    o = swg.layer_norm_fwd(xr)
    swg.layer_norm_bwd(dyr, xr, o["stats"])
    o = swg.token_logprobs_fwd(z, t, top_k=20)
    swg.token_logprobs_bwd(w, z, t, o["stats"], dentropy=w, entropy=o["entropy"], dlogits=dz)
    swg.token_logprobs_fwd(z2, t2, top_k=20)
    s = swg.distill_fwd(z, ids, tl)["stats"]
    swg.distill_bwd(w, z, ids, tl, s, dlogits=dz)
    swg.distill_fwd_bwd(z, ids, tl, w, out={"dlogits": dz})
    s = swg.distill_fwd(z2, ids2, tl2)["stats"]
    swg.distill_fwd_bwd(z2, ids2, tl2, w2)
torch.cuda.synchronize()
swg.swg_check()
print("ok")
