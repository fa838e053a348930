"""The timeout path of the row-wise kernels' bounded waits.

The kernels that stream rows through shared memory, and those whose clusters share a row, wait for one another's
arrivals. A wait that runs out makes its thread silent: it arrives nowhere and sends nothing any more, later waits
only look once, and the block goes on to its end, where it waits for what was sent to it. The fault is made on the
host: swg_inject_stall arms the next launch of one kernel so that the last producer of each cluster stops issuing
copies before a ring entry (or the last block sends no sums from a row on) and its waits give up after about half a
millisecond. The tests check the status, that nothing outside the outputs was written, and that the same call is right
afterwards."""

import pytest
import torch

import oracle

from ._guard import check_all, guarded, workspace
from ._row_ops import EXP, SUM, check, f64

LIMIT = 1 << 20  # cycles, about half a millisecond
BF16, F32, F16 = torch.bfloat16, torch.float32, torch.float16


def _swg():
    import swiglu_ffn_backward_gb300 as swg
    return swg


def test_row_kernels_can_be_armed():
    from swiglu_ffn_backward_gb300 import _binding as b
    for kernel in (b.SWG_INJECT_LAYER_NORM_FWD, b.SWG_INJECT_LAYER_NORM_BWD, b.SWG_INJECT_TOKEN_LOGPROBS,
                   b.SWG_INJECT_DISTILL):
        assert b.lib.swg_inject_stall(kernel, 3, LIMIT) == b.SWG_OK
        assert b.lib.swg_inject_stall(kernel, -1, LIMIT) == b.SWG_ERR_PARAM_INVALID
    assert b.lib.swg_inject_stall(0, 0, 0) == b.SWG_OK
    for kernel in (15, 20):
        assert b.lib.swg_inject_stall(kernel, 1, LIMIT) == b.SWG_ERR_PARAM_INVALID


def _expect_timeout(swg):
    with pytest.raises(swg.SwgError) as e:
        swg.swg_check()
    assert e.value.status == 6  # SWG_ERR_TIMEOUT
    swg.swg_check()  # the status word was cleared


def _logits(T, V, dtype):
    return torch.randn((T, V), generator=torch.Generator("cuda").manual_seed(51), device="cuda").to(dtype)


def _check_sums(z, out):
    m, s, _, _ = oracle.row_softmax(f64(z), 1.0)
    check("max", out["stats"][:, 0], m, F32, 0.0)
    check("sum", out["stats"][:, 1], s, F32, (SUM + EXP + 2.0 ** -22 * 8) * s)


# many rows by blocks of four warps, by blocks of 16, and rows that two to eight blocks share
@pytest.mark.gpu
@pytest.mark.parametrize("T,V,dtype,entry", [(2400, 4096, BF16, 0), (2400, 4096, BF16, 1), (2400, 4096, BF16, 3),
                                             (320, 50001, F16, 0), (320, 50001, F16, 6), (40, 40000, BF16, 0),
                                             (1, 131072, F32, 0), (1, 131072, F32, 1)],
                         ids=lambda v: str(v).replace("torch.", ""))
def test_log_probabilities_wait_runs_out(T, V, dtype, entry):
    swg = _swg()
    z = _logits(T, V, dtype)
    t = torch.arange(T, device="cuda") % V
    gs = dict(logp=guarded((T,), F32), entropy=guarded((T,), F32), stats=guarded((T, 2), F32),
              top_logp=guarded((T, 20), F32), top_idx=guarded((T, 20), torch.int64))
    swg.swg_inject_stall(swg.SWG_INJECT_TOKEN_LOGPROBS, entry, LIMIT)
    swg.token_logprobs_fwd(z, t, top_k=20, out={k: g.t for k, g in gs.items()})
    _expect_timeout(swg)
    check_all(gs)
    out = swg.token_logprobs_fwd(z, t, top_k=20)
    swg.swg_check()
    _check_sums(z, out)
    assert torch.equal(z.gather(1, out["top_idx"][:, :1])[:, 0], z.max(dim=1).values)


@pytest.mark.gpu
@pytest.mark.parametrize("entry", [0, 1, 2, 5])
@pytest.mark.parametrize("step", [False, True], ids=["loss", "step"])
@pytest.mark.parametrize("T,V,K,dtype", [(2400, 4096, 20, BF16), (900, 12000, 64, BF16), (800, 50001, 200, BF16),
                                         (60, 131072, 64, BF16), (3, 131072, 700, F32)],
                         ids=lambda v: str(v).replace("torch.", ""))
def test_distillation_wait_runs_out(T, V, K, dtype, step, entry):
    if V == 131072:  # a row or two a block
        entry = min(entry, 1)
    swg = _swg()
    z = _logits(T, V, dtype)
    ids = (torch.arange(T, device="cuda").unsqueeze(1) * 31 + torch.arange(K, device="cuda") * 17) % V
    tl = torch.randn((T, K), generator=torch.Generator("cuda").manual_seed(52), device="cuda")
    w = torch.ones(T, device="cuda")
    gs = dict(loss=guarded((T,), F32), stats=guarded((T, 2), F32))
    if step:
        gs["dlogits"] = guarded((T, V), dtype)
    out = {k: g.t for k, g in gs.items()}
    call = (lambda out: swg.distill_fwd_bwd(z, ids, tl, w, out=out)) if step else (
        lambda out: swg.distill_fwd(z, ids, tl, out=out))
    before = z.clone()
    swg.swg_inject_stall(swg.SWG_INJECT_DISTILL, entry, LIMIT)
    call(out)
    _expect_timeout(swg)
    check_all(gs)
    assert torch.equal(z, before)
    out = call(out)
    swg.swg_check()
    check_all(gs)
    _check_sums(z, out)
    if step:
        rows = [0, T // 2, T - 1]
        ref = oracle.distill_bwd(f64(w[rows]), f64(z[rows]), f64(ids[rows]).astype(int), f64(tl[rows]), 1.0)
        got = f64(out["dlogits"][rows])
        assert abs(got - ref).max() <= 2.0 ** -8 * abs(ref).max() + 2.0 ** -16


# rows shared by two to eight blocks: whole vectors and ragged, one row a cluster and many
@pytest.mark.gpu
@pytest.mark.parametrize("row", [0, 7, 333])
@pytest.mark.parametrize("M,N,dtype", [(500, 12288, BF16), (400, 9001, BF16), (900, 5000, F32), (400, 32768, F32)],
                         ids=lambda v: str(v).replace("torch.", ""))
def test_layer_norm_wait_runs_out(M, N, dtype, row):
    swg = _swg()
    g = torch.Generator("cuda").manual_seed(53)
    x, dy = (torch.randn((M, N), generator=g, device="cuda").to(dtype) for _ in range(2))
    gamma = 1 + 0.2 * torch.randn(N, generator=g, device="cuda")
    want = swg.layer_norm_fwd(x, gamma)
    wantb = swg.layer_norm_bwd(dy, x, want["stats"], gamma=gamma)
    swg.swg_check()
    gs = dict(y=guarded((M, N), dtype), stats=guarded((M, 2), F32), dx=guarded((M, N), dtype), dgamma=guarded((N,), F32),
              dbeta=guarded((N,), F32), ws=workspace(swg.layer_norm_bwd_workspace_size(M, N)))
    outs = {k: gs[k].t for k in ("y", "stats")}
    swg.swg_inject_stall(swg.SWG_INJECT_LAYER_NORM_FWD, row, LIMIT)
    swg.layer_norm_fwd(x, gamma, out=outs)
    _expect_timeout(swg)
    check_all(gs)
    out = swg.layer_norm_fwd(x, gamma, out=outs)
    swg.swg_check()
    assert all(torch.equal(out[k], want[k]) for k in want)
    grads = dict(dx=gs["dx"].t, dgamma=gs["dgamma"].t, dbeta=gs["dbeta"].t, workspace=gs["ws"].t)
    swg.swg_inject_stall(swg.SWG_INJECT_LAYER_NORM_BWD, row, LIMIT)
    swg.layer_norm_bwd(dy, x, want["stats"], gamma=gamma, **grads)
    _expect_timeout(swg)
    check_all(gs)
    got = swg.layer_norm_bwd(dy, x, want["stats"], gamma=gamma, **grads)
    swg.swg_check()
    check_all(gs)
    assert all(torch.equal(a, b) for a, b in zip(got, wantb))
