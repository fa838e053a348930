"""Argument checks of layer norm, token log probabilities and distillation at the C ABI
(fake, never-dereferenced addresses: every case returns before any CUDA call)."""

import pytest

FAKE = 0x7f0000000000
STEP = 0x10000000


@pytest.fixture(scope="module")
def b():
    from swiglu_ffn_backward_gb300 import _binding
    return _binding


def _p(n):
    return [FAKE + i * STEP for i in range(n)]


def _with(args, **at):
    args = list(args)
    for i, v in at.items():
        args[int(i[1:])] = v
    return args


def test_layer_norm_fwd(b):
    f = b.lib.layer_norm_fwd  # x, residual, gamma, beta, h, y, stats, M, N, ldx, ldr, eps, dtype, wdtype, stream
    ok = _p(7) + [4, 16, 16, 16, 1e-5, b.SWG_BF16, b.SWG_F32, None]
    bad = b.SWG_ERR_PARAM_INVALID
    for change in (dict(a7=-1), dict(a8=-1), dict(a9=15), dict(a9=-16), dict(a10=8), dict(a11=-1.0),
                   dict(a11=float("nan")), dict(a12=3), dict(a13=b.SWG_F16), dict(a1=None), dict(a4=None),
                   dict(a5=FAKE + 8), dict(a6=FAKE + 5 * STEP + 64), dict(a4=FAKE + STEP)):
        assert f(*_with(ok, **change)) == bad, change
    for i in (0, 5, 6):
        assert f(*_with(ok, **{f"a{i}": None})) == b.SWG_ERR_NULLPTR
    for change in (dict(a0=FAKE + 1), dict(a2=FAKE + 2 * STEP + 2), dict(a7=2 ** 31), dict(a8=2 ** 31, a9=2 ** 31, a10=2 ** 31),
                   dict(a9=2 ** 50), dict(a7=2 ** 30, a8=2 ** 30, a9=2 ** 30, a10=2 ** 30)):
        assert f(*_with(ok, **change)) == b.SWG_ERR_UNSUPPORTED, change
    assert f(*([None] * 7), 0, 16, 16, 16, 1e-5, b.SWG_F32, b.SWG_F32, None) == b.SWG_OK
    assert f(*([None] * 7), 5, 0, 0, 0, 1e-5, b.SWG_F32, b.SWG_F32, None) == b.SWG_OK


def test_layer_norm_bwd(b):
    f = b.lib.layer_norm_bwd  # dy x stats gamma dh dx dgamma dbeta M N lddy ldx lddh dtype wdtype ws bytes stream
    need = b.lib.layer_norm_bwd_workspace_size(4, 16)
    assert need > 0 and b.lib.layer_norm_bwd_workspace_size(0, 16) == 0 and b.lib.layer_norm_bwd_workspace_size(4, -1) == 0
    ok = _p(8) + [4, 16, 16, 16, 16, b.SWG_F16, b.SWG_F16, FAKE + 9 * STEP, need, None]
    for change in (dict(a8=-1), dict(a9=-1), dict(a10=3), dict(a11=3), dict(a12=3), dict(a13=9), dict(a14=b.SWG_BF16),
                   dict(a5=FAKE + 32), dict(a6=FAKE + 7 * STEP + 2), dict(a15=FAKE + 5 * STEP)):
        assert f(*_with(ok, **change)) == b.SWG_ERR_PARAM_INVALID, change
    for i in (0, 1, 2, 5):
        assert f(*_with(ok, **{f"a{i}": None})) == b.SWG_ERR_NULLPTR
    for change in (dict(a15=None), dict(a16=need - 1), dict(a15=FAKE + 9 * STEP + 8)):
        assert f(*_with(ok, **change)) == b.SWG_ERR_WORKSPACE, change
    assert f(*_with(ok, a3=FAKE + 3 * STEP + 1)) == b.SWG_ERR_UNSUPPORTED
    assert f(*([None] * 8), 0, 16, 0, 0, 0, b.SWG_F32, b.SWG_F32, None, 0, None) == b.SWG_OK


def test_token_logprobs_fwd(b):
    f = b.lib.token_logprobs_fwd  # logits targets logp entropy stats top_logp top_idx T V ld k tau ignore dtype itype stream
    ok = _p(7) + [4, 100, 100, 5, 1.0, -100, b.SWG_BF16, 1, None]
    for change in (dict(a7=-1), dict(a8=0), dict(a9=99), dict(a10=-1), dict(a10=33), dict(a8=4, a9=4), dict(a11=0.0),
                   dict(a11=-2.0), dict(a11=float("nan")), dict(a11=float("inf")), dict(a11=1e-45), dict(a13=3),
                   dict(a14=2), dict(a3=FAKE), dict(a4=FAKE + 3 * STEP + 8), dict(a6=FAKE + 5 * STEP)):
        assert f(*_with(ok, **change)) == b.SWG_ERR_PARAM_INVALID, change
    for i in (0, 2, 3, 4, 5, 6):
        assert f(*_with(ok, **{f"a{i}": None})) == b.SWG_ERR_NULLPTR, i
    for change in (dict(a0=FAKE + 1), dict(a1=FAKE + STEP + 4), dict(a3=FAKE + 3 * STEP + 2), dict(a8=2 ** 31, a9=2 ** 31),
                   dict(a7=2 ** 31), dict(a9=2 ** 41)):
        assert f(*_with(ok, **change)) == b.SWG_ERR_UNSUPPORTED, change
    assert f(*([None] * 7), 0, 100, 100, 5, 1.0, -100, b.SWG_F32, 0, None) == b.SWG_OK


def test_token_logprobs_bwd(b):
    f = b.lib.token_logprobs_bwd  # dlogp logits targets stats dentropy entropy dlogits T V ld ldo tau ignore dtype itype stream
    ok = _p(7) + [4, 100, 100, 100, 1.0, -100, b.SWG_F32, 0, None]
    for change in (dict(a7=-1), dict(a8=0), dict(a9=1), dict(a10=99), dict(a10=0), dict(a11=0.0), dict(a13=5), dict(a14=5),
                   dict(a6=FAKE + STEP + 400), dict(a6=FAKE + STEP, a10=104), dict(a6=FAKE + 2 * STEP)):
        assert f(*_with(ok, **change)) == b.SWG_ERR_PARAM_INVALID, change
    for i in (0, 1, 3, 5, 6):
        assert f(*_with(ok, **{f"a{i}": None})) == b.SWG_ERR_NULLPTR, i
    for change in (dict(a6=FAKE + 6 * STEP + 2), dict(a10=2 ** 41), dict(a0=FAKE + 1)):
        assert f(*_with(ok, **change)) == b.SWG_ERR_UNSUPPORTED, change


@pytest.mark.parametrize("name", ["distill_fwd", "distill_bwd", "distill_fwd_bwd"])
def test_distill(b, name):
    f = getattr(b.lib, name)
    tail = [1.0, b.SWG_F32, b.SWG_F16, 1, None]
    if name == "distill_fwd":       # logits ids teacher loss stats T V ld K
        ok, required, T, K, ld, out, z = _p(5) + [4, 100, 100, 8] + tail, (0, 1, 2, 3, 4), 5, 8, 7, 3, 0
    elif name == "distill_bwd":     # weight logits ids teacher stats dlogits T V ld ldo K
        ok, required, T, K, ld, out, z = _p(6) + [4, 100, 100, 100, 8] + tail, range(6), 6, 10, 8, 5, 1
    else:                           # logits ids teacher weight loss stats dlogits T V ld ldo K
        ok, required, T, K, ld, out, z = _p(7) + [4, 100, 100, 100, 8] + tail, range(7), 7, 11, 9, 6, 0
    for i in required:
        assert f(*_with(ok, **{f"a{i}": None})) == b.SWG_ERR_NULLPTR, i
    for i, v in ((T, -1), (T + 1, 0), (ld, 50), (K, 0), (K + 1, 0.0), (K + 2, 7), (K + 3, 7), (K + 4, 7),
                 (out, ok[z] + 40)):
        assert f(*_with(ok, **{f"a{i}": v})) == b.SWG_ERR_PARAM_INVALID, (i, v)
    for i, v in ((K, 1025), (T, 2 ** 31), (z, ok[z] + 2), (z + 1, ok[z + 1] + 4), (z + 2, ok[z + 2] + 1)):
        assert f(*_with(ok, **{f"a{i}": v})) == b.SWG_ERR_UNSUPPORTED, (i, v)
    assert f(*_with(ok, **{f"a{T}": 0})) == b.SWG_OK


def test_binding_requires_cuda_tensors(b):
    import torch
    t = torch.zeros(4, 8)
    i = torch.zeros((4, 2), dtype=torch.int64)
    for call in (lambda: b.layer_norm_fwd(t), lambda: b.layer_norm_bwd(t, t, t), lambda: b.token_logprobs_fwd(t),
                 lambda: b.token_logprobs_bwd(t, t, i, t), lambda: b.distill_fwd(t, i, t),
                 lambda: b.distill_bwd(t, t, i, t, t), lambda: b.distill_fwd_bwd(t, i, t, t)):
        with pytest.raises(TypeError):
            call()
