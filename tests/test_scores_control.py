"""The calls that report to a control block of the caller's: argument checks (no GPU needed)."""
import pytest
import torch

import sparse_teacher_kl_gb300 as kd
from sparse_teacher_kl_gb300 import _abi
from sparse_teacher_kl_gb300.build import build_library

P, Q = 1 << 20, 1 << 40   # fake, 256-byte aligned device addresses, never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    build_library()
    return _abi.load()


def call(lib, which, control=P, **kw):
    a = dict(K=8, ws=P, wsb=1 << 30, tau=1.0)
    a.update(kw)
    kl = (P, 0, 4, 256, 256, P, P, a["K"], None, None, a["tau"])
    fused = (P, P, P, None, 256, 64, 1000, 128, a["tau"])
    end = (a["ws"], a["wsb"], control, None)
    if which == "kl_fwd":
        return lib.kd_logits_kl_fwd_ctl(*kl, P, P, None, *end)
    if which == "kl_bwd":
        return lib.kd_logits_kl_bwd_ctl(*kl, P, P, Q, 256, *end)
    if which == "kl_step":
        return lib.kd_logits_kl_step_ctl(*kl, P, P, None, Q, 256, *end)
    if which == "fused_fwd":
        return lib.kd_fused_logprobs_fwd_ctl(*fused, P, P, None, *end)
    return lib.kd_fused_logprobs_bwd_ctl(*fused, P, P, P, P, P, 0, P, 0, *end)


CALLS = ["kl_fwd", "kl_bwd", "kl_step", "fused_fwd", "fused_bwd"]


@pytest.mark.parametrize("which", CALLS)
def test_control_blocks_are_checked(lib, which):
    assert call(lib, which, None) == _abi.KD_ERR_WORKSPACE
    assert call(lib, which, P + 128) == _abi.KD_ERR_WORKSPACE
    assert call(lib, which, ws=None) == _abi.KD_ERR_WORKSPACE
    assert call(lib, which, wsb=256) == _abi.KD_ERR_WORKSPACE
    assert call(lib, which, tau=0.0) == _abi.KD_ERR_INVALID_ARG


@pytest.mark.parametrize("call", [
    lambda z, t: kd.token_logprobs(z, t), lambda z, t: kd.logits_kl(z, t[:, None], z[:, :1]),
    lambda z, t: kd.fused_logprobs(z, z, t), lambda z, t: kd.logits_kl_step(z, t[:, None], z[:, :1])])
def test_differentiable_calls_refuse_host_tensors(call):
    with pytest.raises(ValueError):
        call(torch.zeros((2, 8)), torch.zeros((2,), dtype=torch.int32))
