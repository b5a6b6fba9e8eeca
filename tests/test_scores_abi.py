"""Host-side argument checks of the scoring and distillation calls: refused before any CUDA
work (no GPU needed), by the C entry points and by the torch wrappers."""
import pytest
import torch

import sparse_teacher_kl_gb300 as kd
from sparse_teacher_kl_gb300 import _abi
from sparse_teacher_kl_gb300.build import build_library

P = 1 << 20   # fake, 256-byte aligned device addresses, never dereferenced on these paths
Q = 1 << 40   # far from P: a gradient that does not overlap the logits


@pytest.fixture(scope="module")
def lib():
    build_library()
    return _abi.load()


def _logprobs_fwd(lib, **kw):
    a = dict(z=P, dt=0, N=4, V=256, ld=256, tok=P, M=2, mask=None, tau=1.0, top=5, logp=P, lse=P, ent=P, ids=P,
             tlp=P, ws=P, wsb=4096)
    a.update(kw)
    return lib.kd_token_logprobs_fwd(a["z"], a["dt"], a["N"], a["V"], a["ld"], a["tok"], a["M"], a["mask"], a["tau"],
                                     a["top"], a["logp"], a["lse"], a["ent"], a["ids"], a["tlp"], a["ws"], a["wsb"],
                                     None)


DENSE = [dict(z=None), dict(z=P + 1), dict(dt=3), dict(dt=-1), dict(N=0), dict(N=1 << 31), dict(V=0),
         dict(V=(1 << 30) + 1, ld=1 << 31), dict(ld=255), dict(tau=0.0), dict(tau=-1.0), dict(tau=float("nan")),
         dict(tau=float("inf")), dict(dt=2, z=P + 2)]


@pytest.mark.parametrize("kw", DENSE + [
    dict(tok=None), dict(M=0), dict(M=1025), dict(top=-1), dict(top=129), dict(V=4, ld=4, top=5), dict(logp=None),
    dict(lse=None), dict(ent=P + 2), dict(ids=None), dict(tlp=None), dict(top=0), dict(logp=P + 1)])
def test_logprobs_forward_refuses(lib, kw):
    assert _logprobs_fwd(lib, **kw) == _abi.KD_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(ws=None), dict(ws=P + 16), dict(wsb=100)])
def test_logprobs_refuse_a_bad_workspace(lib, kw):
    assert _logprobs_fwd(lib, **kw) == _abi.KD_ERR_WORKSPACE


def _logprobs_bwd(lib, **kw):
    a = dict(z=P, dt=0, N=4, V=256, ld=256, tok=P, M=2, mask=None, tau=1.0, lse=P, ent=P, gl=P, ge=P, dz=Q, ldg=256,
             ws=P, wsb=4096)
    a.update(kw)
    return lib.kd_token_logprobs_bwd(a["z"], a["dt"], a["N"], a["V"], a["ld"], a["tok"], a["M"], a["mask"], a["tau"],
                                     a["lse"], a["ent"], a["gl"], a["ge"], a["dz"], a["ldg"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw", DENSE + [
    dict(tok=None), dict(M=0), dict(lse=None), dict(gl=None), dict(ent=None), dict(dz=None), dict(dz=Q + 1),
    dict(ldg=255), dict(dz=P, ldg=300, ld=256), dict(dz=P + 512), dict(dz=P - 512)])
def test_logprobs_backward_refuses(lib, kw):
    assert _logprobs_bwd(lib, **kw) == _abi.KD_ERR_INVALID_ARG


def _kl(lib, which, **kw):
    a = dict(z=P, dt=0, N=4, V=256, ld=256, ids=P, t=P, K=8, tl=None, mask=None, tau=1.0, stats=P, g=P, loss=P, kl=None,
             dz=Q, ldg=256, ws=P, wsb=4096)
    a.update(kw)
    head = (a["z"], a["dt"], a["N"], a["V"], a["ld"], a["ids"], a["t"], a["K"], a["tl"], a["mask"], a["tau"])
    tail = (a["ws"], a["wsb"], None)
    if which == "fwd":
        return lib.kd_logits_kl_fwd(*head, a["loss"], a["stats"], a["kl"], *tail)
    if which == "bwd":
        return lib.kd_logits_kl_bwd(*head, a["stats"], a["g"], a["dz"], a["ldg"], *tail)
    return lib.kd_logits_kl_step(*head, a["g"], a["loss"], a["kl"], a["dz"], a["ldg"], *tail)


TEACHER = DENSE + [dict(ids=None), dict(t=None), dict(K=0), dict(K=1025, V=4096, ld=4096), dict(K=257),
                   dict(tl=P + 1), dict(ids=P + 2)]


@pytest.mark.parametrize("which,kw", [(w, k) for w in ("fwd", "bwd", "step") for k in TEACHER]
                         + [("fwd", k) for k in (dict(loss=None), dict(stats=None), dict(stats=P + 4), dict(kl=P + 1))]
                         + [("bwd", k) for k in (dict(stats=None), dict(g=None), dict(dz=None), dict(dz=P + 64))]
                         + [("step", k) for k in (dict(loss=None), dict(g=None), dict(dz=None), dict(ldg=9))])
def test_logits_kl_refuses(lib, which, kw):
    assert _kl(lib, which, **kw) == _abi.KD_ERR_INVALID_ARG


@pytest.mark.parametrize("which", ["fwd", "bwd", "step"])
def test_logits_kl_refuses_workspace_and_width(lib, which):
    assert _kl(lib, which, wsb=256) == _abi.KD_ERR_WORKSPACE
    assert _kl(lib, which, ws=None) == _abi.KD_ERR_WORKSPACE
    assert _kl(lib, which, V=1 << 24, ld=1 << 24) == _abi.KD_ERR_UNSUPPORTED


def test_wrappers_refuse_wrong_tensors():
    z = torch.zeros((2, 8))
    tok = torch.zeros((2,), dtype=torch.int32)
    with pytest.raises(ValueError):
        kd.token_logprobs_forward(z, tok)                 # not a CUDA tensor
    with pytest.raises(ValueError):
        kd.logits_kl_forward(z, tok[:, None], z[:, :1])
    with pytest.raises(ValueError):
        kd.logits_kl_step(z.double(), tok[:, None], z[:, :1])


def _fused(lib, backward, **kw):
    a = dict(H=P, W=P, tok=P, mask=None, N=256, d=64, V=1000, chunk=128, tau=1.0, logp=P, lse=P, ent=P, gl=P, ge=P,
             gH=P, f32=0, gW=P, kind=0, ws=P, wsb=1 << 30)
    a.update(kw)
    head = (a["H"], a["W"], a["tok"], a["mask"], a["N"], a["d"], a["V"], a["chunk"], a["tau"])
    if backward:
        return lib.kd_fused_logprobs_bwd(*head, a["lse"], a["ent"], a["gl"], a["ge"], a["gH"], a["f32"], a["gW"],
                                         a["kind"], a["ws"], a["wsb"], None)
    return lib.kd_fused_logprobs_fwd(*head, a["logp"], a["lse"], a["ent"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("backward,kw", [(b, k) for b in (False, True) for k in (
    dict(N=0), dict(d=0), dict(d=60), dict(V=0), dict(chunk=100), dict(chunk=0), dict(tau=0.0), dict(tau=float("nan")),
    dict(H=None), dict(W=None), dict(H=P + 8), dict(tok=None), dict(tok=P + 1), dict(lse=None), dict(lse=P + 2))]
    + [(False, k) for k in (dict(logp=None), dict(logp=P + 1), dict(ent=P + 2))]
    + [(True, k) for k in (dict(gl=None), dict(ent=None), dict(gH=None), dict(gW=None), dict(gH=P + 4), dict(gW=P + 8),
                           dict(ge=P + 2), dict(kind=3), dict(kind=-1), dict(kind=2, N=129))])
def test_fused_logprobs_refuse(lib, backward, kw):
    assert _fused(lib, backward, **kw) == _abi.KD_ERR_INVALID_ARG


@pytest.mark.parametrize("backward", [False, True])
def test_fused_logprobs_refuse_a_bad_workspace(lib, backward):
    need = lib.kd_fused_logprobs_workspace(256, 64, 1000, 128, int(backward))
    assert _fused(lib, backward, wsb=need - 1) == _abi.KD_ERR_WORKSPACE
    assert _fused(lib, backward, ws=None) == _abi.KD_ERR_WORKSPACE
    assert _fused(lib, backward, ws=P + 64) == _abi.KD_ERR_WORKSPACE
    assert lib.kd_fused_logprobs_workspace(0, 64, 1000, 128, 1) == 0


def test_workspace_clear_refuses(lib):
    assert lib.kd_workspace_clear(None, 4096, None) == _abi.KD_ERR_WORKSPACE
    assert lib.kd_workspace_clear(P + 64, 4096, None) == _abi.KD_ERR_WORKSPACE
    assert lib.kd_workspace_clear(P, 255, None) == _abi.KD_ERR_WORKSPACE
