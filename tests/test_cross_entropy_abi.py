"""Host-side argument checks of the cross entropy: refused before any CUDA work (no GPU needed)."""
import pytest
import torch

import sparse_teacher_kl_gb300 as kd
from sparse_teacher_kl_gb300 import _abi
from sparse_teacher_kl_gb300.build import build_library

P = 1 << 20   # fake, 256-byte aligned device address, never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    build_library()
    return _abi.load()


def call(lib, step, **kw):
    a = dict(H=P, W=P, y=P, mask=None, N=256, d=64, V=1000, chunk=128, smooth=0.0, z=0.0, cap=0.0, ignore=-100, g=None,
             loss=P, lse=P, each=None, gH=P, f32=0, gW=P, kind=0, ws=P, wsb=1 << 30, ctl=P)
    a.update(kw)
    head = (a["H"], a["W"], a["y"], a["mask"], a["N"], a["d"], a["V"], a["chunk"], a["smooth"], a["z"], a["cap"],
            a["ignore"])
    tail = (a["ws"], a["wsb"], a["ctl"], None)
    if step:
        return lib.kd_fused_cross_entropy_step(*head, a["g"], a["loss"], a["lse"], a["each"], a["gH"], a["f32"], a["gW"],
                                               a["kind"], *tail)
    return lib.kd_fused_cross_entropy_fwd(*head, a["loss"], a["lse"], a["each"], *tail)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("step,kw", [(s, k) for s in (False, True) for k in (
    dict(N=0), dict(N=1 << 31), dict(d=0), dict(d=60), dict(V=0), dict(V=1 << 31), dict(chunk=0), dict(chunk=100),
    dict(H=None), dict(W=None), dict(H=P + 8), dict(W=P + 2), dict(y=None), dict(y=P + 1), dict(loss=None),
    dict(loss=P + 2), dict(lse=None), dict(lse=P + 1), dict(each=P + 2), dict(smooth=-0.1), dict(smooth=1.0),
    dict(smooth=NAN), dict(z=-1.0), dict(z=INF), dict(z=NAN), dict(cap=-1.0), dict(cap=INF), dict(cap=NAN), dict(cap=1e-30), dict(cap=9e-7))]
    + [(True, k) for k in (dict(g=P + 1), dict(gH=None), dict(gH=P + 8), dict(gW=None), dict(gW=P + 4), dict(kind=3),
                           dict(kind=-1), dict(kind=2))])
def test_refuses(lib, step, kw):
    assert call(lib, step, **kw) == _abi.KD_ERR_INVALID_ARG


@pytest.mark.parametrize("step", [False, True])
def test_refuses_a_bad_workspace(lib, step):
    need = lib.kd_fused_cross_entropy_workspace(256, 64, 1000, 128, int(step))
    for kw in (dict(wsb=need - 1), dict(ws=None), dict(ws=P + 64), dict(ctl=None), dict(ctl=P + 16)):
        assert call(lib, step, **kw) == _abi.KD_ERR_WORKSPACE
    assert lib.kd_fused_cross_entropy_workspace(0, 64, 1000, 128, 1) == 0


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=P + 8), dict(n=0), dict(n=12), dict(f=None), dict(f=P + 2)])
def test_scale_refuses(lib, kw):
    a = dict(x=P, n=64, f=P)
    a.update(kw)
    assert lib.kd_scale_gradient(a["x"], a["n"], 0, a["f"], None) == _abi.KD_ERR_INVALID_ARG


def test_wrappers_refuse_wrong_tensors():
    H, y = torch.zeros((2, 8), dtype=torch.bfloat16), torch.zeros((2,), dtype=torch.int32)
    for f in (kd.fused_cross_entropy, kd.fused_cross_entropy_forward, kd.fused_cross_entropy_step):
        with pytest.raises(ValueError):
            f(H, H, y)              # not CUDA tensors


def test_ignore_index_is_an_int32():
    H = torch.zeros((2, 8), dtype=torch.bfloat16)
    for f in (kd.fused_cross_entropy, kd.fused_cross_entropy_forward, kd.fused_cross_entropy_step):
        with pytest.raises(ValueError, match="ignore_index"):
            f(H, H, torch.zeros((2,), dtype=torch.int32), ignore_index=2 ** 32 - 100)
