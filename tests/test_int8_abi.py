"""Host-side argument checks of the 8-bit calls: refused before any CUDA work (no GPU needed)."""
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


def quantize(lib, **kw):
    a = dict(x=P, dt=0, N=4, d=64, ld=64, q=P, ldq=64, s=P)
    a.update(kw)
    return lib.kd_quantize_int8(a["x"], a["dt"], a["N"], a["d"], a["ld"], a["q"], a["ldq"], a["s"], None)


@pytest.mark.parametrize("kw", [dict(x=None), dict(x=P + 1), dict(dt=2, x=P + 2), dict(dt=3), dict(dt=-1), dict(N=0),
                                dict(N=1 << 31), dict(d=0), dict(d=1 << 31, ld=1 << 31, ldq=1 << 31), dict(ld=63),
                                dict(ldq=63), dict(q=None), dict(s=None), dict(s=P + 2)])
def test_quantize_refuses(lib, kw):
    assert quantize(lib, **kw) == _abi.KD_ERR_INVALID_ARG


def gemm(lib, **kw):
    a = dict(A=P, lda=64, sa=P, B=P, ldb=64, sb=P, C=P, dt=0, ldc=100, M=8, N=100, K=64, ws=P, wsb=1 << 30, ctl=P)
    a.update(kw)
    return lib.kd_gemm_int8(a["A"], a["lda"], a["sa"], a["B"], a["ldb"], a["sb"], a["C"], a["dt"], a["ldc"], a["M"],
                            a["N"], a["K"], a["ws"], a["wsb"], a["ctl"], None)


@pytest.mark.parametrize("kw", [
    dict(A=None), dict(B=None), dict(C=None), dict(sa=None), dict(sb=None), dict(sa=P + 1), dict(sb=P + 2),
    dict(lda=63), dict(ldb=63), dict(ldc=99), dict(M=0), dict(N=0), dict(K=0), dict(M=1 << 31), dict(N=1 << 31), dict(M=(1 << 31) - 512), dict(N=(1 << 31) - 1, ldc=1 << 31),
    dict(K=65537, lda=65537, ldb=65537), dict(dt=3), dict(dt=-1), dict(C=P + 1), dict(dt=2, C=P + 2),
    dict(M=(1 << 31) - 1, N=(1 << 31) - 1, ldc=1 << 31)])
def test_gemm_refuses(lib, kw):
    assert gemm(lib, **kw) == _abi.KD_ERR_INVALID_ARG


def test_gemm_refuses_a_bad_workspace(lib):
    for at, ld in ((P, 64), (P + 1, 64), (P, 65)):
        fits = int(at % 16 == 0 and ld % 16 == 0)
        need = lib.kd_gemm_int8_workspace(8, 100, 64, fits)
        assert gemm(lib, B=at, ldb=ld, wsb=need - 1) == _abi.KD_ERR_WORKSPACE
    assert lib.kd_gemm_int8_workspace(80, 100, 64, 0) > lib.kd_gemm_int8_workspace(80, 100, 64, 1)
    for kw in (dict(ws=None), dict(ws=P + 64), dict(ctl=None), dict(ctl=P + 16)):
        assert gemm(lib, **kw) == _abi.KD_ERR_WORKSPACE
    assert lib.kd_gemm_int8_workspace(0, 100, 64, 1) == 0


def teacher(lib, **kw):
    a = dict(H=P, ldh=64, hs=P, W=P, ldw=64, wsc=P, N=8, d=64, V=100, K=10, chunk=4, ids=P, vals=P, lse=None, drop=None,
             ws=P, wsb=1 << 30, ctl=P)
    a.update(kw)
    return lib.kd_teacher_topk_int8(a["H"], a["ldh"], a["hs"], a["W"], a["ldw"], a["wsc"], a["N"], a["d"], a["V"], a["K"],
                                    a["chunk"], a["ids"], a["vals"], a["lse"], a["drop"], a["ws"], a["wsb"], a["ctl"],
                                    None)


@pytest.mark.parametrize("kw", [
    dict(H=None), dict(W=None), dict(hs=None), dict(wsc=P + 1), dict(ldh=63), dict(ldw=63), dict(N=0), dict(d=0),
    dict(V=0), dict(K=0), dict(K=101), dict(K=1025, V=2000), dict(chunk=0), dict(ids=None), dict(vals=None),
    dict(ids=P + 2), dict(lse=P + 1), dict(drop=P + 2)])
def test_teacher_refuses(lib, kw):
    assert teacher(lib, **kw) == _abi.KD_ERR_INVALID_ARG


def test_teacher_refuses_a_bad_workspace(lib):
    need = lib.kd_teacher_topk_int8_workspace(8, 64, 100, 10, 4, 1)
    for kw in (dict(wsb=need - 1), dict(ws=None), dict(ws=P + 64), dict(ctl=None), dict(ctl=P + 16)):
        assert teacher(lib, **kw) == _abi.KD_ERR_WORKSPACE
    assert lib.kd_teacher_topk_int8_workspace(0, 64, 100, 10, 4, 1) == 0


def test_wrappers_refuse_wrong_tensors():
    x, q, s = torch.zeros((2, 8)), torch.zeros((2, 8), dtype=torch.int8), torch.ones((2,))
    with pytest.raises(ValueError):
        kd.quantize_int8(x)                    # not a CUDA tensor
    with pytest.raises(ValueError):
        kd.gemm_int8(q, s, q, s)
    with pytest.raises(ValueError):
        kd.teacher_topk_int8(q, s, q, s, 2)
