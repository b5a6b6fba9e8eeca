"""Host-side argument checks of the cross entropy in two calls: refused before any CUDA work (no GPU needed)."""
import pytest

from sparse_teacher_kl_gb300 import _abi
from sparse_teacher_kl_gb300.build import build_library

P = 1 << 20   # fake, 256-byte aligned device address, never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    build_library()
    return _abi.load()


def keep(lib, **kw):
    a = dict(H=P, W=P, y=P, mask=None, N=200, d=64, V=1000, smooth=0.0, z=0.0, cap=0.0, ignore=-100, loss=P, lse=P,
             each=None, ws=P, wsb=1 << 30, ctl=P)
    a.update(kw)
    return lib.kd_fused_cross_entropy_keep(a["H"], a["W"], a["y"], a["mask"], a["N"], a["d"], a["V"], a["smooth"], a["z"],
                                           a["cap"], a["ignore"], a["loss"], a["lse"], a["each"], a["ws"], a["wsb"],
                                           a["ctl"], None)


def bwd(lib, **kw):
    a = dict(W=P, N=200, d=64, V=1000, smooth=0.0, cap=0.0, g=P, gH=P, f32=0, gW=P, kind=2, kept=P, kb=1 << 30, ws=P,
             wsb=1 << 30, ctl=P)
    a.update(kw)
    return lib.kd_fused_cross_entropy_bwd(a["W"], a["N"], a["d"], a["V"], a["smooth"], a["cap"], a["g"], a["gH"],
                                          a["f32"], a["gW"], a["kind"], a["kept"], a["kb"], a["ws"], a["wsb"], a["ctl"],
                                          None)


SIZES = [dict(N=0), dict(N=1 << 31), dict(N=(1 << 63) - 1), dict(d=0), dict(d=60), dict(V=0), dict(V=1 << 31),
         dict(W=None), dict(W=P + 2), dict(smooth=1.0), dict(smooth=float("nan")), dict(cap=1e-30), dict(cap=-1.0)]


@pytest.mark.parametrize("kw", SIZES + [dict(H=None), dict(y=None), dict(loss=None), dict(lse=P + 1), dict(each=P + 2),
                                        dict(z=-1.0)])
def test_keep_refuses(lib, kw):
    assert keep(lib, **kw) == _abi.KD_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", SIZES + [dict(g=P + 1), dict(gH=None), dict(gH=P + 8), dict(gW=None), dict(gW=P + 4),
                                        dict(kind=3), dict(kind=-1)])
def test_bwd_refuses(lib, kw):
    assert bwd(lib, **kw) == _abi.KD_ERR_INVALID_ARG


def test_bad_workspaces(lib):
    kept, ws = lib.kd_fused_cross_entropy_kept(200, 64, 1000), lib.kd_fused_cross_entropy_bwd_workspace(200, 64, 1000)
    # one layout: what is kept, and what the gradients need besides, is the step's workspace
    assert kept + ws == lib.kd_fused_cross_entropy_workspace(200, 64, 1000, 256, 1)
    for kw in (dict(wsb=kept - 1), dict(ws=None), dict(ws=P + 64), dict(ctl=None), dict(ctl=P + 16)):
        assert keep(lib, **kw) == _abi.KD_ERR_WORKSPACE
    for kw in (dict(kb=kept - 1), dict(kept=None), dict(kept=P + 64), dict(wsb=ws - 1), dict(ws=None), dict(ws=P + 64),
               dict(ctl=None), dict(ctl=P + 16)):
        assert bwd(lib, **kw) == _abi.KD_ERR_WORKSPACE
    assert lib.kd_fused_cross_entropy_kept(0, 64, 1000) == lib.kd_fused_cross_entropy_bwd_workspace(0, 64, 1000) == 0


@pytest.mark.parametrize("N,d,V,chunk", [(1, 8, 1, 128), (4096, 2880, 201088, 4096), (8192, 2048, 32000, 4096),
                                         (509, 1000, 50257, 8192)])
def test_workspaces_are_as_documented(lib, N, d, V, chunk):
    """The header's sums, sizes to whole tiles (128 positions, 128 columns; 64 of the 16-bit logits), nine parts each
    to 256 bytes."""
    up = lambda x, to: -(-x // to) * to
    c, room = up(min(N, chunk), 128), 9 * 256
    forward = c * (up(V, 128) // 8 + 2 * d + 20) + 8 * N
    more = c * (2 * up(V, 64) + 32 * d)
    for step, most in ((0, forward), (1, forward + more)):
        need = lib.kd_fused_cross_entropy_workspace(N, d, V, chunk, step)
        assert most - 256 <= need <= most + room + 256
