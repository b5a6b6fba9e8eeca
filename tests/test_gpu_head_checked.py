"""The cross entropy and the 8-bit calls run clean in the checked build, which reports a bad index."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r'''
import torch
import sparse_teacher_kl_gb300 as kd

assert kd._abi.LIB_PATH.endswith("libkdkl_debug.so")
g = torch.Generator(device="cuda").manual_seed(4)
for N, d, V, chunk, valid in [(1, 8, 1, 128, 1.0), (300, 72, 1001, 128, 0.5), (513, 64, 320, 512, 0.9), (700, 128, 5000, 1024, 0.0)]:
    H = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn((V, d), generator=g, device="cuda").to(torch.bfloat16)
    y = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    y[torch.rand((N,), generator=g, device="cuda") >= valid] = -100
    ws = kd.workspace(kd._abi.kd_fused_cross_entropy_workspace(N, d, V, chunk, 1), "cuda")
    for kw in (dict(), dict(label_smoothing=0.1, z_loss=1e-3, softcap=20.0)):
        a, gH, gW = kd.fused_cross_entropy_step(H, W, y, chunk=chunk, ws=ws, **kw)
        b, _, _ = kd.fused_cross_entropy_forward(H, W, y, chunk=chunk, ws=ws, **kw)
        assert torch.equal(a, b) and torch.isfinite(gH).all() and torch.isfinite(gW).all()
        st, detail = kd.device_error(ws)
        assert st == 0, f"device error {st}, detail {detail:#x}"
for M, N, K, pad in [(1, 300, 100, 3), (4, 1000, 333, 0), (9, 129, 64, 0), (300, 1000, 1003, 5), (1000, 500, 128, 16)]:
    x = torch.randn((M, K), generator=g, device="cuda")
    w = torch.empty((N, K + pad), dtype=torch.int8, device="cuda")[:, :K]
    w, ws = kd.quantize_int8(torch.randn((N, K), generator=g, device="cuda"), q=w)
    q, s = kd.quantize_int8(x)
    out = kd.gemm_int8(q, s, w, ws, out_dtype=torch.float32)
    want = ((q.double() @ w.double().T).float() * s[:, None]) * ws
    assert torch.equal(out, want)
    ids, vals = kd.teacher_topk_int8(q, s, w, ws, 10, chunk=256)
    assert (vals[:, 0] >= vals[:, -1]).all() and int(ids.max()) < N
st, detail = kd.device_error(kd.control_block())
assert st == 0, f"device error {st}, detail {detail:#x}"
print("checked build ok")
'''


def test_checked_build(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library(debug=True)
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=dict(os.environ, KD_DEBUG="1"), capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "checked build ok" in r.stdout
