"""The cross entropy in two calls, and under every code of its logits, runs clean in the checked build, which reports a
bad index."""
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
for N, d, V, valid in [(1, 8, 1, 1.0), (300, 72, 1001, 0.5), (513, 64, 320, 0.9), (700, 128, 5000, 0.0)]:
    H = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn((V, d), generator=g, device="cuda").to(torch.bfloat16)
    y = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    y[torch.rand((N,), generator=g, device="cuda") >= valid] = -100
    for cap in (0.0, 1e-3, 10.0, 30.0, 100.0):
        for chunk in (1024, 128):
            h, w = H.clone().requires_grad_(), W.clone().requires_grad_()
            loss = kd.fused_cross_entropy(h, w, y, chunk=chunk, softcap=cap, label_smoothing=0.1)
            a = torch.autograd.grad(loss, (h, w), torch.tensor(0.3, device="cuda"), retain_graph=True)
            b = torch.autograd.grad(loss, (h, w), torch.tensor(0.3, device="cuda"))
            assert torch.isfinite(loss) and all(torch.isfinite(t).all() for t in a)
            if N <= chunk:
                assert all(torch.equal(p, q) for p, q in zip(a, b))
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
