"""Several rows a block, shared groups, small temperatures and padding run clean in the checked build."""
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
one = torch.ones(1, device="cuda")


def clean(ws):
    st, detail = kd.device_error(ws)
    assert st == 0, f"device error {st}, detail {detail:#x}"


for N, V, K, dtype in [(4000, 701, 40, torch.bfloat16), (2600, 9001, 33, torch.float16), (1300, 32000, 100, torch.bfloat16),
                       (700, 70001, 20, torch.bfloat16), (200, 201088, 20, torch.float32)]:
    z = torch.randn((N, V), generator=g, device="cuda").to(dtype)
    ids = torch.argsort(torch.rand((N, V), generator=g, device="cuda"), dim=1)[:, :K].to(torch.int32).contiguous()
    ids[::7, 1] = ids[::7, 0]
    t = torch.randn((N, K), generator=g, device="cuda")
    mask = (torch.rand((N,), generator=g, device="cuda") < 0.7).to(torch.uint8)
    ws = kd.workspace(kd._abi.kd_logits_kl_workspace(N, V, K), "cuda")
    for t_lse in (None, torch.logsumexp(t, 1) + 0.2):
        a, dz = kd.logits_kl_step(z, ids, t, mask, t_lse=t_lse, ws=ws)
        b, stats, _ = kd.logits_kl_forward(z, ids, t, mask, t_lse=t_lse, ws=ws)
        dz2 = kd.logits_kl_backward(z, ids, t, mask, stats, one, t_lse=t_lse, ws=ws)
        assert abs(float(a) - float(b)) < 1e-4 and (dz.float() - dz2.float()).abs().max() < 1e-3
        clean(ws)
ws = kd.workspace(256, "cuda")
for N, V, dtype in [(460, 140000, torch.float32), (930, 1003, torch.bfloat16)]:
    z = torch.randn((N, V), generator=g, device="cuda").to(dtype)
    tok = torch.randint(0, V, (N, 2), generator=g, device="cuda", dtype=torch.int32)
    for tau in (1.0, 1e-9):
        r = kd.token_logprobs_forward(z, tok, tau=tau, top=20, entropy=True, ws=ws)
        kd.token_logprobs_backward(z, tok, r.lse, torch.ones_like(r.logp), tau=tau, entropy=r.entropy,
                                   grad_entropy=r.entropy, ws=ws)
        clean(ws)
H = torch.randn((300, 72), generator=g, device="cuda").to(torch.bfloat16)
W = torch.randn((1001, 72), generator=g, device="cuda").to(torch.bfloat16)
tok = torch.arange(300, dtype=torch.int32, device="cuda")
for tau in (1.0, 1e-9):
    ws = kd.workspace(kd._abi.kd_fused_logprobs_workspace(300, 72, 1001, 128, 1), "cuda")
    logp, lse, ent, _ = kd.fused_logprobs_forward(H, W, tok, chunk=128, tau=tau, entropy=True, ws=ws)
    kd.fused_logprobs_backward(H, W, tok, lse, logp, chunk=128, tau=tau, entropy=ent, grad_entropy=ent, ws=ws)
    clean(ws)
print("checked build ok")
'''


def test_checked_build(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library(debug=True)
    r = subprocess.run([sys.executable, "-c", CHILD], cwd=ROOT, env=dict(os.environ, KD_DEBUG="1"), capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "checked build ok" in r.stdout
