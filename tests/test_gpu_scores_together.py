"""The example runs, and the scoring and distillation kernels run clean in the checked build."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _run(args, env=None):
    r = subprocess.run([sys.executable, *args], cwd=ROOT, env=env, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    return r.stdout


def test_example_runs(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    out = _run([os.path.join("examples", "distill_step.py"), "--steps", "40"])
    assert "dense: loss" in out and "fused: loss" in out and out.count("top 3:") == 4


CHILD = r'''
import torch
import sparse_teacher_kl_gb300 as kd

assert kd._abi.LIB_PATH.endswith("libkdkl_debug.so")
g = torch.Generator(device="cuda").manual_seed(3)


def clean(ws):
    st, detail = kd.device_error(ws)
    assert st == 0, f"device error {st}, detail {detail:#x}"


for N, V, top, dtype in [(1, 201088, 128, torch.bfloat16), (3, 60001, 20, torch.float32), (40, 9001, 64, torch.float16),
                         (900, 513, 5, torch.bfloat16)]:
    z = torch.randn((N, V), generator=g, device="cuda").to(dtype)
    z[0] = (torch.arange(V, device="cuda") % 2).to(dtype)      # ties everywhere
    tok = torch.randint(0, V, (N, 3), generator=g, device="cuda", dtype=torch.int32)
    ws = kd.workspace(256, "cuda")
    r = kd.token_logprobs_forward(z, tok, top=top, entropy=True, ws=ws)
    kd.token_logprobs_backward(z, tok, r.lse, torch.ones_like(r.logp), entropy=r.entropy, grad_entropy=r.entropy, ws=ws)
    want = torch.log_softmax(z.double(), 1)
    assert (r.logp - want.gather(1, tok.long())).abs().max() < 1e-4
    clean(ws)
    K = 33
    ids = torch.argsort(torch.rand((N, V), generator=g, device="cuda"), dim=1)[:, :K].to(torch.int32).contiguous()
    ids[0, 1] = ids[0, 0]
    t = torch.randn((N, K), generator=g, device="cuda")
    ws = kd.workspace(kd._abi.kd_logits_kl_workspace(N, V, K), "cuda")
    for t_lse in (None, torch.logsumexp(t, 1) + 0.2):
        a, dz = kd.logits_kl_step(z, ids, t, t_lse=t_lse, ws=ws)
        b, stats, _ = kd.logits_kl_forward(z, ids, t, t_lse=t_lse, ws=ws)
        dz2 = kd.logits_kl_backward(z, ids, t, None, stats, torch.ones(1, device="cuda"), t_lse=t_lse, ws=ws)
        assert abs(float(a) - float(b)) < 1e-4 and (dz.float() - dz2.float()).abs().max() < 1e-3
        clean(ws)
H = torch.randn((300, 72), generator=g, device="cuda").to(torch.bfloat16)
W = torch.randn((1001, 72), generator=g, device="cuda").to(torch.bfloat16) * 0.1
for n in (1, 4, 300):
    tok = torch.arange(n, dtype=torch.int32, device="cuda")
    ws = kd.workspace(kd._abi.kd_fused_logprobs_workspace(n, 72, 1001, 128, 1), "cuda")
    logp, lse, ent, _ = kd.fused_logprobs_forward(H[:n], W, tok, chunk=128, entropy=True, ws=ws)
    kd.fused_logprobs_backward(H[:n], W, tok, lse, logp, chunk=128, entropy=ent, grad_entropy=ent, ws=ws)
    clean(ws)
print("checked build ok")
'''


def test_checked_build(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library(debug=True)
    assert "checked build ok" in _run(["-c", CHILD], dict(os.environ, KD_DEBUG="1"))
