"""fused_logprobs (hidden states to log probability, entropy and gradients) against the
float64 oracle on the logits of identical bf16 inputs.

Tolerances.  A logit is a sum of d exact bf16 products in fp32: its error is below
2^-23 sqrt(d) sum |h w| (rounding to nearest of a chain of d additions, as a random walk), at
most 2.5e-4 for d <= 2048 with |h| ~ 1, |w| ~ 1.5 / sqrt(d), and the logsumexp's is no larger:
  logp, lse : 5e-4 absolute     entropy : 5e-4 (1 + H)
Gradients are products with dZ rounded to bf16 (2^-9 of each entry) and, for bf16 outputs, one
more rounding: 1e-2 of the tensor's largest entry covers the sum of both with entries of mixed
sign.
"""
import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


def case(N, d, V, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    H = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn((V, d), generator=g, device="cuda") * (1.5 / d ** 0.5)).to(torch.bfloat16)
    tokens = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    gl = torch.randn((N,), generator=g, device="cuda")
    ge = torch.randn((N,), generator=g, device="cuda") * 0.2
    return H, W, tokens, gl, ge


def host(x):
    return None if x is None else x.double().cpu().numpy() if x.is_floating_point() else x.cpu().numpy()


def reference(H, W, tokens, mask, tau, gl=None, ge=None):
    H, W, tok = host(H), host(W), host(tokens).copy()
    z = H @ W.T
    m = host(mask)
    if m is not None:
        tok[m == 0] = 0
    s = oracle.token_logprobs(z, tok, m, tau)
    if gl is None:
        return s, None, None
    dz = oracle.token_logprobs_grad(z, tok, host(gl), host(ge), m, tau)
    return s, dz @ W, dz.T @ H


def off(got, ref):
    return float(np.max(np.abs(host(got) - ref))) / max(float(np.max(np.abs(ref))), 1e-30)


def check(kd, H, W, tokens, gl, ge, mask=None, tau=1.0, chunk=4096, fp32=True):
    N, d = H.shape
    ws = kd.workspace(kd._abi.kd_fused_logprobs_workspace(N, d, W.shape[0], chunk, 1), "cuda")
    logp, lse, ent, _ = kd.fused_logprobs_forward(H, W, tokens, mask, chunk, tau, entropy=True, ws=ws)
    gH, gW = kd.fused_logprobs_backward(H, W, tokens, lse, gl, mask, chunk, tau, ent, ge, ws=ws, grad_H_fp32=fp32)
    torch.cuda.synchronize()
    assert kd.device_error(ws)[0] == 0
    s, rH, rW = reference(H, W, tokens, mask, tau, gl, ge)
    assert np.max(np.abs(host(logp) - s.logp[:, 0])) <= 5e-4
    assert np.max(np.abs(host(lse) - s.lse)) <= 5e-4
    assert np.max(np.abs(host(ent) - s.entropy) / (1 + s.entropy)) <= 5e-4
    assert off(gH, rH) <= 1e-2 and off(gW, rW) <= 1e-2
    return logp, lse, ent, gH, gW


@pytest.mark.parametrize("N,d,V,chunk,tau", [
    (1, 64, 1000, 128, 1.0),       # one token: a tile of one row
    (3, 8, 2, 128, 1.0),           # the narrowest head
    (5, 72, 257, 128, 0.7),
    (128, 256, 4096, 4096, 1.0),
    (129, 136, 1001, 256, 2.0),    # a pair of row tiles, one row in the second
    (300, 72, 1000, 128, 1.0),     # three chunks, the last short
    (600, 320, 2100, 256, 1.3),    # pairs, then a single-tile chunk
    (257, 2048, 3001, 1024, 1.0),
])
def test_matches_oracle(kd, cuda_device, N, d, V, chunk, tau):
    check(kd, *case(N, d, V, seed=N + V), tau=tau, chunk=chunk)


@pytest.mark.parametrize("chunk", [128, 512])
def test_padding(kd, cuda_device, chunk):
    H, W, tokens, gl, ge = case(400, 128, 900)
    mask = (torch.rand(400, generator=torch.Generator().manual_seed(3)) < 0.6).to(torch.uint8).cuda()
    tokens[mask == 0] = -100
    out = check(kd, H, W, tokens, gl, ge, mask, chunk=chunk)
    for t in out[:4]:
        assert not t[mask == 0].any()


def test_forward_workspace_is_enough_and_entropy_is_optional(kd, cuda_device):
    H, W, tokens, gl, _ = case(200, 64, 1500)
    logp, lse, ent, ws = kd.fused_logprobs_forward(H, W, tokens, chunk=128)
    assert ent is None and ws.numel() == kd._abi.kd_fused_logprobs_workspace(200, 64, 1500, 128, 0)
    assert ws.numel() < kd._abi.kd_fused_logprobs_workspace(200, 64, 1500, 128, 1)
    gH, gW = kd.fused_logprobs_backward(H, W, tokens, lse, gl, chunk=128, grad_H_fp32=True)
    s, rH, rW = reference(H, W, tokens, None, 1.0, gl, torch.zeros_like(gl))
    assert np.max(np.abs(host(logp) - s.logp[:, 0])) <= 5e-4
    assert off(gH, rH) <= 1e-2 and off(gW, rW) <= 1e-2


def test_grad_W_accumulates(kd, cuda_device):
    H, W, tokens, gl, ge = case(130, 64, 700)
    logp, lse, ent, _ = kd.fused_logprobs_forward(H, W, tokens, entropy=True)
    _, once = kd.fused_logprobs_backward(H, W, tokens, lse, gl, entropy=ent, grad_entropy=ge)
    base = torch.randn_like(once)
    _, twice = kd.fused_logprobs_backward(H, W, tokens, lse, gl, entropy=ent, grad_entropy=ge, grad_W=base.clone())
    assert torch.allclose(twice, once + base, atol=1e-6, rtol=0)


@pytest.mark.parametrize("N,d,V", [(1, 64, 1000), (130, 72, 257), (512, 192, 3000)])
def test_grad_W_kinds(kd, cuda_device, N, d, V):
    """Stored fp32 and bf16 gradients: nothing of what the memory held before is left in them."""
    H, W, tokens, gl, ge = case(N, d, V)
    _, lse, ent, _ = kd.fused_logprobs_forward(H, W, tokens, entropy=True)
    _, _, rW = reference(H, W, tokens, None, 1.0, gl, ge)
    zero = torch.zeros((V, d), device="cuda")
    _, added = kd.fused_logprobs_backward(H, W, tokens, lse, gl, entropy=ent, grad_entropy=ge, grad_W=zero)
    junk = torch.full((V, d), float("nan"), device="cuda")
    del junk   # its memory is likely the next allocation's
    _, stored = kd.fused_logprobs_backward(H, W, tokens, lse, gl, entropy=ent, grad_entropy=ge)
    _, narrow = kd.fused_logprobs_backward(H, W, tokens, lse, gl, entropy=ent, grad_entropy=ge, grad_W_bf16=True)
    assert torch.equal(stored, added) and narrow.dtype == torch.bfloat16
    assert torch.equal(narrow, stored.to(torch.bfloat16))
    assert off(stored, rW) <= 1e-2
    _, chunked = kd.fused_logprobs_backward(H, W, tokens, lse, gl, chunk=128, entropy=ent, grad_entropy=ge)
    assert off(chunked, rW) <= 1e-2
    if N > 128:
        with pytest.raises(kd.KDError):
            kd.fused_logprobs_backward(H, W, tokens, lse, gl, chunk=128, entropy=ent, grad_entropy=ge, grad_W_bf16=True)


def test_autograd(kd, cuda_device):
    H, W, tokens, gl, ge = case(140, 96, 800)
    s, rH, rW = reference(H, W, tokens, None, 1.0, gl, ge)
    Hr, Wr = H.clone().requires_grad_(True), W.clone().requires_grad_(True)
    logp, ent = kd.fused_logprobs(Hr, Wr, tokens, chunk=128)
    ((logp * gl).sum() + (ent * ge).sum()).backward()
    assert Hr.grad.dtype == torch.bfloat16 and Wr.grad.dtype == torch.bfloat16
    assert off(Hr.grad, rH) <= 1e-2 and off(Wr.grad, rW) <= 1e-2
    Hr.grad = None
    logp, ent = kd.fused_logprobs(Hr, Wr, tokens, chunk=128)
    ent.sum().backward()     # the entropy alone
    _, rH, _ = reference(H, W, tokens, None, 1.0, torch.zeros_like(gl), torch.ones_like(ge))
    assert off(Hr.grad, rH) <= 1e-2


def test_gradient_matches_differences(kd, cuda_device):
    """Central differences over one direction of H (bf16-exact steps of 1/8 on entries that stay
    representable): truncation (step^2 / 6)|f'''| and the forward's 5e-4 each side over 2 steps."""
    g = torch.Generator(device="cuda").manual_seed(5)
    H = (torch.randint(-8, 9, (2, 64), generator=g, device="cuda") / 8.0).to(torch.bfloat16)
    W = (torch.randint(-8, 9, (300, 64), generator=g, device="cuda") / 16.0).to(torch.bfloat16)
    tokens = torch.tensor([7, 299], dtype=torch.int32, device="cuda")
    one = torch.ones((2,), device="cuda")

    def f(x):
        logp, _, ent, _ = kd.fused_logprobs_forward(x, W, tokens, entropy=True)
        return float(logp.double().sum() + 0.5 * ent.double().sum())

    _, lse, ent, _ = kd.fused_logprobs_forward(H, W, tokens, entropy=True)
    gH, _ = kd.fused_logprobs_backward(H, W, tokens, lse, one, entropy=ent, grad_entropy=0.5 * one, grad_H_fp32=True)
    for j in (0, 31, 63):
        hi, lo = H.clone(), H.clone()
        hi[0, j] += 0.125
        lo[0, j] -= 0.125
        assert abs(float(gH[0, j]) - (f(hi) - f(lo)) / 0.25) <= 1e-2


def test_agrees_with_the_dense_operator(kd, cuda_device):
    H, W, tokens, _, _ = case(64, 256, 5000)
    logp, lse, ent, _ = kd.fused_logprobs_forward(H, W, tokens, entropy=True)
    z = (H.double() @ W.double().T).float()
    r = kd.token_logprobs_forward(z, tokens, entropy=True)
    assert (logp - r.logp).abs().max() <= 5e-4 and (ent - r.entropy).abs().max() <= 5e-3


def test_bad_token_is_reported(kd, cuda_device):
    H, W, tokens, gl, _ = case(150, 64, 400)
    tokens[131] = 400
    logp, lse, _, ws = kd.fused_logprobs_forward(H, W, tokens)
    assert kd.device_error(ws) == (kd._abi.KD_ERR_DEVICE, 131)
    assert torch.isnan(logp[131]) and int(torch.isnan(logp).sum()) == 1
    gH, gW = kd.fused_logprobs_backward(H, W, tokens, lse, gl, grad_H_fp32=True)
    gl[131], tokens[131] = 0, 0
    _, rH, rW = reference(H, W, tokens, None, 1.0, gl, torch.zeros_like(gl))
    assert off(gH, rH) <= 1e-2 and off(gW, rW) <= 1e-2


def test_repeats_are_bit_identical_on_any_stream(kd, cuda_device):
    H, W, tokens, gl, ge = case(300, 128, 2000)

    def go():
        logp, lse, ent, _ = kd.fused_logprobs_forward(H, W, tokens, chunk=128, entropy=True)
        return (logp, lse, ent, *kd.fused_logprobs_backward(H, W, tokens, lse, gl, None, 128, 1.0, ent, ge))

    first = go()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = go()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, again))
