"""fused_logprobs entry by entry, and with a few hidden states.

Tolerances.  With d <= 2048 a logit is within 5e-4 (test_gpu_fused_logprobs.py); dZ is rounded to bf16
(2^-9 of each entry, one binade of slack) and its terms carry the logits' error (2e-3 of each): an entry of
a gradient is within (2^-8 + 2e-3) of the sum of its terms' sizes, whatever cancels among them.
"""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_fused_logprobs import case, host

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


def terms(H, W, tokens, gl, ge, mask, tau):
    """dZ of the valid rows and the sizes of its terms, both [N, V] in float64."""
    z = host(H) @ host(W).T / tau
    lp = z - np.log(np.exp(z - z.max(1, keepdims=True)).sum(1, keepdims=True)) - z.max(1, keepdims=True)
    p = np.exp(lp)
    ent = -(p * lp).sum(1, keepdims=True)
    on = (np.ones(len(z)) if mask is None else host(mask).astype(float))[:, None] / tau
    l, e = host(gl)[:, None], host(ge)[:, None]
    one = np.zeros_like(p)
    tok = host(tokens)
    ok = (tok >= 0) & (tok < p.shape[1])
    one[np.flatnonzero(ok), tok[ok]] = 1
    l = l * ok[:, None]
    return on * (l * one - p * (l + e * (lp + ent))), on * (np.abs(l) * one + p * (np.abs(l) + np.abs(e) * (-lp + ent)))


def check_gradients(kd, H, W, tokens, gl, ge, mask=None, tau=1.0, chunk=4096):
    _, lse, ent, _ = kd.fused_logprobs_forward(H, W, tokens, mask, chunk, tau, entropy=True)
    gH, gW = kd.fused_logprobs_backward(H, W, tokens, lse, gl, mask, chunk, tau, ent, ge, grad_H_fp32=True)
    dz, size = terms(H, W, tokens, gl, ge, mask, tau)
    h, w = host(H), host(W)
    for got, ref, bound in ((gH, dz @ w, size @ np.abs(w)), (gW, dz.T @ h, size.T @ np.abs(h))):
        off = np.abs(host(got) - ref) - (2.0 ** -8 + 2e-3) * bound
        assert off.max() <= 0, f"off by {off.max()} more than allowed"


@pytest.mark.parametrize("N,d,V,chunk,tau", [
    (1, 64, 1000, 128, 1.0), (3, 8, 2, 128, 1.0), (5, 72, 257, 128, 0.7), (128, 256, 4096, 4096, 1.0),
    (129, 136, 1001, 256, 2.0), (300, 72, 1000, 128, 1.0), (600, 320, 2100, 256, 1.3), (257, 2048, 3001, 1024, 1.0)])
def test_every_entry_of_the_gradients(kd, cuda_device, N, d, V, chunk, tau):
    H, W, tokens, gl, ge = case(N, d, V, seed=N + V)
    check_gradients(kd, H, W, tokens, gl, ge, None, tau, chunk)
    mask = (torch.rand((N,), generator=torch.Generator().manual_seed(3)) < 0.6).to(torch.uint8).cuda()
    tokens[mask == 0] = -100
    check_gradients(kd, H, W, tokens, gl, ge, mask, tau, chunk)


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5])
@pytest.mark.parametrize("d,V", [(64, 33), (72, 1000), (2880, 5003)])
@pytest.mark.parametrize("tau", [1.0, 0.6])
def test_few_hidden_states(kd, cuda_device, N, d, V, tau):
    """Values of every row, with padding in each place and with a token out of range."""
    H, W, tokens, _, _ = case(N, d, V, seed=d + N)
    z = host(H) @ host(W).T
    for out in range(-1, N):
        mask, tok = None, tokens.clone()
        if out >= 0:
            mask = torch.ones((N,), dtype=torch.uint8, device="cuda")
            mask[out] = 0
            tok[out] = -7
        logp, lse, ent, ws = kd.fused_logprobs_forward(H, W, tok, mask, tau=tau, entropy=True)
        assert kd.device_error(ws)[0] == 0
        safe = host(tok).copy()
        safe[safe < 0] = 0
        s = oracle.token_logprobs(z, safe, host(mask), tau)
        assert np.max(np.abs(host(logp) - s.logp[:, 0])) <= 5e-4
        assert np.max(np.abs(host(lse) - s.lse)) <= 5e-4
        assert np.max(np.abs(host(ent) - s.entropy) / (1 + s.entropy)) <= 5e-4
    tok = tokens.clone()
    tok[N - 1] = V
    logp, lse, ent, ws = kd.fused_logprobs_forward(H, W, tok, tau=tau, entropy=True)
    assert kd.device_error(ws) == (kd._abi.KD_ERR_DEVICE, N - 1)
    s = oracle.token_logprobs(z, np.minimum(host(tok), V - 1), None, tau)
    assert torch.isnan(logp[N - 1]) and np.max(np.abs(host(lse) - s.lse)) <= 5e-4
    assert N == 1 or np.max(np.abs(host(logp) - s.logp[:, 0])[:N - 1]) <= 5e-4


@pytest.mark.parametrize("N,d,V", [(1, 2048, 40001), (1, 8192, 10000), (2, 2048, 80003), (2, 4096, 40000)])
@pytest.mark.parametrize("tau", [1.0, 0.01])
def test_one_and_two_hidden_states_of_a_large_head(kd, cuda_device, N, d, V, tau):
    """Heads beyond 150 MB a row, which are streamed without the tensor cores: values, padding in each place,
    a token out of range."""
    H, W, tokens, _, _ = case(N, d, V, seed=d + N)
    W = (W.float() * 2).to(torch.bfloat16)
    x = H.double() @ W.double().T / tau
    lp = torch.log_softmax(x, 1)
    lse, ent = torch.logsumexp(x, 1), -(lp.exp() * lp).sum(1)
    # a logit is within 2^-23 sqrt(d) of the sum of its products' sizes
    off = float((H.double().abs() @ W.double().abs().T).max()) * 2.0 ** -23 * d ** 0.5 / tau
    assert off < 0.2
    want = lp.gather(1, tokens.long()[:, None])[:, 0]
    for out in range(-1, N):
        mask, tok = None, tokens.clone()
        on = torch.ones((N,), dtype=torch.float64, device="cuda")
        if out >= 0:
            on[out] = 0
            mask, tok[out] = on.to(torch.uint8), -7
        logp, got, h, ws = kd.fused_logprobs_forward(H, W, tok, mask, tau=tau, entropy=True)
        assert kd.device_error(ws)[0] == 0
        assert ((logp - want * on).abs() <= 2 * off + 5e-5 + 4e-7 * want.abs()).all()
        assert ((got - lse * on).abs() <= off + 5e-5 + 4e-7 * lse.abs()).all()
        # dH = -sum of (ln p + H) dp, |dp| <= 2 off p
        spread = (lp.exp() * (lp + ent[:, None]).abs()).sum(1)
        assert ((h - ent * on).abs() <= 2 * off * spread + 5e-5 * (1 + ent)).all()
    tokens[N - 1] = V
    logp, _, _, ws = kd.fused_logprobs_forward(H, W, tokens, tau=tau)
    assert kd.device_error(ws) == (kd._abi.KD_ERR_DEVICE, N - 1) and torch.isnan(logp[N - 1])
    assert N == 1 or float((logp[0] - want[0]).abs()) <= 2 * off + 5e-5 + 4e-7 * float(want[0].abs())
