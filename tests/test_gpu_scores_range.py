"""Logits and temperatures anywhere in fp32's range: token_logprobs, logits_kl and fused_logprobs
against the float64 oracle.

Tolerances as in test_gpu_logprobs.py and test_gpu_logits_kl.py: with logits that are exact in fp32
their differences are rounded once, and scaled once by 1 / tau.  Temperatures are fp32 values.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from test_gpu_logprobs import EPS, check_both, check_forward, check_grad, draw, near, run_both, tokens_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


def f32(x):
    return float(np.float32(x))


# ------------------------------------------------------------- dense scores

@pytest.mark.parametrize("V", [40, 2051, 201088])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tau", [1e-30, 1e-10, 4e-9, 1.0])
def test_entropy_of_rows_of_zeros(kd, cuda_device, dtype, V, tau):
    """Logits of 0 and -inf: at 1 / tau above 2e8 the stand-in for an element that is not there stays finite."""
    z = torch.zeros((3, V), dtype=dtype, device="cuda")
    z[1, 1::2] = -math.inf
    z[2, :V - 1] = -math.inf
    ref = oracle.token_logprobs(z.double().cpu().numpy(), np.zeros((3, 1), np.int32), None, f32(tau), 3)
    r = kd.token_logprobs_forward(z, torch.zeros((3, 1), dtype=torch.int32, device="cuda"), tau=tau, top=3,
                                  entropy=True)
    check_forward(r, ref, 3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("N,V", [(3, 40), (5, 2051), (2, 201088)])
@pytest.mark.parametrize("tau", [1e-30, 1e-10, 4e-9, 1e-7, 1e-5, 1e-3])
def test_small_temperatures(kd, cuda_device, dtype, N, V, tau):
    z = draw(N, V, dtype, 5)
    z[1, ::2] = -math.inf
    tok = tokens_for(N, V, 2, 3)
    tok[:, 0] = z.argmax(1).to(torch.int32)
    if dtype is torch.float16:       # its gradients would not fit the type
        r = kd.token_logprobs_forward(z, tok, tau=tau, top=3, entropy=True)
        check_forward(r, oracle.token_logprobs(z.double().cpu().numpy(), tok.cpu().numpy(), None, f32(tau), 3), 3)
    else:
        check_both(kd, z, tok, tau=f32(tau), top=3)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tau", [1e-30, 1e-10, 4e-9, 1e-7, 1e-5, 1e-3])
def test_small_temperatures_of_many_rows(kd, cuda_device, dtype, tau):
    """Among many rows some have both tokens on the largest logit, where the gradient's terms cancel: 1e-5
    of the terms' sizes in the place of the row's largest entry."""
    z = draw(930, 1003, dtype, 5)
    z[1, ::2] = -math.inf
    tok = tokens_for(930, 1003, 2, 3)
    tok[:, 0] = z.argmax(1).to(torch.int32)
    r, dz, gl, ge = run_both(kd, z, tok, tau=f32(tau), top=3)
    host, t = z.double().cpu().numpy(), tok.cpu().numpy()
    check_forward(r, oracle.token_logprobs(host, t, None, f32(tau), 3), 3)
    ref = oracle.token_logprobs_grad(host, t, gl.cpu().numpy(), ge.cpu().numpy(), None, f32(tau))
    terms = (gl.abs().sum(1) + 40 * ge.abs()).double().cpu().numpy()[:, None] / f32(tau)
    near(dz.double().cpu(), ref, (EPS[dtype] + 1e-4) * np.abs(ref) + 1e-5 * terms)


def far_rows(dtype, V=6007):
    """Rows whose largest logit is far from zero, as a finite mask leaves them, at every size that leaves
    their differences representable; with a few logits just above the others; with two far values."""
    low = [-1e4, -6e4] if dtype is torch.float16 else [-1e6, -1e9, -1e10, -1e15, -1e20, -9e28, -1e30, -1e38]
    z = torch.stack([torch.full((V,), x, device="cuda") for x in low + [-x for x in low]]).to(dtype)
    step = z.abs() * 2.0 ** -8                    # representable in every type
    g = torch.Generator(device="cuda").manual_seed(3)
    up = torch.rand(z.shape, generator=g, device="cuda") < 0.01
    near_top = torch.where(up, (z.float() + step).to(dtype), z)
    mixed = z.clone()
    mixed[:, ::3] = (-z.float() * 0.5).to(dtype)[:, ::3]
    masked = z.clone()
    masked[:, 7::501] = 2.5
    return torch.cat([z, near_top, mixed, masked])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tau", [1.0, 1.7])
def test_rows_far_from_zero(kd, cuda_device, dtype, tau):
    z = far_rows(dtype)
    check_both(kd, z, tokens_for(z.shape[0], z.shape[1], 2, 1), tau=f32(tau), top=5)


# ------------------------------------------------------------- KL on dense logits

def kl_rows(dtype, V=5003, K=12):
    """Student rows as far_rows, the cached ids with logits of their own or masked like the rest."""
    z = far_rows(dtype, V)
    N = z.shape[0]
    g = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.argsort(torch.rand((N, V), generator=g, device="cuda"), dim=1)[:, :K]
    own = torch.arange(N, device="cuda") % 2 == 0
    z[own] = z[own].scatter(1, ids[own], torch.randn((int(own.sum()), K), generator=g, device="cuda").to(dtype))
    t = torch.randn((N, K), generator=g, device="cuda") * 2
    return z, ids.to(torch.int32).contiguous(), t.contiguous(), torch.logsumexp(t, 1) + 0.25


def check_kl(kd, z, ids, t, t_lse, tau, grad=0.75):
    """Forward, backward and step; each row's KL to 4e-7 of itself."""
    def host(x):
        return None if x is None else x.double().cpu().numpy() if x.is_floating_point() else x.cpu().numpy()

    ref = oracle.logits_kl(host(z), host(ids), host(t), None, tau, host(t_lse), grad)
    N, V = z.shape
    g = torch.full((1,), grad, device="cuda")
    tol = 6e-5 + 8e-7 * np.abs(np.nan_to_num(ref.kl, posinf=0))
    ws = kd.workspace(kd._abi.kd_logits_kl_workspace(N, V, ids.shape[1]), "cuda")
    kl = torch.empty((N,), device="cuda")
    _, stats, _ = kd.logits_kl_forward(z, ids, t, None, tau, t_lse, ws=ws, kl_out=kl)
    dz = kd.logits_kl_backward(z, ids, t, None, stats, g, tau, t_lse, ws=ws)
    near(kl.cpu(), ref.kl, tol)
    check_grad(dz, ref.grad, z.dtype)
    _, dz = kd.logits_kl_step(z, ids, t, None, tau, t_lse, g, ws=ws, kl_out=kl)
    near(kl.cpu(), ref.kl, tol)
    check_grad(dz, ref.grad, z.dtype)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
def test_kl_of_rows_far_from_zero(kd, cuda_device, dtype, tail):
    z, ids, t, t_lse = kl_rows(dtype)
    check_kl(kd, z, ids, t, t_lse if tail else None, 1.0)


def test_gradient_where_the_logsumexp_overflows(kd, cuda_device):
    """A row of fp32's lowest value at tau < 1: the logsumexp is -inf in fp32, and the row is still uniform;
    rows of nothing but -inf have no gradient."""
    z = torch.full((3, 1003), torch.finfo(torch.float32).min, device="cuda")
    z[1] = -math.inf
    z[2] = -torch.finfo(torch.float32).min
    tok = tokens_for(3, 1003, 1, 2)
    r, dz, gl, ge = run_both(kd, z, tok, tau=0.5)
    ref = oracle.token_logprobs_grad(z.double().cpu().numpy(), tok.cpu().numpy(), gl.cpu().numpy(), ge.cpu().numpy(),
                                     None, 0.5)
    check_grad(dz, ref, torch.float32)
    assert r.lse.tolist() == [-math.inf, -math.inf, math.inf]
    near(r.logp.cpu()[[0, 2]], np.full((2, 1), -math.log(1003)), 5e-5)


@pytest.mark.parametrize("tau", [1e-38, 1e-40, 1e-45, 1e38])
def test_temperatures_at_the_ends_of_fp32(kd, cuda_device, tau):
    """1 / tau above or near fp32's largest: one-hot rows, uniform at the other end; no NaN."""
    z = draw(4, 515, torch.float32, 9)
    tok = torch.stack([z.argmax(1), z.argmin(1)], 1).to(torch.int32)
    r, dz, _, _ = run_both(kd, z, tok, tau=tau)
    zero = kd.token_logprobs_backward(z, tok, r.lse, torch.zeros_like(r.logp), tau=tau)
    assert not zero.any()
    if tau < 1:
        assert r.logp[:, 0].tolist() == [0.0] * 4 and (r.logp[:, 1] < -1e37).all() and not r.entropy.any()
    else:
        near(r.logp.cpu(), np.full((4, 2), -math.log(515)), 5e-5)
        near(r.entropy.cpu(), np.full(4, math.log(515)), 4e-4)
        assert torch.isfinite(dz).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tau", [1e-30, 1e-10, 4e-9, 1e-7, 1e-5, 1e-3])
def test_kl_at_small_temperatures(kd, cuda_device, dtype, tau):
    z = draw(40, 1003, dtype, 6)
    g = torch.Generator(device="cuda").manual_seed(4)
    ids = torch.argsort(torch.rand((40, 1003), generator=g, device="cuda"), dim=1)[:, :9].to(torch.int32).contiguous()
    t = torch.randn((40, 9), generator=g, device="cuda") * 2
    check_kl(kd, z, ids, t, None, f32(tau))


# ------------------------------------------------------------- from hidden states

@pytest.mark.parametrize("N", [1, 4, 5, 300])
@pytest.mark.parametrize("V", [33, 1000, 1024, 5003])
@pytest.mark.parametrize("tau", [1e-30, 1e-10, 1.0])
def test_fused_entropy_of_equal_logits(kd, cuda_device, N, V, tau):
    """Logits of 0: the columns past the vocabulary in its last tile weigh nothing at any temperature."""
    H = torch.zeros((N, 64), dtype=torch.bfloat16, device="cuda")
    W = torch.ones((V, 64), dtype=torch.bfloat16, device="cuda")
    tok = torch.full((N,), V - 1, dtype=torch.int32, device="cuda")
    logp, lse, ent, _ = kd.fused_logprobs_forward(H, W, tok, tau=tau, entropy=True)
    near(ent.cpu(), np.full(N, math.log(V)), 4e-5 * (1 + math.log(V)))
    near(lse.cpu(), np.full(N, math.log(V)), 5e-5)
    near(logp.cpu(), np.full(N, -math.log(V)), 5e-5)


def exact_case(N, V, d=64, seed=0, scale=4.0):
    """Hidden states and a head whose logits are exact in fp32 whatever the order of the sum."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    H = (torch.randint(-16, 17, (N, d), generator=g, device="cuda") / 16.0 * scale).to(torch.bfloat16)
    W = (torch.randint(-16, 17, (V, d), generator=g, device="cuda") / 32.0).to(torch.bfloat16)
    tok = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    z = (H.double() @ W.double().T).cpu().numpy()
    tok[::2] = torch.from_numpy(z.argmax(1)).to(torch.int32).cuda()[::2]
    return H, W, tok, z


@pytest.mark.parametrize("N,V", [(1, 1000), (3, 1003), (4, 4096), (5, 1000), (40, 1024), (300, 1000)])
@pytest.mark.parametrize("tau", [1e-30, 1e-10, 4e-9, 1e-5])
def test_fused_entropy_and_logsumexp_at_small_temperatures(kd, cuda_device, N, V, tau):
    H, W, tok, z = exact_case(N, V)
    s = oracle.token_logprobs(z, tok.cpu().numpy(), None, f32(tau))
    _, lse, ent, _ = kd.fused_logprobs_forward(H, W, tok, tau=tau, entropy=True)
    near(lse.double().cpu(), s.lse, 4e-5 + 4e-7 * np.abs(s.lse))
    near(ent.double().cpu(), s.entropy, 4e-5 * (1 + s.entropy))


@pytest.mark.parametrize("N,V", [(1, 1000), (3, 1003), (4, 4096), (5, 1000), (40, 1024), (300, 1000)])
@pytest.mark.parametrize("tau", [1e-30, 1e-10, 4e-9, 1e-5])
def test_fused_scores_at_small_temperatures(kd, cuda_device, N, V, tau):
    H, W, tok, z = exact_case(N, V)
    s = oracle.token_logprobs(z, tok.cpu().numpy(), None, f32(tau))
    logp, lse, ent, _ = kd.fused_logprobs_forward(H, W, tok, tau=tau, entropy=True)
    check_forward(kd.TokenLogprobs(logp, lse, ent, None, None), s, 0)


@pytest.mark.parametrize("N,V", [(1, 1000), (4, 1003), (5, 1000), (300, 4096)])
@pytest.mark.parametrize("tau", [0.001, 0.01, 0.5])
def test_fused_log_probabilities_keep_their_digits(kd, cuda_device, N, V, tau):
    """The log probability's error is that of the difference to the largest logit, not of the logit over tau."""
    H, W, tok, z = exact_case(N, V, seed=1)
    s = oracle.token_logprobs(z, tok.cpu().numpy(), None, f32(tau))
    logp, _, _, _ = kd.fused_logprobs_forward(H, W, tok, tau=tau)
    near(logp.double().cpu(), s.logp[:, 0], 4e-5 + 4e-7 * np.abs(s.logp[:, 0]))


@pytest.mark.parametrize("N,V,chunk", [(1, 1000, 128), (5, 1003, 128), (300, 1000, 128), (300, 4096, 512)])
@pytest.mark.parametrize("tau", [1e-30, 1e-10, 1e-7, 1e-4, 0.02, 0.05])
def test_fused_gradients_at_small_temperatures(kd, cuda_device, N, V, chunk, tau):
    """Each entry within bf16's rounding of dZ (2^-9 of its terms, one binade of slack) and 1e-3 of the terms."""
    H, W, tok, z = exact_case(N, V, seed=2)
    tau = f32(tau)
    g = torch.Generator(device="cuda").manual_seed(7)
    gl = torch.randn((N,), generator=g, device="cuda")
    ge = torch.randn((N,), generator=g, device="cuda") * 0.2
    mask = (torch.rand((N,), generator=g, device="cuda") < 0.8).to(torch.uint8)
    logp, lse, ent, _ = kd.fused_logprobs_forward(H, W, tok, mask, chunk, tau, entropy=True)
    gH, gW = kd.fused_logprobs_backward(H, W, tok, lse, gl, mask, chunk, tau, ent, ge, grad_H_fp32=True)
    lp = torch.log_softmax(torch.from_numpy(z) / tau, 1).numpy()
    p = np.exp(lp)
    slope = np.where(p > 0, np.maximum(lp, -1e300), 0)
    H_row = -(p * slope).sum(1, keepdims=True)
    on = mask.cpu().numpy()[:, None] / tau
    l, e = gl.double().cpu().numpy()[:, None], ge.double().cpu().numpy()[:, None]
    one = np.zeros_like(p)
    one[np.arange(N), tok.cpu().numpy()] = 1
    dz = on * (l * one - p * (l + e * (slope + H_row)))
    bound = on * (np.abs(l) * one + p * (np.abs(l) + np.abs(e) * (np.abs(slope) + H_row)))
    h, w = H.double().cpu().numpy(), W.double().cpu().numpy()
    for got, ref, size in ((gH, dz @ w, bound @ np.abs(w)), (gW, dz.T @ h, bound.T @ np.abs(h))):
        near(got.double().cpu(), ref, (2.0 ** -8 + 1e-3) * size + 1e-30)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tau", [1.0, 0.3])
def test_kl_of_cached_ids_masked_with_the_lowest_value(kd, cuda_device, dtype, tau, tail):
    """The teacher keeps a little mass on tokens that the student masks with its type's lowest value, cached or
    (with the rest class) not: the KL is that mass times 3e38 / tau, in range although its unnormalised sums are
    not.  To 4e-6 of itself, and the rest's mass to 2^-21 (1 + t_lse)."""
    N, V, K = 20, 2000, 300
    low = torch.finfo(dtype).min
    g = torch.Generator(device="cuda").manual_seed(8)
    z = torch.randn((N, V), generator=g, device="cuda").to(dtype)
    ids = torch.argsort(torch.rand((N, V), generator=g, device="cuda"), dim=1)[:, :K].to(torch.int32).contiguous()
    t = torch.sort(torch.randn((N, K), generator=g, device="cuda") * 0.3, dim=1, descending=True)[0].contiguous()
    t_lse = torch.logsumexp(t / tau, 1) + 0.05 if tail else None
    if tail:
        z.masked_fill_(torch.ones_like(z, dtype=torch.bool).scatter_(1, ids.long(), False), low)
    z.scatter_(1, ids[:, K - 60:].long(), low)
    host = [x.double().cpu().numpy() if x is not None and x.is_floating_point() else x for x in (z, t, t_lse)]
    ref = oracle.logits_kl(host[0], ids.cpu().numpy(), host[1], None, f32(tau), host[2])
    assert (ref.kl > 1e36).all() and (ref.kl < 3e38).all()
    tol = 4e-6 * ref.kl
    if tail:
        tol = tol + 2.0 ** -21 * (1 + np.abs(host[2])) * 3.4e38 / tau
    kl = torch.empty((N,), device="cuda")
    kd.logits_kl_forward(z, ids, t, None, tau, t_lse, kl_out=kl)
    near(kl.cpu(), ref.kl, tol)
    loss, dz = kd.logits_kl_step(z, ids, t, None, tau, t_lse, kl_out=kl)
    near(kl.cpu(), ref.kl, tol)
    near(loss.cpu(), [ref.loss], tol.max())
    check_grad(dz, ref.grad, dtype)
