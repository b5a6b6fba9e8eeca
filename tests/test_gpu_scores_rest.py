"""A teacher whose cache holds all of its mass although the vocabulary is larger: what 1 - sum of p leaves
is the rounding of t_lse and the sum, not mass, and no student can be wrong about it."""
import math

import numpy as np
import pytest
import torch

import oracle
from test_gpu_logits_kl import host
from test_gpu_logprobs import check_grad, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


@pytest.mark.parametrize("V,K,dtype,shift", [(700, 40, torch.float32, 0.0), (700, 40, torch.bfloat16, 17.0),
                                             (33000, 1024, torch.float32, -30.0), (5000, 100, torch.float16, 5.0)])
@pytest.mark.parametrize("fill", ["inf", "lowest"])
def test_everything_outside_the_cache_is_banned(kd, cuda_device, V, K, dtype, shift, fill):
    N = 200 if V < 10000 else 40
    g = torch.Generator(device="cuda").manual_seed(V)
    ids = torch.argsort(torch.rand((N, V), generator=g, device="cuda"), dim=1)[:, :K]
    t = (torch.randn((N, K), generator=g, device="cuda") * 3 + shift).contiguous()
    t_lse = torch.logsumexp(t, 1)                     # of the whole row: its other logits are -inf
    low = -math.inf if fill == "inf" else torch.finfo(dtype).min
    z = torch.full((N, V), low, device="cuda").scatter_(1, ids, t + torch.randn((N, K), generator=g, device="cuda"))
    z = z.to(dtype)
    ids = ids.to(torch.int32).contiguous()
    # test_scores_rest.py: within 1e-4 of the value without a rest class
    ref = oracle.logits_kl(host(z), host(ids), host(t), None, 1.0, host(t_lse), 0.75)
    assert np.isfinite(ref.kl).all()
    tol = 6e-5 + 8e-7 * (ref.kl + 40)
    one = torch.full((1,), 0.75, device="cuda")
    kl = torch.empty((N,), device="cuda")
    loss, stats, ws = kd.logits_kl_forward(z, ids, t, None, 1.0, t_lse, kl_out=kl)
    near(kl.cpu(), ref.kl, tol)
    near(loss.cpu(), [ref.loss], tol.max())
    check_grad(kd.logits_kl_backward(z, ids, t, None, stats, one, 1.0, t_lse, ws=ws), ref.grad, dtype)
    loss, dz = kd.logits_kl_step(z, ids, t, None, 1.0, t_lse, one, ws=ws, kl_out=kl)
    near(kl.cpu(), ref.kl, tol)
    check_grad(dz, ref.grad, dtype)
    assert np.isfinite(float(loss))


@pytest.mark.parametrize("rest", [1e-4, 1e-3])
def test_a_small_rest_is_still_mass(kd, cuda_device, rest):
    N, V, K = 50, 2000, 30
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn((N, V), generator=g, device="cuda")
    ids = torch.argsort(torch.rand((N, V), generator=g, device="cuda"), dim=1)[:, :K].to(torch.int32).contiguous()
    t = torch.randn((N, K), generator=g, device="cuda")
    t_lse = (torch.logsumexp(t.double(), 1) - math.log1p(-rest)).float()
    ref = oracle.logits_kl(host(z), host(ids), host(t), None, 1.0, host(t_lse))
    kl = torch.empty((N,), device="cuda")
    kd.logits_kl_step(z, ids, t, None, 1.0, t_lse, kl_out=kl)
    # p_R within 2^-21 (1 + t_lse) of the float64 value, times |ln p_R / q_R| + 1
    near(kl.cpu(), ref.kl, 6e-5 + 2.0 ** -21 * (1 + np.abs(host(t_lse))) * (1 + abs(math.log(rest))))
    assert (ref.kl - oracle.logits_kl(host(z), host(ids), host(t)).kl).min() < -1e-6   # the rest is seen


def test_a_teacher_row_of_nothing(kd, cuda_device):
    """Every teacher logit of a row -inf, its logsumexp too: no divergence and no gradient in that row."""
    g = torch.Generator(device="cuda").manual_seed(1)
    z = torch.randn((6, 900), generator=g, device="cuda")
    ids = torch.argsort(torch.rand((6, 900), generator=g, device="cuda"), dim=1)[:, :7].to(torch.int32).contiguous()
    t = torch.randn((6, 7), generator=g, device="cuda")
    t_lse = torch.logsumexp(t, 1) + 0.3
    t[2], t_lse[2] = -math.inf, -math.inf
    ref = oracle.logits_kl(host(z), host(ids), host(t), None, 1.0, host(t_lse))
    kl = torch.empty((6,), device="cuda")
    _, dz = kd.logits_kl_step(z, ids, t, None, 1.0, t_lse, kl_out=kl)
    near(kl.cpu(), ref.kl, 6e-5)
    rows = [0, 1, 3, 4, 5]
    check_grad(dz[rows], ref.grad[rows], torch.float32)
    # q_R - 1 is the rounding of the row's sum (2^-22), spread over the row
    assert abs(float(kl[2])) <= 1e-6 and float(dz[2].abs().max()) <= 1e-6 / 6
