"""logits_kl with several rows for every persistent block, and the padding rows between them.

The forward pass and the step run a grid of resident blocks over all rows; which variant runs goes by a
row's bytes.  Every case here gives each block at least two rows, against a float64 torch reference on
the GPU (itself compared with the oracle).  Tolerances as in test_gpu_logits_kl.py.
"""
import numpy as np
import pytest
import torch

import oracle
from test_gpu_logits_kl import case, host
from test_gpu_logprobs import EPS, TINY

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


def reference(z, ids, t, mask, t_lse, grad, tau=1.0):
    """KL [N] and gradient [N, V] in float64 (distinct ids, finite logits)."""
    x, at = z.double() / tau, ids.long()
    on = torch.ones(z.shape[0], dtype=torch.float64, device=z.device) if mask is None else mask.double()
    lq = x - torch.logsumexp(x, 1, keepdim=True)
    del x
    lp = t.double() / tau
    lp = lp - (torch.logsumexp(lp, 1) if t_lse is None else t_lse.double())[:, None]
    p, lq_s = lp.exp(), lq.gather(1, at)
    kl = (p * (lp - lq_s)).sum(1)
    dz = lq.exp_()
    if t_lse is not None:
        p_rest = (1 - p.sum(1)).clamp(min=0)
        dz.scatter_(1, at, 0.0)
        q_rest = dz.sum(1)
        kl += p_rest * (p_rest / q_rest).log()
        dz *= (1 - p_rest / q_rest)[:, None]
    dz.scatter_(1, at, lq_s.exp() - p)
    dz *= (on * grad / (on.sum().clamp(min=1) * tau))[:, None]
    return kl * on, dz


def close(got, ref, tol):
    bad = ((got.double() - ref).abs() - tol).max()
    assert float(bad) <= 0, f"off by {float(bad)} more than allowed"      # NaN fails


def close_grad(got, ref, dtype):
    close(got, ref, (EPS[dtype] + 1e-4) * ref.abs() + 1e-5 * ref.abs().amax(1, keepdim=True) + TINY[dtype])


def check(kd, z, ids, t, t_lse, mask, passes=("forward", "step")):
    N, V = z.shape
    kl, dz = reference(z, ids, t, mask, t_lse, 0.75)
    loss = kl.sum() / (N if mask is None else max(1, int(mask.sum())))
    tol = 4e-5 + 4e-7 * (kl + 40)
    g = torch.full((1,), 0.75, device="cuda")
    ws = kd.workspace(kd._abi.kd_logits_kl_workspace(N, V, ids.shape[1]), "cuda")
    got = torch.full((N,), -1.0, device="cuda")
    if "forward" in passes:
        total, stats, _ = kd.logits_kl_forward(z, ids, t, mask, 1.0, t_lse, ws=ws, kl_out=got)
        close(got, kl, tol)
        close(total[0], loss, tol.max())
        close_grad(kd.logits_kl_backward(z, ids, t, mask, stats, g, 1.0, t_lse, ws=ws), dz, z.dtype)
    if "step" in passes:
        got.fill_(-1.0)
        total, grad = kd.logits_kl_step(z, ids, t, mask, 1.0, t_lse, g, ws=ws, kl_out=got)
        close(got, kl, tol)
        close(total[0], loss, tol.max())
        close_grad(grad, dz, z.dtype)
    assert kd.device_error(ws)[0] == 0


def padded(z, ids, t, t_lse, mask):
    """Padding rows hold NaN, ids out of range, NaN teachers: nothing of them is looked at."""
    out = mask == 0
    clean = z.clone(), ids.clone(), t.clone(), None if t_lse is None else t_lse.clone()
    z[out], ids[out], t[out] = float("nan"), -100, float("nan")
    return clean


def stripes(N, period, kept=1, of=2):
    """Rows of a block lie `period` apart: the first `kept` of every `of` of them are valid."""
    return (torch.arange(N, device="cuda") // period % of < kept).to(torch.uint8)


@pytest.mark.parametrize("V", [64, 700, 4096])
@pytest.mark.parametrize("of", [2, 3])
def test_forward_with_a_padding_row_between_two_of_a_block(kd, cuda_device, V, of):
    """Without the rest class and without a gradient, short rows: valid, padding (or two), valid in one block."""
    blocks = 10 * torch.cuda.get_device_properties(0).multi_processor_count
    N = blocks * (2 * of + 1)
    z, ids, t, _ = case(N, V, 8, torch.bfloat16, seed=V)
    mask = stripes(N, blocks, 1, of)
    kl, dz = reference(z, ids, t, mask, None, 1.0)
    tol = 4e-5 + 4e-7 * (kl + 40)
    for _ in range(5):
        got = torch.full((N,), -1.0, device="cuda")
        _, stats, ws = kd.logits_kl_forward(z, ids, t, mask, kl_out=got)
        close(got, kl, tol)
        close_grad(kd.logits_kl_backward(z, ids, t, mask, stats, torch.ones(1, device="cuda"), ws=ws), dz, z.dtype)


def test_reference_is_the_oracle(cuda_device):
    for tail in (False, True):
        z, ids, t, t_lse = case(30, 300, 7, torch.float32, tail=tail, seed=3)
        mask = stripes(30, 3, 2, 3)
        kl, dz = reference(z, ids, t, mask, t_lse, 0.75)
        ref = oracle.logits_kl(host(z), host(ids), host(t), host(mask), 1.0, host(t_lse), 0.75)
        assert np.allclose(host(kl), ref.kl, atol=1e-12) and np.allclose(host(dz), ref.grad, atol=1e-14)


# rows of up to 16, 48, 96, 208 and 416 KB, and of more (clusters of two): how many resident blocks or
# clusters of an SM take them
VARIANTS = [
    ("10 blocks on an SM", 700, torch.float32, 10, 4597),
    ("10 blocks on an SM", 2053, torch.bfloat16, 10, 3500),
    ("8 blocks on an SM", 9001, torch.float16, 8, 2600),
    ("4 blocks on an SM", 32000, torch.bfloat16, 4, 1500),
    ("2 blocks on an SM", 70001, torch.bfloat16, 2, 800),
    ("one block on an SM", 150000, torch.bfloat16, 1, 400),
    ("clusters of two", 201088, torch.float32, 0.5, 230),
]


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("pattern", ["all", "random", "stripes"])
@pytest.mark.parametrize("V,dtype,per_sm,N", [v[1:] for v in VARIANTS], ids=[f"{v[0]}, V={v[1]}" for v in VARIANTS])
def test_every_variant_with_several_rows_a_block(kd, cuda_device, V, dtype, per_sm, N, pattern, tail):
    z, ids, t, t_lse = case(N, V, 20, dtype, tail=tail, seed=V)
    mask = None
    if pattern == "random":
        g = torch.Generator(device="cuda").manual_seed(2)
        mask = (torch.rand((N,), generator=g, device="cuda") < 0.7).to(torch.uint8)
    elif pattern == "stripes":
        mask = stripes(N, int(per_sm * torch.cuda.get_device_properties(0).multi_processor_count))
    check(kd, z, ids, t, t_lse, mask)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("V,dtype", [(515, torch.bfloat16), (9001, torch.float32)])
def test_padding_is_not_looked_at_in_any_pass(kd, cuda_device, V, dtype, tail):
    N = 3100 if V < 1000 else 1300
    z, ids, t, t_lse = case(N, V, 9, dtype, tail=tail)
    g = torch.Generator(device="cuda").manual_seed(5)
    mask = (torch.rand((N,), generator=g, device="cuda") < 0.6).to(torch.uint8)
    zc, idc, tc, lc = padded(z, ids, t, t_lse, mask)
    kl, dz = reference(zc, idc, tc, mask, lc, 0.75)
    one = torch.full((1,), 0.75, device="cuda")
    ws = kd.workspace(kd._abi.kd_logits_kl_workspace(N, V, 9), "cuda")
    got = torch.full((N,), -1.0, device="cuda")
    _, stats, _ = kd.logits_kl_forward(z, ids, t, mask, 1.0, t_lse, ws=ws, kl_out=got)
    close(got, kl, 4e-5 + 4e-7 * (kl + 40))
    close_grad(kd.logits_kl_backward(z, ids, t, mask, stats, one, 1.0, t_lse, ws=ws), dz, dtype)
    _, grad = kd.logits_kl_step(z, ids, t, mask, 1.0, t_lse, one, ws=ws, kl_out=got)
    close(got, kl, 4e-5 + 4e-7 * (kl + 40))
    close_grad(grad, dz, dtype)
    _, same = kd.logits_kl_step(z, ids, t, mask, 1.0, t_lse, one, ws=ws, grad_logits=z)   # in place
    assert same is z and torch.equal(z, grad)
    assert kd.device_error(ws)[0] == 0


@pytest.mark.parametrize("N", [8192, 8193, 20011])
def test_the_valid_rows_are_counted_either_way(kd, cuda_device, N):
    """Steps of up to 8192 rows count their valid rows in every block, longer ones ahead."""
    z, ids, t, t_lse = case(N, 128, 5, torch.bfloat16, tail=True)
    g = torch.Generator(device="cuda").manual_seed(8)
    check(kd, z, ids, t, t_lse, (torch.rand((N,), generator=g, device="cuda") < 0.5).to(torch.uint8))
