"""logits_kl (forward, backward, step) against the float64 oracle.

Tolerances, as in test_gpu_logprobs.py (fp32 sums of at most V / 512 + 14 sequential additions):
  kl, loss  : 4e-5 absolute (each class's log probability, weighted by p) plus 4e-7 of its parts
  gradients : the type's half unit in the last place with a binade of slack, 1e-4 of the value,
              1e-5 of the row's largest, half a subnormal step
"""
import math

import numpy as np
import pytest
import torch

import oracle
from test_gpu_logprobs import check_grad, framed, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


def case(N, V, K, dtype, tau=1.0, tail=False, seed=0, rest=(0.02, 0.5)):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn((N, V), generator=g, device="cuda") * 1.5
    ids = torch.argsort(torch.rand((N, V), generator=g, device="cuda"), dim=1)[:, :K]
    t = torch.randn((N, K), generator=g, device="cuda") * 2 + 3
    z.scatter_(1, ids, t + torch.randn((N, K), generator=g, device="cuda"))
    t_lse = None
    if tail:
        out = rest[0] + (rest[1] - rest[0]) * torch.rand((N,), generator=g, device="cuda")
        t_lse = torch.logsumexp(t / tau, 1) - torch.log1p(-out)
    return z.to(dtype), ids.to(torch.int32).contiguous(), t.contiguous(), t_lse


def host(x):
    return None if x is None else x.double().cpu().numpy() if x.is_floating_point() else x.cpu().numpy()


def check(kd, z, ids, t, t_lse=None, mask=None, tau=1.0, grad=0.75):
    """Forward + backward, and the single call, each against the oracle."""
    ref = oracle.logits_kl(host(z), host(ids), host(t), host(mask), tau, host(t_lse), grad)
    N, V = z.shape
    g = torch.full((1,), grad, device="cuda")
    tol = 4e-5 + 4e-7 * (np.abs(np.nan_to_num(ref.kl, posinf=0)) + 40)
    ws = kd.workspace(kd._abi.kd_logits_kl_workspace(N, V, ids.shape[1]), "cuda")
    kl = torch.full((N,), -1.0, device="cuda")
    loss, stats, _ = kd.logits_kl_forward(z, ids, t, mask, tau, t_lse, ws=ws, kl_out=kl)
    dz = kd.logits_kl_backward(z, ids, t, mask, stats, g, tau, t_lse, ws=ws)
    near(kl.cpu(), ref.kl, tol)
    near(loss.cpu(), [ref.loss], tol.max())
    check_grad(dz, ref.grad, z.dtype)
    kl2 = torch.full((N,), -1.0, device="cuda")
    loss2, dz2 = kd.logits_kl_step(z, ids, t, mask, tau, t_lse, g, ws=ws, kl_out=kl2)
    near(kl2.cpu(), ref.kl, tol)
    near(loss2.cpu(), [ref.loss], tol.max())
    check_grad(dz2, ref.grad, z.dtype)
    torch.cuda.synchronize()
    assert kd.device_error(ws)[0] == 0
    return dz2, ref


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("N,V,K,tau", [
    (1, 1, 1, 1.0),                # K = V: nothing outside the cache
    (2, 9, 3, 2.0),
    (3, 64, 64, 1.0),
    (40, 1003, 17, 0.7),
    (5, 4096, 100, 1.0),
    (3, 2051, 1024, 1.0),
    (4, 33000, 100, 1.5),
    (2, 201088, 100, 1.0),
])
def test_matches_oracle(kd, cuda_device, dtype, tail, N, V, K, tau):
    check(kd, *case(N, V, K, dtype, tau, tail, seed=V + K), tau=tau)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_padding(kd, cuda_device, tail, dtype):
    z, ids, t, t_lse = case(50, 700, 9, dtype, tail=tail)
    mask = (torch.rand(50, generator=torch.Generator().manual_seed(3)) < 0.6).to(torch.uint8).cuda()
    z[mask == 0] = math.nan        # padding is not looked at
    ids[mask == 0] = -100
    t[mask == 0] = math.nan
    keep = mask.bool().cpu().numpy()
    ws = kd.workspace(kd._abi.kd_logits_kl_workspace(50, 700, 9), "cuda")
    kl = torch.empty((50,), device="cuda")
    loss, dz = kd.logits_kl_step(z, ids, t, mask, 1.0, t_lse, None, ws=ws, kl_out=kl)
    assert kd.device_error(ws)[0] == 0
    ref = oracle.logits_kl(host(z)[keep], host(ids)[keep], host(t)[keep], t_lse=None if t_lse is None else host(t_lse)[keep])
    near(kl.cpu()[keep], ref.kl, 6e-5)
    near(loss.cpu(), [ref.loss], 6e-5)
    check_grad(dz[mask.bool()], ref.grad, dtype)
    assert not dz[mask == 0].any() and not kl[mask == 0].any()
    nothing = torch.zeros_like(mask)
    loss, dz = kd.logits_kl_step(z, ids, t, nothing, 1.0, t_lse)
    assert float(loss) == 0.0 and not dz.any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("lead,pad", [(1, 0), (0, 3), (5, 9)])
def test_any_alignment_and_nothing_outside_the_rows(kd, cuda_device, dtype, lead, pad):
    z, ids, t, t_lse = case(7, 2053, 12, dtype, tail=True)
    want, _ = check(kd, z, ids, t, t_lse)
    g = torch.full((1,), 0.75, device="cuda")
    buf, zv = framed(z, lead, pad)
    out, gv = framed(torch.zeros_like(z), 3, 2, fill=7.0)
    kd.logits_kl_step(zv, ids, t, None, 1.0, t_lse, g, grad_logits=gv)
    ref = oracle.logits_kl(host(z), host(ids), host(t), t_lse=host(t_lse), grad_loss=0.75)
    check_grad(gv, ref.grad, dtype)
    inside = torch.zeros_like(out, dtype=torch.bool)
    inside[3:3 + 7 * 2055].view(7, 2055)[:, :2053] = True
    assert (out[~inside] == 7.0).all()
    _, res = kd.logits_kl_step(zv, ids, t, None, 1.0, t_lse, g, grad_logits=zv)  # in place
    assert torch.equal(zv, gv) and int(torch.isnan(buf).sum()) == buf.numel() - 7 * 2053


@pytest.mark.parametrize("tail", [False, True])
def test_absent_repeated_and_missing_entries(kd, cuda_device, tail):
    z, ids, t, t_lse = case(5, 900, 8, torch.float32, tail=tail)
    t[0, 5:] = -math.inf
    ids[0, 5:] = -1                      # absent entries' ids are not looked at
    ids[1, 3] = ids[1, 0]                # a repeated id adds up
    ids[4, 1], ids[4, 7], ids[4, 2] = 0, 0, 0
    if not tail:
        t[2] = -math.inf                 # nothing cached: no KL, no gradient
    # repeated ids: the student's mass of S counts each id once
    ids_o = ids.clone()
    ids_o[0, 5:] = 0
    ref = oracle.logits_kl(host(z), host(ids_o), host(t), t_lse=host(t_lse), grad_loss=0.75)
    loss, stats, ws = kd.logits_kl_forward(z, ids, t, None, 1.0, t_lse)
    g = torch.full((1,), 0.75, device="cuda")
    check_grad(kd.logits_kl_backward(z, ids, t, None, stats, g, 1.0, t_lse, ws=ws), ref.grad, torch.float32)
    loss2, dz = kd.logits_kl_step(z, ids, t, None, 1.0, t_lse, g, ws=ws)
    check_grad(dz, ref.grad, torch.float32)
    near(loss.cpu(), [ref.loss], 6e-5)
    near(loss2.cpu(), [ref.loss], 6e-5)
    assert kd.device_error(ws)[0] == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("fill", ["inf", "lowest"])
def test_masked_vocabularies(kd, cuda_device, dtype, tail, fill):
    """Half the vocabulary masked outside the cached ids; an empty row; a cached id that is masked."""
    z, ids, t, t_lse = case(4, 3000, 10, dtype, tail=tail)
    low = -math.inf if fill == "inf" else torch.finfo(dtype).min
    drop = torch.rand((4, 3000), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") < 0.5
    drop.scatter_(1, ids.long(), False)
    z.masked_fill_(drop, low)
    check(kd, z, ids, t, t_lse)
    z[1] = low
    z[2, int(ids[2, 4])] = -math.inf     # KL is +inf there; its gradient is finite
    check(kd, z, ids, t, t_lse)


@pytest.mark.parametrize("tail", [False, True])
@pytest.mark.parametrize("where", ["cached", "other"])
def test_nan_and_infinity_stay_in_their_rows(kd, cuda_device, tail, where):
    z, ids, t, t_lse = case(5, 2500, 9, torch.bfloat16, tail=tail)
    other = [c for c in range(20) if c not in ids[1].tolist() and c not in ids[3].tolist()][0]
    z[1, int(ids[1, 2]) if where == "cached" else other] = math.nan
    z[3, int(ids[3, 0]) if where == "cached" else other] = math.inf
    kl = torch.empty((5,), device="cuda")
    loss, dz = kd.logits_kl_step(z, ids, t, None, 1.0, t_lse, kl_out=kl)
    assert math.isnan(float(loss)) and torch.isnan(kl[[1, 3]]).all() and torch.isnan(dz[[1, 3]]).any(1).all()
    rows = [0, 2, 4]
    ref = oracle.logits_kl(host(z)[rows], host(ids)[rows], host(t)[rows],
                           t_lse=None if t_lse is None else host(t_lse)[rows], grad_loss=3 / 5)
    near(kl.cpu()[rows], ref.kl, 6e-5)
    check_grad(dz[rows], ref.grad, torch.bfloat16)


@pytest.mark.parametrize("q_rest", [1e-3, 1e-6, 1e-12, 1e-30])
def test_rest_class_keeps_its_digits(kd, cuda_device, q_rest):
    """The student's mass outside the cache is tiny: it is summed alone, not as 1 minus the cached mass."""
    V, K = 5000, 50
    z, ids, t, t_lse = case(3, V, K, torch.float32, tail=True)
    outside = torch.ones((3, V), dtype=torch.bool, device="cuda").scatter_(1, ids.long(), False)
    lse_s = torch.logsumexp(z.gather(1, ids.long()).double(), 1)
    lse_o = torch.logsumexp(z.double().masked_fill(~outside, -math.inf), 1)
    z = torch.where(outside, (z.double() + (lse_s - lse_o + math.log(q_rest))[:, None]).float(), z)
    check(kd, z, ids, t, t_lse)


def test_rest_class_without_mass(kd, cuda_device):
    """t_lse of the cached logits alone (nothing dropped): the same as without it, off S included."""
    z, ids, t, _ = case(4, 800, 800, torch.float32)
    check(kd, z, ids, t, torch.logsumexp(t, 1))


def test_bad_id_is_reported_and_left_out(kd, cuda_device):
    z, ids, t, _ = case(5, 300, 6, torch.float32)
    ids[3, 2] = 300
    ws = kd.workspace(kd._abi.kd_logits_kl_workspace(5, 300, 6), "cuda")
    kd.logits_kl_step(z, ids, t, ws=ws)
    assert kd.device_error(ws) == (kd._abi.KD_ERR_DEVICE, 3)
    assert kd.device_error(ws)[0] == 0


def test_row_offsets_past_32_bits(kd, cuda_device):
    N, V, ld = 1030, 1000, 1 << 21
    buf = torch.empty(((N - 1) * ld + V + 1,), dtype=torch.bfloat16, device="cuda")
    src, ids, t, t_lse = case(N, V, 10, torch.bfloat16, tail=True)
    z = buf.as_strided((N, V), (ld, 1), 1)
    z.copy_(src)
    loss, want = kd.logits_kl_step(src, ids, t, None, 1.0, t_lse)
    loss2, _ = kd.logits_kl_step(z, ids, t, None, 1.0, t_lse, grad_logits=z)
    assert abs(float(loss) - float(loss2)) <= 1e-6
    # the two lay out their sums differently: equal to one rounding
    assert ((z.float() - want.float()).abs() <= 2.0 ** -7 * want.float().abs() + 1e-9).all()


@pytest.mark.parametrize("N,V", [(1, 100000), (70, 6000)])
def test_repeats_are_bit_identical_on_any_stream(kd, cuda_device, N, V):
    z, ids, t, t_lse = case(N, V, 30, torch.bfloat16, tail=True)
    ids[0, 1] = ids[0, 0]
    ids[0, 2] = ids[0, 0]
    loss, dz = kd.logits_kl_step(z, ids, t, None, 1.0, t_lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        loss2, dz2 = kd.logits_kl_step(z, ids, t, None, 1.0, t_lse)
    torch.cuda.synchronize()
    assert torch.equal(loss, loss2) and torch.equal(dz, dz2)


def test_matches_the_fused_loss(kd, cuda_device):
    """The same loss from hidden states: H = rows of the identity make the logits W's columns."""
    z, ids, t, _ = case(128, 1000, 16, torch.bfloat16)
    H = torch.eye(128, dtype=torch.bfloat16, device="cuda")
    W = z.T.contiguous()
    a = kd.fused_kl(H, W, ids, t, chunk=128)
    b = kd.logits_kl(z, ids, t)
    assert abs(float(a) - float(b)) <= 6e-5


@pytest.mark.parametrize("tail", [False, True])
def test_gradient_matches_differences(kd, cuda_device, tail):
    """Central differences of the fp32 forward, step 1/16 (truncation below 7e-4)."""
    z, ids, t, t_lse = case(2, 60, 5, torch.float32, tail=tail)
    zr = z.clone().requires_grad_(True)
    kd.logits_kl(zr, ids, t, None, 1.0, t_lse).backward()
    step = 1.0 / 16
    for v in [int(ids[0, 0]), int(ids[0, 4]), 0, 59]:
        hi, lo = z.clone(), z.clone()
        hi[0, v] += step
        lo[0, v] -= step
        slope = (float(kd.logits_kl(hi, ids, t, None, 1.0, t_lse)) - float(kd.logits_kl(lo, ids, t, None, 1.0, t_lse)))
        assert abs(float(zr.grad[0, v]) - slope / (2 * step)) < 3e-3


def test_from_cache_to_gradient(kd, cuda_device):
    """A cache built by topk_cache with its logsumexp feeds the rest class; a student equal to the teacher has
    KL 0 and no gradient."""
    g = torch.Generator(device="cuda").manual_seed(0)
    zt = (torch.randn((16, 4096), generator=g, device="cuda") * 2).to(torch.bfloat16)
    ids, vals, lse = kd.topk_cache(zt, 32, with_lse=True)
    loss, dz = kd.logits_kl_step(zt, ids, vals, t_lse=lse)
    assert abs(float(loss)) <= 1e-5 and dz.abs().max() <= 1e-6
