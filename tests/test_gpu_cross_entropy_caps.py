"""fused_cross_entropy's gradients under softcaps from 1e-6 to beyond the logits, entry by entry.

H's rows are unit vectors, so a position's logits are a column of W (exact bf16 numbers) and grad_W is dZ, every
entry of which is compared.  Its error bound, with t = z'/c: the rounding of dZ to bf16 (2^-8 of it); what the 16
bits that z' is kept in (and fp32's roundings, 2^-20 of c) leave open of it, dz, makes p dz; what they
leave open of the slope 1 - t^2 is 2 dt.
  c <= 16  |t| = 1 - w^2, w in steps of 1 / 32767: off by half of one, h = 2^-16, so dt = 2 w h + h^2.
  c > 16   steps of 1 / 2048 below the largest of 128 columns: dz = 2^-12, dt = dz / c.  28 and further below, where
           p is below e^-28 of that column's and only known to be: t = 2 w^2 - 1, w in steps of 1 / 8191, h = 2^-14,
           the slope 4 w^2 (1 - w^2) off by 8 w h + 8 h^2 at most.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


def inputs(cap, V):
    g = torch.Generator(device="cuda").manual_seed(int(V))
    spread = torch.tensor([0.3 * cap, cap, 2 * cap, 4 * cap, 8 * cap, 70.0, 1.5, 0.01], device="cuda")
    W = torch.randn((V, 8), generator=g, device="cuda") * spread
    W[100:116, 4] = 6 * cap       # saturated at the top, in a group of its own spread
    W[200:230, 1] = -5 * cap
    W[:128, 7] = torch.linspace(-70, 70, 128, device="cuda")   # both ends in one group of 128 columns
    labels = torch.tensor([3, 130, V - 1, 7, 110, 200, 1, 64], device="cuda", dtype=torch.int32)
    return torch.eye(8, device="cuda").to(torch.bfloat16), W.to(torch.bfloat16), labels


def reference(W, labels, cap, smooth, z_loss):
    """losses [N], dZ [N, V] of the sum of losses, and its bound."""
    x = W.double().T / cap
    t = x.tanh()
    z = cap * t
    rest = 2 / ((2 * x.abs()).exp() + 1)           # 1 - |t|
    slope = rest * (2 - rest)
    V, rows = z.shape[1], torch.arange(8)
    lse = z.logsumexp(1, keepdim=True)
    a = (z - lse).exp() * (1 + 2 * z_loss * lse)
    dz = a - smooth / V
    y = labels.long()
    losses = lse[:, 0] - (1 - smooth) * z[rows, y] - smooth * z.mean(1) + z_loss * lse[:, 0] ** 2
    off_z = cap * 2.0 ** -20 + 2e-5 * min(1.0, cap)
    if cap <= 16:
        h = 2.0 ** -16
        dt = 2 * rest.sqrt() * h + h * h + 2.0 ** -20
        off_z, off_slope, lost = cap * dt + off_z, 2 * dt, 0.0
    else:
        pad = -V % 128
        blocks = torch.nn.functional.pad(z, (0, pad), value=-math.inf).view(8, -1, 128)
        far = (blocks.amax(2, keepdim=True) - blocks).view(8, -1)[:, :V] > 28 - 2.0 ** -12
        off_z = 2.0 ** -12 + off_z
        h, w = 2.0 ** -14, ((1 + t) / 2).sqrt()
        off_slope = torch.where(far, 8 * w * h + 8 * h * h, 2 * off_z / cap) + 2.0 ** -20
        lost = far * math.exp(-28) * slope * (1 + 2 * z_loss * lse).abs()
    bound = 1.02 * slope * a.abs() * off_z + (a.abs() + smooth / V) * off_slope + lost
    # the label's own entry comes from its fp32 logit
    bound[rows, y] = (slope * a.abs() * (cap * 2.0 ** -20 + 2e-5) + 2.0 ** -19)[rows, y]
    dz[rows, y] -= 1 - smooth
    dz *= slope
    return losses, dz, bound + 2.0 ** -8 * dz.abs() + 1e-9 * dz.abs().amax(1, keepdim=True)


@pytest.mark.parametrize("cap", [1e-6, 1e-4, 1e-3, 0.01, 0.1, 0.5, 1.0, 4.0, 15.9, 16.0, 16.1, 30.0, 50.0, 64.0, 65.0,
                                 300.0, 1e5, 1e30])
@pytest.mark.parametrize("smooth,z_loss", [(0.0, 0.0), (0.1, 0.0), (0.1, 1e-3)])
def test_every_entry(kd, cuda_device, cap, smooth, z_loss):
    V = 1000
    H, W, labels = inputs(min(cap, 300.0), V)
    each = torch.empty((8,), device="cuda")
    _, gH, gW = kd.fused_cross_entropy_step(H, W, labels, label_smoothing=smooth, z_loss=z_loss, softcap=cap,
                                            loss_out=each, grad_H_fp32=True)
    losses, dz, bound = reference(W, labels, cap, smooth, z_loss)
    # beside the cap's roundings those of fp32 numbers as large as the loss (its square and its sums: four halves of
    # 2^-23) and the logits (|z| reaches 8000 under the wide caps, lse is no smaller; four again, times the loss's slope in lse)
    most = (W.double().T.abs().amax(1)).clamp(max=cap)
    tol = (2e-5 + min(cap, 300.0) * 2.0 ** -20) * (1 + 2 * z_loss * 300)
    tol = tol + 2.0 ** -22 * (losses.abs() + most * (1 + 2 * z_loss * most))
    assert ((each.double() - losses).abs() <= tol).all()
    worst = ((gW.double().T * 8 - dz).abs() / bound).amax(1)
    assert torch.isfinite(gW).all() and float(worst.max()) <= 1.0, worst.tolist()
    limit = bound @ W.double().abs() + 2.0 ** -20 * (dz.abs() @ W.double().abs())
    assert torch.isfinite(gH).all() and ((gH.double() * 8 - dz @ W.double()).abs() <= limit).all()


@pytest.mark.parametrize("cap", [1e-6, 1e-3])
def test_no_gradient_at_the_cap(kd, cuda_device, cap):
    """Logits of +-1.5 far beyond the cap: a slope of 0, and no gradient at all."""
    H, W, labels = inputs(cap, 600)
    W = torch.where(torch.arange(600, device="cuda")[:, None] % 3 == 0, 1.5, -1.5).expand(600, 8).to(torch.bfloat16)
    _, gH, gW = kd.fused_cross_entropy_step(H, W, labels % 600, label_smoothing=0.1, softcap=cap)
    assert not gW.any() and not gH.any()
