"""fused_cross_entropy where its numbers end: logits far from zero and beyond 2^64, columns and labels at -inf.

One position a coordinate: H has a single 1 (or one power of two) in each row, so a row's logits are a column of W
times it, exact bf16 numbers, and grad_W holds dZ itself.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def close(got, want, each):
    """dZ: rounded to bf16 once (2^-8 of the entry), 2^-11 of a probability for its 16-bit distance, 1e-6 the rest."""
    assert torch.isfinite(got).all()
    assert ((got.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -11) * want.abs() + each).all()


@pytest.mark.parametrize("size", [1e4, 1e5, 1e6, 1e9, 1e15])
@pytest.mark.parametrize("smooth", [0.0, 0.1])
def test_equal_logits_far_from_zero(kd, cuda_device, size, smooth):
    """Row n has n + 2 logits at its largest, so far from zero that lse = size + ln(n + 2) is not an fp32 number:
    each of them has a probability of 1 / (n + 2)."""
    N, V = 8, 1000
    H = torch.eye(N, device="cuda").to(torch.bfloat16)
    W = (torch.randn((V, N), generator=gen(3), device="cuda") * 0.1 * size).clamp(max=0.5 * size)
    for n in range(N):
        W[torch.arange(n + 2) * 90 + 3 * n, n] = size
    W = W.to(torch.bfloat16)
    labels = torch.arange(N, device="cuda", dtype=torch.int32) * 3
    labels[::2] += 1                            # half of the labels among them
    _, _, gW = kd.fused_cross_entropy_step(H, W, labels, label_smoothing=smooth)
    want = W.double().T.softmax(1) - smooth / V
    want[torch.arange(N), labels.long()] -= 1 - smooth
    close(gW.T, want / N, 1e-6)


@pytest.mark.parametrize("size", [1e18, 3e19, 1e25, 1e37])
def test_logits_whose_squares_overflow(kd, cuda_device, size):
    N, V = 8, 1000
    H = torch.eye(N, device="cuda").to(torch.bfloat16)
    W = (torch.randn((V, N), generator=gen(1), device="cuda") * size).to(torch.bfloat16)
    labels = torch.arange(0, 8 * N, 8, device="cuda", dtype=torch.int32)
    each = torch.empty((N,), device="cuda")
    _, gH, gW = kd.fused_cross_entropy_step(H, W, labels, loss_out=each, grad_H_fp32=True)
    z = W.double().T
    want = z.softmax(1)
    want[torch.arange(N), labels.long()] -= 1
    losses = z.logsumexp(1) - z.gather(1, labels.long()[:, None])[:, 0]
    assert ((each.double() - losses).abs() <= 1e-6 * z.abs().amax(1)).all()
    close(gW.T, want / N, 1e-6)
    full = want / N @ W.double()
    assert torch.isfinite(gH).all() and ((gH.double() - full).abs() <= 2 * 2.0 ** -8 * (want.abs() / N @ W.double().abs())).all()


@pytest.mark.parametrize("V", [300, 1000])
def test_columns_of_nothing_but_minus_infinity(kd, cuda_device, V):
    """Columns 128 .. 255 overflow to -inf for every position: no probability, no gradient, the others as ever."""
    N, d = 6, 16
    H = torch.zeros((N, d), device="cuda")
    H[:, :N] = torch.eye(N)
    H[:, 8] = 1e20
    W = torch.randn((V, d), generator=gen(2), device="cuda") * 2
    W[:, 8] = 0
    W[128:256, 8] = -1e20
    H, W = H.to(torch.bfloat16), W.to(torch.bfloat16)
    labels = torch.tensor([0, 5, 127, 256, 270, 299], device="cuda", dtype=torch.int32)
    loss, gH, gW = kd.fused_cross_entropy_step(H, W, labels, grad_H_fp32=True)
    z = H.double() @ W.double().T
    lp = z.log_softmax(1)
    dz = lp.exp()
    dz[torch.arange(N), labels.long()] -= 1
    dz /= N
    assert abs(float(loss) + float(lp.gather(1, labels.long()[:, None]).mean())) < 1e-5
    assert not gW[128:256].any()
    close(gW[:, :N].T, dz, 1e-6)
    keep = [i for i in range(d) if i != 8]
    bound = 2 * 2.0 ** -8 * (dz.abs() @ W.double().abs())
    assert torch.isfinite(gH).all() and ((gH.double() - dz @ W.double()).abs() <= bound + 1e-6)[:, keep].all()


@pytest.mark.parametrize("smooth", [0.0, 0.1])
def test_label_at_minus_infinity(kd, cuda_device, smooth):
    """A logit that overflows to -inf has no probability: as a label its loss is +inf, the gradients stay finite."""
    N, V, d = 4, 500, 16
    H = torch.zeros((N, d), device="cuda")
    H[:, :N] = torch.eye(N)
    H[:2, 8] = 1e20
    W = torch.randn((V, d), generator=gen(4), device="cuda")
    W[:, 8] = 0
    W[300, 8] = -1e20
    H, W = H.to(torch.bfloat16), W.to(torch.bfloat16)
    labels = torch.tensor([300, 7, 300, 8], device="cuda", dtype=torch.int32)
    each = torch.empty((N,), device="cuda")
    loss, gH, gW = kd.fused_cross_entropy_step(H, W, labels, label_smoothing=smooth, loss_out=each)
    # with smoothing a logit of -inf is in every loss of its row, by e / V
    assert each[0] == INF and loss[0] == INF and torch.isfinite(each[2:]).all()
    assert torch.isfinite(each[1]) if smooth == 0 else each[1] == INF
    z = H.double() @ W.double().T
    dz = z.softmax(1) - smooth / V
    dz[torch.arange(N), labels.long()] -= 1 - smooth
    close(gW[:, :N].T, dz / N, 1e-6)
