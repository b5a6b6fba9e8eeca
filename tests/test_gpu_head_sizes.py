"""The cross entropy and the 8-bit calls at the ends of their sizes: many positions and few columns, the other way
round, deep reductions, logits whose offsets pass 32 bits, caches of next to nothing.

Losses and gradients: as in test_gpu_cross_entropy (2.5e-4, and the rounding of bf16 dZ, 2^-8 + 2^-10 of the parts'
magnitudes; fp32 outputs).  8-bit products and caches are equal to their definitions.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def case(N, d, V, seed):
    g = gen(seed)
    H = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn((V, d), generator=g, device="cuda") * (1.5 / d ** 0.5)).to(torch.bfloat16)
    labels = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    return H, W, labels


@pytest.mark.parametrize("N,d,V,chunk", [
    (70001, 8, 33, 70016),       # one chunk of many positions
    (70001, 8, 33, 4096),
    (3, 8, 400001, 128),         # few positions, many columns
    (40, 16384, 70, 128),        # a deep reduction of the logits
    (9, 8, 1, 128),              # a vocabulary of one has no loss
])
@pytest.mark.parametrize("smooth", [0.0, 0.1])
def test_cross_entropy(kd, cuda_device, N, d, V, chunk, smooth):
    H, W, labels = case(N, d, V, N)
    loss, gH, gW = kd.fused_cross_entropy_step(H, W, labels, chunk=chunk, label_smoothing=smooth, grad_H_fp32=True)
    z = H.double() @ W.double().T
    lp = z.log_softmax(1)
    y = labels.long()[:, None]
    ref = -(1 - smooth) * lp.gather(1, y)[:, 0] - smooth * lp.mean(1)
    dz = lp.exp() - smooth / V
    size = lp.exp() + smooth / V
    dz.scatter_add_(1, y, torch.full_like(ref, smooth - 1)[:, None])
    size.scatter_(1, y, dz.abs().gather(1, y) + 1e-3)
    assert abs(float(loss) - float(ref.mean())) <= 2.5e-4
    part = (2.0 ** -8 + 2.0 ** -10) / N
    assert ((gH.double() - dz @ W.double() / N).abs() <= part * (size @ W.double().abs()) + 1e-12).all()
    # the sum over the positions rounds too: 2^-24 of the magnitudes for each of the chunks, and the tensor cores' cut-off
    # additions of 16 positions, 2^-23
    sums = (N / 16 * 2.0 ** -23 + (N / chunk + 1) * 2.0 ** -24) / N
    assert ((gW.double() - dz.T @ H.double() / N).abs() <= (part + sums) * (size.T @ H.double().abs()) + 1e-12).all()


def test_cross_entropy_offsets_past_32_bits(kd, cuda_device):
    """A chunk's logits and dZ of more than 2^32 entries: the same as in chunks of 2^29, and as the definition at their end."""
    N, d, V = 8192, 16, 600000
    H, W, labels = case(N, d, V, 1)
    labels[-1] = V - 1
    each = torch.empty((N,), device="cuda")
    loss, gH, gW = kd.fused_cross_entropy_step(H, W, labels, chunk=8192, loss_out=each, grad_H_fp32=True)
    each2 = torch.empty((N,), device="cuda")
    loss2, gH2, gW2 = kd.fused_cross_entropy_step(H, W, labels, chunk=1024, loss_out=each2, grad_H_fp32=True)
    assert torch.equal(each, each2) and torch.equal(loss, loss2)
    # the reductions are split and chunked otherwise.  Each step of 16 cuts off up to 2^-23 of the sum so far, which is
    # below the terms' magnitudes: N / 16 steps for grad_W; V / 16 for grad_H, whose rows of |dZ| add up to 2 / N at most
    assert float((gH - gH2).abs().max()) <= V / 16 * 2.0 ** -23 * 2 / N * float(W.abs().max())
    most = torch.zeros((V, d), device="cuda")
    for a in range(0, N, 1024):
        p = (H[a:a + 1024].float() @ W.float().T).softmax(1)
        most += p.scatter_add_(1, labels[a:a + 1024].long()[:, None], torch.ones((1024, 1), device="cuda")).T @ H[a:a + 1024].float().abs()
    assert ((gW - gW2).abs() <= (N / 16 * 2.0 ** -23 + 8 * 2.0 ** -24) * 1.01 * most / N).all()
    z = H[-64:].double() @ W.double().T
    lp = z.log_softmax(1)
    y = labels[-64:].long()[:, None]
    assert ((each[-64:].double() + lp.gather(1, y)[:, 0]).abs() <= 2.5e-4).all()
    dz = lp.exp().scatter_add_(1, y, torch.full((64, 1), -1.0, dtype=torch.float64, device="cuda"))
    bound = (2.0 ** -8 + 2.0 ** -10) * (dz.abs() @ W.double().abs()) + 1e-3 * W.double().abs().amax()
    assert ((gH[-64:].double() * N - dz @ W.double()).abs() <= bound).all()


def product(A, sa, B, sb, dtype):
    total = A.double() @ B.double().T
    assert float(total.abs().max()) < 2 ** 24
    return ((total.float() * sa[:, None]) * sb[None, :]).to(dtype)


@pytest.mark.parametrize("M,N,K,pad", [(300001, 5, 32, 0), (300001, 5, 32, 3), (20, 40, 65536, 0), (300, 40, 65536, 5),
                                       (1, 1, 65536, 1), (4, 3, 65536, 0), (4, 3, 16384, 1), (100, 1, 1, 0), (2, 70000, 1, 0)])
def test_products(kd, cuda_device, M, N, K, pad):
    g = gen(M + N)
    most = 128 if K <= 1024 else 16
    A = torch.randint(-most, most, (M, K + pad), generator=g, device="cuda", dtype=torch.int8)[:, :K]
    B = torch.randint(-most, most, (N, K + pad), generator=g, device="cuda", dtype=torch.int8)[:, :K]
    sa, sb = torch.rand((M,), generator=g, device="cuda"), torch.rand((N,), generator=g, device="cuda")
    assert torch.equal(kd.gemm_int8(A, sa, B, sb, out_dtype=torch.float32), product(A, sa, B, sb, torch.float32))


@pytest.mark.parametrize("N,d,V,K,chunk", [(1, 1, 1, 1, 1), (5, 3, 7, 7, 2), (9, 16, 9, 1, 4), (130, 8, 1024, 1024, 64),
                                           (300, 32, 5000, 1000, 5000), (3000, 8, 300, 5, 7)])
def test_caches(kd, cuda_device, N, d, V, K, chunk):
    """The same as topk_cache of the product's bf16 logits, with their logsumexp and dropped mass."""
    g = gen(N + V)
    H, W = torch.randn((N, d), generator=g, device="cuda"), torch.randn((V, d), generator=g, device="cuda")
    h8, hs = kd.quantize_int8(H)
    w8, ws = kd.quantize_int8(W)
    z = torch.zeros((N, (V + 7) // 8 * 8), dtype=torch.bfloat16, device="cuda")
    z[:, :V] = product(h8, hs, w8, ws, torch.bfloat16)
    ids, vals, lse, dropped = kd.teacher_topk_int8(h8, hs, w8, ws, K, chunk=chunk, with_lse=True, with_dropped=True)
    want, wid = torch.sort(z[:, :V], dim=1, descending=True, stable=True)
    assert torch.equal(vals, want[:, :K].float()) and torch.equal(ids.long(), wid[:, :K])
    ref = z[:, :V].double().logsumexp(1)
    assert ((lse.double() - ref).abs() < 1e-5 * (1 + ref.abs())).all()
    rest = 1 - (vals.double() - ref[:, None]).exp().sum(1)
    assert ((dropped.double() - rest).abs() < 1e-5).all()


def test_cache_of_a_row_without_numbers(kd, cuda_device):
    """A hidden state with a NaN quantises to a scale of NaN: its logits are NaN, the others' caches are as ever."""
    g = gen(3)
    H, W = torch.randn((6, 32), generator=g, device="cuda"), torch.randn((500, 32), generator=g, device="cuda")
    h8, hs = kd.quantize_int8(H)
    w8, ws = kd.quantize_int8(W)
    good = kd.teacher_topk_int8(h8, hs, w8, ws, 9)
    H[2, 5] = float("nan")
    b8, bs = kd.quantize_int8(H)
    ids, vals = kd.teacher_topk_int8(b8, bs, w8, ws, 9)
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(ids[keep], good[0][keep]) and torch.equal(vals[keep], good[1][keep])
    assert torch.isnan(vals[2]).all() and kd.device_error(kd.control_block())[0] == 0
