"""fused_cross_entropy (hidden states to mean cross entropy and gradients) against its definition in float64 on
identical bf16 inputs.

Tolerances.  A logit is a sum of d exact bf16 products in fp32; taken as a random walk its error is below
2^-23 sqrt(d) sum |h w|, at most 1e-4 here (d <= 2048, |h| ~ 1, |w| ~ 1.5 / sqrt(d)), the logsumexp's is no larger
and a softcap adds a few roundings of c = 30 (1e-5):
  losses, lse : 2.5e-4 (1 + 2 z_loss |lse|) absolute (two such logits, and the square's slope)
  gradients   : dZ carries its own rounding to bf16 (half a step: 2^-8 of the entry), that of its 16-bit logit
                (2^-12) and of the logits above (2.5e-4 < 2^-11), so every entry of a product may be off by
                (2^-8 + 2^-10) |dZ| |W|, plus the rounding of a bf16 output (2^-8 of it).  The parts of dZ are
                bounded by their sum of magnitudes, p (1 + 2 l lse) + e / V + [v = y], since they may cancel.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

IGNORE = -100


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


def case(N, d, V, valid=1.0, seed=0, lean=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    W = (torch.randn((V, d), generator=g, device="cuda") * (1.5 / d ** 0.5)).to(torch.bfloat16)
    labels = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    H = torch.randn((N, d), generator=g, device="cuda")
    some = (torch.rand((N, 1), generator=g, device="cuda") < 0.5).float()
    H = (H + lean * some * W[labels.long()].float()).to(torch.bfloat16)
    labels[torch.rand((N,), generator=g, device="cuda") >= valid] = IGNORE
    return H, W, labels


def reference(H, W, labels, mask=None, smooth=0.0, z_loss=0.0, cap=0.0, g=1.0):
    """loss, losses, lse, grad_H, grad_W and the two gradients' error bounds before output rounding."""
    on = labels != IGNORE
    if mask is not None:
        on &= mask != 0
    Hd = torch.where(on[:, None], H.double(), 0.0)
    Wd = W.double()
    V = Wd.shape[0]
    z = Hd @ Wd.T
    slope = torch.ones_like(z)
    if cap:
        t = (z / cap).tanh()
        z, slope = cap * t, 1 - t * t
    lse = z.logsumexp(1)
    y = torch.where(on, labels, 0).long()[:, None]
    losses = lse - (1 - smooth) * z.gather(1, y)[:, 0] - smooth * z.mean(1) + z_loss * lse ** 2
    keep = on.double()
    n = max(1.0, float(keep.sum()))
    a = (z - lse[:, None]).exp() * (1 + 2 * z_loss * lse[:, None])
    hot = torch.zeros_like(z).scatter_(1, y, 1 - smooth)
    G = (keep * g / n)[:, None]
    dz = G * (a - smooth / V - hot) * slope
    size = G.abs() * (a.abs() + smooth / V + hot) * slope
    # the label's own entry is not taken from its 16-bit logit: its parts may cancel, its error is fp32's
    size.scatter_(1, y, dz.abs().gather(1, y) + G.abs() * 1e-3 * slope.gather(1, y))
    part = 2.0 ** -8 + 2.0 ** -10
    return (losses * keep).sum() / n, losses * keep, lse * keep, dz @ Wd, dz.T @ Hd, part * (size @ Wd.abs()), \
        part * (size.T @ Hd.abs())


def near(got, ref, bound, bf16):
    limit = bound + (2.0 ** -8 * ref.abs() if bf16 else 0.0) + 1e-30
    worst = ((got.double() - ref).abs() / limit).max()
    assert torch.isfinite(got).all() and float(worst) <= 1.0, float(worst)


def check(kd, H, W, labels, mask=None, chunk=4096, smooth=0.0, z_loss=0.0, cap=0.0, g=None, bf16=False):
    N, d = H.shape
    opt = dict(chunk=chunk, label_smoothing=smooth, z_loss=z_loss, softcap=cap)
    grad = None if g is None else torch.full((1,), g, device="cuda")
    loss_r, each_r, lse_r, gH_r, gW_r, bH, bW = reference(H, W, labels, mask, smooth, z_loss, cap, 1.0 if g is None else g)
    each = torch.full((N,), 7.0, device="cuda")
    ws = kd.workspace(kd._abi.kd_fused_cross_entropy_workspace(N, d, W.shape[0], chunk, 1), "cuda")
    loss, gH, gW = kd.fused_cross_entropy_step(H, W, labels, mask, **opt, grad_loss=grad, ws=ws, loss_out=each,
                                               grad_H_fp32=not bf16, grad_W_bf16=bf16)
    assert kd.device_error(ws)[0] == 0
    tol = 2.5e-4 * (1 + 2 * z_loss * lse_r.abs())
    assert ((each.double() - each_r).abs() <= tol).all()
    assert abs(float(loss) - float(loss_r)) <= float(tol.max())
    near(gH, gH_r, bH, bf16)
    near(gW, gW_r, bW, bf16)
    each2 = torch.full((N,), 7.0, device="cuda")
    loss2, lse, _ = kd.fused_cross_entropy_forward(H, W, labels, mask, **opt, loss_out=each2)
    assert torch.equal(loss2, loss) and torch.equal(each2, each)
    assert ((lse.double() - lse_r).abs() <= 2.5e-4).all()
    return loss, each, gH, gW


@pytest.mark.parametrize("N,d,V,chunk", [
    (1, 8, 1, 128),            # a vocabulary of one
    (1, 64, 1000, 128),
    (3, 8, 2, 128),
    (5, 72, 257, 128),         # one column in the second tile
    (128, 256, 4096, 4096),
    (129, 136, 1001, 256),     # one row in the second row tile
    (300, 72, 1000, 128),      # three chunks, the last short
    (600, 320, 2100, 256),
    (257, 2048, 3001, 1024),
    (513, 64, 320, 512),       # one row in the second chunk
])
def test_matches_definition(kd, cuda_device, N, d, V, chunk):
    check(kd, *case(N, d, V, seed=N + V), chunk=chunk)


@pytest.mark.parametrize("smooth,z_loss,cap,g", [
    (0.1, 0.0, 0.0, None), (0.0, 1e-2, 0.0, None), (0.0, 0.0, 5.0, None), (0.0, 0.0, 30.0, 0.3), (0.1, 1e-4, 30.0, -2.0),
    (0.9, 0.1, 2.0, 1024.0)])
@pytest.mark.parametrize("N,d,V,valid", [(70, 64, 500, 1.0), (300, 200, 1111, 0.6)])
def test_options(kd, cuda_device, N, d, V, valid, smooth, z_loss, cap, g):
    check(kd, *case(N, d, V, valid, seed=N), smooth=smooth, z_loss=z_loss, cap=cap, g=g)


@pytest.mark.parametrize("valid", [0.02, 0.3, 0.5, 0.97])
@pytest.mark.parametrize("chunk", [128, 512])
def test_ignored_positions(kd, cuda_device, valid, chunk):
    H, W, labels = case(700, 128, 900, valid, seed=3)
    off = labels == IGNORE
    H[off] = float("nan")      # never read
    loss, each, gH, gW = check(kd, H, W, labels, chunk=chunk)
    assert not each[off].any() and not gH[off].any()


def test_mask_and_ignored_labels_together(kd, cuda_device):
    H, W, labels = case(400, 64, 700, 0.7, seed=5)
    mask = (torch.rand(400, generator=torch.Generator().manual_seed(1)) < 0.6).to(torch.uint8).cuda()
    labels[mask == 0] = 2 ** 31 - 1   # not looked at
    check(kd, H, W, labels, mask)
    got, _, _ = kd.fused_cross_entropy_forward(H, W, torch.where(labels == IGNORE, 5, labels), mask, ignore_index=5)
    keep = (labels != IGNORE) & (labels != 5) & (mask != 0)
    want = reference(H, W, torch.where(keep, labels, IGNORE))[0]
    assert abs(float(got) - float(want)) <= 2.5e-4


@pytest.mark.parametrize("N", [1, 129, 300])
def test_nothing_valid(kd, cuda_device, N):
    H, W, labels = case(N, 64, 500)
    labels[:] = IGNORE
    H[:] = float("inf")
    each = torch.full((N,), 7.0, device="cuda")
    for bf16 in (False, True):
        loss, gH, gW = kd.fused_cross_entropy_step(H, W, labels, chunk=512, loss_out=each, grad_W_bf16=bf16)
        assert float(loss) == 0 and not each.any() and not gH.any() and not gW.any()
    base = torch.randn((500, 64), device="cuda")
    _, _, gW = kd.fused_cross_entropy_step(H, W, labels, chunk=128, grad_W=base.clone())
    assert torch.equal(gW, base)


def test_gradient_kinds(kd, cuda_device):
    H, W, labels = case(500, 192, 3000, 0.8)
    check(kd, H, W, labels, bf16=True, chunk=512)
    _, _, once = kd.fused_cross_entropy_step(H, W, labels, chunk=256)
    base = torch.randn_like(once)
    given = base.clone()
    before = given._version
    _, _, twice = kd.fused_cross_entropy_step(H, W, labels, chunk=256, grad_W=given)
    assert twice is given and given._version > before
    assert torch.allclose(twice, once + base, atol=1e-6, rtol=0)
    gH = torch.full((500, 192), float("nan"), dtype=torch.bfloat16, device="cuda")
    _, a, _ = kd.fused_cross_entropy_step(H, W, labels, chunk=256, grad_H=gH)
    assert a is gH and torch.isfinite(gH).all()
    with pytest.raises(kd.KDError):
        kd.fused_cross_entropy_step(H, W, labels, chunk=256, grad_W_bf16=True)


def test_against_differences(kd, cuda_device):
    """Directional differences of the operator's own loss: inputs on a grid of 2^-5 below 4 in size, where bf16
    steps are 2^-6 at most, so that steps of 2^-5 are exact.  The loss's third derivative along the unit-size
    direction is below 1, its fp32 error below 2e-6: off by h^2 / 6 + 2e-6 / h < 3e-4 + 7e-5."""
    g = torch.Generator(device="cuda").manual_seed(2)
    N, d, V, h = 40, 64, 300, 2.0 ** -5
    grid = lambda *s: (torch.randint(-64, 65, s, generator=g, device="cuda") * h).to(torch.bfloat16)
    H, W = grid(N, d), (torch.randint(-8, 9, (V, d), generator=g, device="cuda") * h).to(torch.bfloat16)
    labels = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    opt = dict(label_smoothing=0.1, z_loss=1e-3, softcap=20.0)
    _, gH, gW = kd.fused_cross_entropy_step(H, W, labels, **opt, grad_H_fp32=True)
    value = lambda a, b: float(kd.fused_cross_entropy_forward(a, b, labels, **opt)[0].double())
    for i in range(4):
        u = torch.zeros_like(H)
        u[i * 7, i * 11] = h
        num = (value(H + u, W) - value(H - u, W)) / (2 * h)
        assert abs(num - float(gH[i * 7, i * 11])) <= 4e-4 + 0.01 * abs(num)
        u = torch.zeros_like(W)
        u[int(labels[i]), i * 5] = h
        num = (value(H, W + u) - value(H, W - u)) / (2 * h)
        assert abs(num - float(gW[int(labels[i]), i * 5])) <= 4e-4 + 0.01 * abs(num)


def test_autograd(kd, cuda_device):
    H, W, labels = case(300, 128, 1000, 0.9)
    _, gH, gW = kd.fused_cross_entropy_step(H, W, labels, chunk=512, z_loss=1e-4, grad_W_bf16=True)
    for chunk in (512, 128):
        h, w = H.clone().requires_grad_(), W.clone().requires_grad_()
        loss = kd.fused_cross_entropy(h, w, labels, chunk=chunk, z_loss=1e-4)
        a = torch.autograd.grad(loss, (h, w), retain_graph=True)
        b = torch.autograd.grad(loss, (h, w), torch.tensor(4.0, device="cuda"), retain_graph=True)
        c = torch.autograd.grad(loss * 0.5 + loss.detach(), (h, w))
        assert a[0].dtype == a[1].dtype == torch.bfloat16
        for x, y, z, r in zip(a, b, c, (gH, gW)):
            assert torch.equal(x * 4, y) and torch.equal(x * 0.5, z)
            # other chunks add up in another order: one rounding to bf16
            assert torch.equal(x, r) if chunk == 512 else torch.allclose(x.float(), r.float(), rtol=2 ** -7, atol=1e-7)
    h = H.clone().requires_grad_()
    loss = kd.fused_cross_entropy(h, W, labels, chunk=512, z_loss=1e-4)
    loss.backward()
    assert torch.equal(h.grad, gH)
    with torch.no_grad():
        assert torch.equal(kd.fused_cross_entropy(h, W, labels, chunk=512, z_loss=1e-4), loss)
    (once,) = torch.autograd.grad(kd.fused_cross_entropy(h, W, labels), h, create_graph=True)
    with pytest.raises(RuntimeError):
        once.sum().backward()


def test_label_out_of_range(kd, cuda_device):
    H, W, labels = case(200, 64, 500)
    labels[150] = 500
    ws = kd.workspace(kd._abi.kd_fused_cross_entropy_workspace(200, 64, 500, 128, 1), "cuda")
    each = torch.empty((200,), device="cuda")
    loss, gH, gW = kd.fused_cross_entropy_step(H, W, labels, chunk=128, ws=ws, loss_out=each)
    st, detail = kd.device_error(ws)
    assert st == kd._abi.KD_ERR_DEVICE and detail == 150
    assert torch.isnan(each).nonzero().flatten().tolist() == [150] and torch.isnan(loss).all()
    assert not gH[150].any() and torch.isfinite(gW).all()
    kd.fused_cross_entropy_forward(H, W, labels, chunk=128)
    kd.fused_cross_entropy_step(H, W, labels, chunk=128)
    assert kd.device_error(kd.control_block())[0] == kd._abi.KD_ERR_DEVICE


def test_logits_far_from_zero(kd, cuda_device):
    """Logits of +-600: probabilities of 0 and 1, the label among both."""
    g = torch.Generator(device="cuda").manual_seed(4)
    W = torch.randint(-8, 9, (700, 64), generator=g, device="cuda").to(torch.bfloat16)
    H = torch.randint(-4, 5, (60, 64), generator=g, device="cuda").to(torch.bfloat16)
    z = H.float() @ W.float().T
    labels = torch.where(torch.arange(60, device="cuda") % 2 == 0, z.argmax(1), z.argmin(1)).to(torch.int32)
    loss_r, each_r, _, gH_r, gW_r, bH, bW = reference(H, W, labels)
    each = torch.empty((60,), device="cuda")
    loss, gH, gW = kd.fused_cross_entropy_step(H, W, labels, loss_out=each, grad_H_fp32=True)
    assert ((each.double() - each_r).abs() <= 2.5e-4).all()
    near(gH, gH_r, bH + 1e-10, False)
    near(gW, gW_r, bW + 1e-10, False)


def test_captured_and_replayed(kd, cuda_device):
    H, W, labels = case(300, 128, 1000, 0.8)
    kd.fused_cross_entropy_step(H, W, labels, chunk=512)   # warm-up
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kd.fused_cross_entropy_step(H, W, labels, chunk=512)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, gH, gW = kd.fused_cross_entropy_step(H, W, labels, chunk=512)
    for seed in (7, 8):
        H2, W2, l2 = case(300, 128, 1000, 0.1 * seed, seed)
        H.copy_(H2), W.copy_(W2), labels.copy_(l2)
        graph.replay()
        torch.cuda.synchronize()
        want = kd.fused_cross_entropy_step(H2, W2, l2, chunk=512)
        for x, y in zip((loss, gH, gW), want):
            assert torch.equal(x, y)


def test_two_streams(kd, cuda_device):
    cases = [case(260, 128, 2000, 0.9, seed) for seed in (1, 2)]
    want = [kd.fused_cross_entropy_step(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        got = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(kd.fused_cross_entropy_step(*c))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(x, y))


@pytest.mark.parametrize("cap", [64.0, 65.0, 1e3, 1e5, 1e30])
def test_wide_softcaps(kd, cuda_device, cap):
    """Logits of +-70 under caps from near to far: the wider, the nearer to no cap at all."""
    H, W, labels = case(130, 64, 600, 0.9, seed=6)
    H = (H.float() * 8).to(torch.bfloat16)
    loss_r, each_r, lse_r, gH_r, gW_r, bH, bW = reference(H, W, labels, cap=cap)
    each = torch.empty((130,), device="cuda")
    loss, gH, gW = kd.fused_cross_entropy_step(H, W, labels, softcap=cap, loss_out=each, grad_H_fp32=True)
    # logits, and so their errors, 8 times those of the other cases: 1.6e-3 of a probability beside 2^-8 and 2^-12
    assert ((each.double() - each_r).abs() <= 8 * 2.5e-4).all()
    near(gH, gH_r, 1.25 * bH, False)
    near(gW, gW_r, 1.25 * bW, False)


def test_called_by_keyword(kd, cuda_device):
    H, W, labels = case(64, 64, 200)
    a = kd.fused_cross_entropy(H, W, labels)
    assert torch.equal(kd.fused_cross_entropy(labels=labels, W=W, H=H), a)
    assert torch.equal(kd.fused_cross_entropy_forward(H=H, W=W, labels=labels)[0][0], a)


def test_autograd_captured_and_replayed(kd, cuda_device):
    H, W, labels = case(200, 128, 700, 0.8)
    h, w = H.clone().requires_grad_(), W.clone().requires_grad_()
    def step():
        return torch.autograd.grad(0.5 * kd.fused_cross_entropy(h, w, labels), (h, w))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    H2, W2, l2 = case(200, 128, 700, 0.3, seed=9)
    with torch.no_grad():
        h.copy_(H2), w.copy_(W2), labels.copy_(l2)
    graph.replay()
    torch.cuda.synchronize()
    _, gH, gW = kd.fused_cross_entropy_step(H2, W2, l2, grad_W_bf16=True)
    assert torch.equal(got[0], gH * 0.5) and torch.equal(got[1], gW * 0.5)


def test_without_gradients(kd, cuda_device):
    H, W, labels = case(100, 64, 300)
    want = kd.fused_cross_entropy_forward(H, W, labels)[0][0]
    with torch.inference_mode():
        assert torch.equal(kd.fused_cross_entropy(H, W, labels), want)
    w = W.clone().requires_grad_()
    loss = kd.fused_cross_entropy(H, w, labels)
    loss.backward()
    assert torch.equal(loss.detach(), want) and torch.isfinite(w.grad).all()
    first = w.grad.clone()
    kd.fused_cross_entropy(H, w, labels).backward()     # added to, as any gradient
    assert torch.equal(w.grad, first + first)
