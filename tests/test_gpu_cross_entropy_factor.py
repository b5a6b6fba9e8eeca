"""fused_cross_entropy under autograd: the factor that arrives joins the gradients before their one rounding, and what
the forward pass keeps for the backward pass.

A gradient in bf16 is the fp32 one of fused_cross_entropy_step for that grad_loss, rounded once.  Where both take the
same products in the same order they are the same numbers, bit for bit.  Over several chunks the factor multiplies the
sum and not its terms: of grad_W those of up to 5 chunks, of grad_H those of up to 8 splits of its reduction, and they may
cancel.  Either order has up to 8 additions and 2 products of 2^-24 of what they add up to at most, the sum of the
terms' magnitudes, and that is below |dZ|^T |H| (|dZ| |W|) with dZ's parts all positive: 20 * 2^-24 < 2^-19 of it.  The
rounding to bf16 is of a value that near to the other.
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


def case(N, d, V, valid=1.0, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    H = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn((V, d), generator=g, device="cuda") * (1.5 / d ** 0.5)).to(torch.bfloat16)
    labels = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
    labels[torch.rand((N,), generator=g, device="cuda") >= valid] = -100
    return H, W, labels


def magnitudes(H, W, labels, label_smoothing=0.0, z_loss=0.0, softcap=0.0):
    """|dZ| |W| and |dZ|^T |H| with the parts of dZ (probability, smoothing, label) added up, for a factor of 1."""
    on = labels >= 0
    z = H.double() @ W.double().T
    if softcap:
        z = softcap * (z / softcap).tanh()
    lse = z.logsumexp(1, keepdim=True)
    size = (z - lse).exp() * (1 + 2 * z_loss * lse.abs()) + label_smoothing / W.shape[0]
    size.scatter_add_(1, labels.clamp(min=0).long()[:, None], torch.ones_like(lse))
    size *= on[:, None] / max(1, int(on.sum()))
    return size @ W.double().abs(), size.T @ H.double().abs()


OPTIONS = [dict(), dict(label_smoothing=0.1, z_loss=1e-3, softcap=30.0), dict(softcap=5.0, label_smoothing=0.2)]


@pytest.mark.parametrize("opt", OPTIONS)
@pytest.mark.parametrize("factor", [1 / 3, 1.0, 0.7, -1e-3, 1000 / 3])
@pytest.mark.parametrize("N,d,V,valid", [(1, 8, 3, 1.0), (300, 128, 1000, 0.8), (513, 72, 2100, 0.5)])
def test_one_rounding(kd, cuda_device, N, d, V, valid, factor, opt):
    H, W, labels = case(N, d, V, valid, seed=N)
    g = torch.full((1,), factor, device="cuda")
    for chunk in (1024, 128):
        h, w = H.clone().requires_grad_(), W.clone().requires_grad_()
        loss = kd.fused_cross_entropy(h, w, labels, chunk=chunk, **opt)
        first = torch.autograd.grad(loss, (h, w), g[0], retain_graph=True)
        second = torch.autograd.grad(loss, (h, w), g[0])
        step, *want = kd.fused_cross_entropy_step(H, W, labels, chunk=chunk, grad_loss=g, grad_H_fp32=True, **opt)
        assert torch.equal(step[0], loss)
        for got in (first, second):
            for a, b, most in zip(got, want, magnitudes(H, W, labels, **opt)):
                assert a.dtype == torch.bfloat16
                if N <= chunk:
                    assert torch.equal(a, b.to(torch.bfloat16))
                else:
                    off = abs(factor) * 2.0 ** -19 * most
                    low, high = b - off - 1e-30, b + off + 1e-30
                    assert ((a >= low.to(torch.bfloat16)) & (a <= high.to(torch.bfloat16))).all()


def test_factor_from_a_sum_of_losses(kd, cuda_device):
    """The example's use: a share of the loss, the rest of it something else."""
    H, W, labels = case(200, 64, 700, 0.9)
    h, w = H.clone().requires_grad_(), W.clone().requires_grad_()
    (0.3 * kd.fused_cross_entropy(h, w, labels, chunk=256) + 0.0 * h.float().sum()).backward()
    g = torch.full((1,), 0.3, device="cuda")
    _, gH, gW = kd.fused_cross_entropy_step(H, W, labels, chunk=256, grad_loss=g, grad_W_bf16=True)
    assert torch.equal(h.grad, gH) and torch.equal(w.grad, gW)


def test_kept_through_saved_tensor_hooks(kd, cuda_device):
    """What waits for the backward pass is saved as tensors: offloading sees it, and freeing the graph frees it."""
    for N, chunk in ((200, 256), (200, 128)):
        H, W, labels = case(N, 64, 5000)
        h, w = H.clone().requires_grad_(), W.clone().requires_grad_()
        want = torch.autograd.grad(kd.fused_cross_entropy(h, w, labels, chunk=chunk), (h, w))
        with torch.autograd.graph.save_on_cpu():
            loss = kd.fused_cross_entropy(h, w, labels, chunk=chunk)
        got = torch.autograd.grad(loss, (h, w))
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    loss = kd.fused_cross_entropy(h, w, labels, chunk=256)
    held = torch.cuda.memory_allocated() - before
    assert held < 2 * 256 * 5056 + 16 * 256 * 41 + 2 * 256 * 64 + 40 * 256 + 8192   # logits, partials, states, lists
    del loss
    assert torch.cuda.memory_allocated() <= before


def test_positions_without_a_loss(kd, cuda_device):
    H, W, labels = case(300, 64, 500)
    labels[:] = -100
    H[:] = float("nan")
    for chunk in (512, 128):
        h, w = H.clone().requires_grad_(), W.clone().requires_grad_()
        loss = kd.fused_cross_entropy(h, w, labels, chunk=chunk)
        gH, gW = torch.autograd.grad(loss, (h, w), torch.tensor(3.0, device="cuda"))
        assert float(loss.detach()) == 0 and not gH.any() and not gW.any()


@pytest.mark.parametrize("chunk", [0, 100, 129, -128])
def test_chunks_are_refused_with_and_without_gradients(kd, cuda_device, chunk):
    H, W, labels = case(64, 64, 500)
    for h in (H, H.clone().requires_grad_()):
        with pytest.raises(kd.KDError):
            kd.fused_cross_entropy(h, W, labels, chunk=chunk)


def test_changed_inputs_are_refused(kd, cuda_device):
    H, W, labels = case(100, 64, 500)
    h, w = H.clone().requires_grad_(), W.clone().requires_grad_()
    loss = kd.fused_cross_entropy(h, w, labels)
    with torch.no_grad():
        w += 1
    with pytest.raises(RuntimeError):
        loss.backward()


def test_backward_on_its_own_in_a_graph(kd, cuda_device):
    """Forward and backward captured together, replayed with other inputs and another factor."""
    H, W, labels = case(300, 128, 1000, 0.8)
    factor = torch.full((), 0.25, device="cuda")
    h, w = H.clone().requires_grad_(), W.clone().requires_grad_()
    def step():
        return torch.autograd.grad(kd.fused_cross_entropy(h, w, labels, chunk=512, softcap=20.0), (h, w), factor)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed, f in ((5, 1 / 3), (6, 7.0)):
        H2, W2, l2 = case(300, 128, 1000, 0.4, seed)
        with torch.no_grad():
            h.copy_(H2), w.copy_(W2), labels.copy_(l2), factor.fill_(f)
        graph.replay()
        torch.cuda.synchronize()
        _, gH, gW = kd.fused_cross_entropy_step(H2, W2, l2, chunk=512, softcap=20.0, grad_W_bf16=True,
                                                grad_loss=torch.full((1,), f, device="cuda"))
        assert torch.equal(got[0], gH) and torch.equal(got[1], gW)


@pytest.mark.parametrize("chunk", [512, 128])
def test_forward_and_backward_in_graphs_of_their_own(kd, cuda_device, chunk):
    """What the forward graph keeps, the backward graph spends, replay after replay."""
    H, W, labels = case(300, 64, 1000, 0.8)
    h, w = H.clone().requires_grad_(), W.clone().requires_grad_()
    step = torch.cuda.make_graphed_callables(lambda a, b: kd.fused_cross_entropy(a, b, labels, chunk=chunk), (h, w))
    for seed, factor in ((1, 1 / 3), (2, 1.0), (3, -5.0)):
        H2, W2, l2 = case(300, 64, 1000, 0.3 * seed, seed)
        labels.copy_(l2)
        a, b = H2.clone().requires_grad_(), W2.clone().requires_grad_()
        loss = step(a, b)
        (loss * factor).backward()
        h2, w2 = H2.clone().requires_grad_(), W2.clone().requires_grad_()
        want = kd.fused_cross_entropy(h2, w2, l2, chunk=chunk)
        (want * factor).backward()
        assert torch.equal(loss, want) and torch.equal(a.grad, h2.grad) and torch.equal(b.grad, w2.grad)


def test_nothing_kept(kd, cuda_device):
    """What no forward pass has kept, or another one's, or what is spent: an error, zero gradients, nothing out of place."""
    N, d, V = 200, 64, 700
    H, W, labels = case(N, d, V, 0.9)
    abi, stream = kd._abi, torch.cuda.current_stream().cuda_stream
    control = kd.workspace(256, "cuda")
    kept = torch.full((abi.kd_fused_cross_entropy_kept(N, d, V),), 0x7F, dtype=torch.uint8, device="cuda")
    ws = torch.empty((abi.kd_fused_cross_entropy_bwd_workspace(N, d, V),), dtype=torch.uint8, device="cuda")
    f32 = lambda *s: torch.full(s, 7.0, device="cuda")
    loss, lse = f32(1), f32(N)

    def backward(cap=0.0, smooth=0.0):
        gH, gW, base = f32(N, d), f32(V, d), f32(V, d)
        for g, kind in ((gW, abi.KD_GRAD_STORE_F32), (base, abi.KD_GRAD_ADD_F32)):
            st = abi.kd_fused_cross_entropy_bwd(W.data_ptr(), N, d, V, smooth, cap, None, gH.data_ptr(), 1, g.data_ptr(), kind,
                                                kept.data_ptr(), kept.numel(), ws.data_ptr(), ws.numel(),
                                                control.data_ptr(), stream)
            assert st == 0
            if kind == abi.KD_GRAD_STORE_F32:
                found = kd.device_error(control)[0], gH.clone(), gW
        # the second of the two finds it spent in any case
        assert kd.device_error(control)[0] == abi.KD_ERR_DEVICE and not gH.any() and (base == 7).all()
        return found

    def forward():
        st = abi.kd_fused_cross_entropy_keep(H.data_ptr(), W.data_ptr(), labels.data_ptr(), None, N, d, V, 0.0, 0.0, 0.0,
                                             -100, loss.data_ptr(), lse.data_ptr(), None, kept.data_ptr(), kept.numel(),
                                             control.data_ptr(), stream)
        assert st == 0

    st, gH, gW = backward()
    assert st == abi.KD_ERR_DEVICE and not gH.any() and not gW.any()
    forward()
    st, gH, gW = backward()
    _, wH, wW = kd.fused_cross_entropy_step(H, W, labels, chunk=256, grad_H_fp32=True)
    assert st == 0 and torch.equal(gH, wH) and torch.equal(gW, wW)
    forward()
    st, gH, gW = backward(cap=5.0)
    assert st == abi.KD_ERR_DEVICE and not gH.any() and not gW.any()
    forward()
    kd.fused_cross_entropy_forward(H, W, labels, ws=kept, chunk=256)   # another call's workspace since
    st, gH, gW = backward()
    assert st == abi.KD_ERR_DEVICE and not gH.any() and not gW.any()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_scale_gradient(kd, cuda_device, dtype):
    x = torch.randn((8 * 1003,), device="cuda").to(dtype)
    for f in (1.0, 1 / 3, -2.0):
        y, g = x.clone(), torch.full((1,), f, device="cuda")
        st = kd._abi.kd_scale_gradient(y.data_ptr(), y.numel(), int(dtype == torch.float32), g.data_ptr(),
                                       torch.cuda.current_stream().cuda_stream)
        assert st == 0 and torch.equal(y, (x.float() * g).to(dtype))
