"""The differentiable calls under autograd's own rules: inputs rewritten between the passes, gradients
written over the logits, second derivatives."""
import pytest
import torch

from test_gpu_logits_kl import case
from test_gpu_logprobs import tokens_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


def calls(kd):
    """(output of the differentiable call, its tensors by name)."""
    z, ids, t, t_lse = case(6, 200, 5, torch.float32, tail=True)
    mask = torch.tensor([1, 0, 1, 1, 1, 0], dtype=torch.uint8, device="cuda")
    zr = z.clone().requires_grad_(True)
    yield kd.logits_kl(zr, ids, t, mask, 1.0, t_lse), zr, dict(ids=ids, tlog=t, mask=mask, t_lse=t_lse)
    tok, mask = tokens_for(6, 200, 2, 1), mask.clone()
    zr = z.clone().requires_grad_(True)
    logp, ent = kd.token_logprobs(zr, tok, mask)
    yield logp.sum() + ent.sum(), zr, dict(tokens=tok, mask=mask)
    mask = mask.clone()
    H = torch.randn((6, 64), device="cuda").to(torch.bfloat16).requires_grad_(True)
    W = torch.randn((300, 64), device="cuda").to(torch.bfloat16)
    tok = tokens_for(6, 300, 1, 1)[:, 0].contiguous()
    logp, ent = kd.fused_logprobs(H, W, tok, mask)
    yield logp.sum() + ent.sum(), H, dict(W=W, tokens=tok, mask=mask)


def test_inputs_rewritten_before_the_backward_pass_are_noticed(kd, cuda_device):
    names = [(i, name) for i, (_, _, inputs) in enumerate(calls(kd)) for name in inputs]
    assert len(names) == 4 + 2 + 3
    for i, name in names:
        out, _, inputs = list(calls(kd))[i]
        inputs[name].add_(1)
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            out.backward()


def test_gradients_written_over_the_logits_are_noticed(kd, cuda_device):
    """token_logprobs keeps the logits for its backward pass; a gradient of another call takes their place."""
    z, ids, t, _ = case(6, 200, 5, torch.float32)
    one = torch.ones(1, device="cuda")
    tok = tokens_for(6, 200, 1, 1)
    r = kd.token_logprobs_forward(z, tok)
    _, stats, _ = kd.logits_kl_forward(z, ids, t)

    def step(x):
        kd.logits_kl_step(x, ids, t, grad_logits=x)

    def kl_backward(x):
        kd.logits_kl_backward(x, ids, t, None, stats, one, grad_logits=x)

    def score_backward(x):
        kd.token_logprobs_backward(x, tok, r.lse, torch.ones_like(r.logp), grad_logits=x)

    for write in (step, kl_backward, score_backward):
        leaf = z.clone().requires_grad_(True)
        logits = leaf * 1.0
        logp, _ = kd.token_logprobs(logits, tok)
        write(logits.detach())
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            logp.sum().backward()


def test_gradients_written_into_a_callers_tensors_are_noticed(kd, cuda_device):
    H = torch.randn((5, 64), device="cuda").to(torch.bfloat16)
    W = torch.randn((300, 64), device="cuda").to(torch.bfloat16)
    tok = tokens_for(5, 300, 1, 1)[:, 0].contiguous()
    logp, lse, _, _ = kd.fused_logprobs_forward(H, W, tok)
    gH, gW = torch.zeros((5, 64), device="cuda"), torch.zeros((300, 64), device="cuda")
    before = gH._version, gW._version
    kd.fused_logprobs_backward(H, W, tok, lse, torch.ones_like(logp), grad_H=gH, grad_W=gW)
    assert gH._version > before[0] and gW._version > before[1]
    kl = torch.zeros((6,), device="cuda")
    z, ids, t, _ = case(6, 200, 5, torch.float32)
    before = kl._version
    kd.logits_kl_step(z, ids, t, kl_out=kl)
    assert kl._version > before
    before = kl._version
    kd.logits_kl_forward(z, ids, t, kl_out=kl)
    assert kl._version > before


def test_in_place_gradients_under_inference_mode(kd, cuda_device):
    z, ids, t, _ = case(6, 200, 5, torch.float32)
    want = kd.logits_kl_step(z, ids, t)[1]
    with torch.inference_mode():
        x = z.clone()
        kd.logits_kl_step(x, ids, t, grad_logits=x)
    assert torch.equal(x, want)
    x = None
    with torch.inference_mode():
        x = z.clone()
    kd.logits_kl_step(x, ids, t, grad_logits=x)       # an inference tensor outside inference mode
    assert torch.equal(x, want)


def test_second_derivatives_are_refused(kd, cuda_device):
    for i in range(3):
        out, x, _ = list(calls(kd))[i]
        (g,) = torch.autograd.grad(out, x, create_graph=True)
        with pytest.raises(RuntimeError, match="once_differentiable"):
            (g.float() * x.float()).sum().backward()


def test_first_derivatives_with_create_graph_keep_their_values(kd, cuda_device):
    for i in range(2):
        out, x, _ = list(calls(kd))[i]
        out2, x2, _ = list(calls(kd))[i]
        (a,) = torch.autograd.grad(out, x, create_graph=True)
        (b,) = torch.autograd.grad(out2, x2)
        assert torch.equal(a, b)
