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
