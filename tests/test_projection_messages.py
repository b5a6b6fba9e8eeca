"""What the calls on hidden states and a head say of a wrong tensor: its own name."""
import types

import pytest
import torch

import sparse_teacher_kl_gb300 as kd


def stand_in(shape, dtype, device="cuda:0"):
    """What the checks look at of a tensor on a GPU that is not here."""
    return types.SimpleNamespace(shape=torch.Size(shape), dtype=dtype, device=torch.device(device),
                                 is_cuda=device != "cpu", dim=lambda: len(shape), is_contiguous=lambda: True)


def test_names_of_the_checks():
    H, W = stand_in((4, 8), torch.bfloat16), stand_in((10, 8), torch.bfloat16)
    good = stand_in((4,), torch.int32)
    for bad in (stand_in((4,), torch.int64), stand_in((5,), torch.int32), stand_in((4,), torch.int32, "cpu")):
        with pytest.raises(ValueError, match="^tokens must be"):
            kd._check_projection(H, W, bad, None)
        with pytest.raises(ValueError, match="^labels must be"):
            kd._check_projection(H, W, bad, None, "labels")
    with pytest.raises(ValueError, match="^mask must be"):
        kd._check_projection(H, W, good, stand_in((4,), torch.bool))
    with pytest.raises(ValueError, match="^H must be"):
        kd._check_projection(stand_in((4, 8), torch.float32), W, good, None)
    with pytest.raises(ValueError, match="^W must be"):
        kd._check_projection(H, stand_in((10, 8), torch.float16), good, None)
    assert kd._check_projection(H, W, good, None) == (4, 8, 10, torch.device("cuda:0"))


@pytest.mark.gpu
def test_public_calls(cuda_device):
    H, W = torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda"), torch.zeros((10, 8), dtype=torch.bfloat16, device="cuda")
    labels = torch.zeros((4,), dtype=torch.int64, device="cuda")
    for f in (kd.fused_cross_entropy, kd.fused_cross_entropy_forward, kd.fused_cross_entropy_step):
        with pytest.raises(ValueError, match="^labels must be a contiguous torch.int32"):
            f(H, W, labels)
    for f in (kd.fused_logprobs, kd.fused_logprobs_forward):
        with pytest.raises(ValueError, match="^tokens must be a contiguous torch.int32"):
            f(H, W, labels)
