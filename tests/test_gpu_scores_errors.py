"""Where the error word of a call without a workspace is read, and that nobody else clears it."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


@pytest.mark.parametrize("device", [None, "cuda", "cuda:0", torch.device("cuda"), 0])
def test_any_name_of_the_device(kd, cuda_device, device):
    assert kd.control_block(device) is kd.control_block(torch.device("cuda", 0))
