"""Logits and temperatures anywhere in fp32's range: token_logprobs, logits_kl and fused_logprobs
against the float64 oracle.

Tolerances as in test_gpu_logprobs.py and test_gpu_logits_kl.py: with logits that are exact in fp32
their differences are rounded once, and scaled once by 1 / tau.  Temperatures are fp32 values.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from test_gpu_logprobs import check_forward

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


def f32(x):
    return float(np.float32(x))


# ------------------------------------------------------------- dense scores

@pytest.mark.parametrize("V", [40, 2051, 201088])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("tau", [1e-30, 1e-10, 4e-9, 1.0])
def test_entropy_of_rows_of_zeros(kd, cuda_device, dtype, V, tau):
    """Logits of 0 and -inf: at 1 / tau above 2e8 the stand-in for an element that is not there stays finite."""
    z = torch.zeros((3, V), dtype=dtype, device="cuda")
    z[1, 1::2] = -math.inf
    z[2, :V - 1] = -math.inf
    ref = oracle.token_logprobs(z.double().cpu().numpy(), np.zeros((3, 1), np.int32), None, f32(tau), 3)
    r = kd.token_logprobs_forward(z, torch.zeros((3, 1), dtype=torch.int32, device="cuda"), tau=tau, top=3,
                                  entropy=True)
    check_forward(r, ref, 3)
