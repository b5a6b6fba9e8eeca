"""Sizes whose last tile would end beyond 2^31 are refused before any CUDA work: the kernels count rows and columns
in 32 bits, up to a tile behind the last one (no GPU needed)."""
import pytest

from sparse_teacher_kl_gb300 import _abi
from sparse_teacher_kl_gb300.build import build_library

P = 1 << 20   # fake, 256-byte aligned device address, never dereferenced on these paths
MOST = (1 << 31) - 1024   # the largest size that is taken


@pytest.fixture(scope="module")
def lib():
    build_library()
    return _abi.load()


def cross_entropy(lib, N, d, V, step):
    head = (P, P, P, None, N, d, V, 128, 0.0, 0.0, 0.0, -100)
    if step:
        return lib.kd_fused_cross_entropy_step(*head, None, P, P, None, P, 0, P, 1, P, 256, P, None)
    return lib.kd_fused_cross_entropy_fwd(*head, P, P, None, P, 256, P, None)


def logprobs(lib, N, d, V, step):
    if step:
        return lib.kd_fused_logprobs_bwd(P, P, P, None, N, d, V, 128, 1.0, P, None, P, None, P, 0, P, 1, P, 256, None)
    return lib.kd_fused_logprobs_fwd(P, P, P, None, N, d, V, 128, 1.0, P, P, None, P, 256, None)


@pytest.mark.parametrize("call", [cross_entropy, logprobs])
@pytest.mark.parametrize("step", [False, True])
def test_positions_and_vocabulary(lib, call, step):
    for at in range(3):
        for size in (MOST + 8, (1 << 31) - 8):
            sizes = [256, 64, 1000]
            sizes[at] = size
            assert call(lib, *sizes, step) == _abi.KD_ERR_INVALID_ARG
        sizes[at] = MOST
        assert call(lib, *sizes, step) == _abi.KD_ERR_WORKSPACE   # taken as far as its workspace


def test_quantized_columns(lib):
    """A row's last vector index, one step of 256 threads further, is still an int."""
    for d in (MOST + 1, (1 << 31) - 200, (1 << 31) - 1):
        assert lib.kd_quantize_int8(P, 0, 1, d, d, P, d, P, None) == _abi.KD_ERR_INVALID_ARG
