"""Where the error word of a call without a workspace is read, and that nobody else clears it."""
import threading

import pytest
import torch

from test_gpu_logprobs import draw, tokens_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


def reported(kd, row):
    block = kd.control_block(torch.device("cuda", 0))
    assert kd.device_error(block) == (kd._abi.KD_ERR_DEVICE, row)
    assert kd.device_error(block)[0] == 0


@pytest.fixture(autouse=True)
def clean(kd):
    kd.device_error(kd.control_block(torch.device("cuda", 0)))
    junk = torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda")   # what fresh memory is likely to hold
    del junk


def test_token_logprobs_backward_reports_to_the_callers_block(kd, cuda_device):
    z, tok = draw(6, 100, torch.float32, 1).requires_grad_(True), tokens_for(6, 100, 1, 1)
    tok[4] = 100
    logp, _ = kd.token_logprobs(z, tok)
    reported(kd, 4)
    logp.nan_to_num().sum().backward()      # runs on autograd's own thread
    reported(kd, 4)


def test_streams_and_threads_have_blocks_of_their_own(kd, cuda_device):
    dev = torch.device("cuda", 0)
    z, tok = draw(3, 90, torch.float32, 1), tokens_for(3, 90, 1, 1)
    tok[2] = -1
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        kd.token_logprobs_forward(z, tok)
    side.synchronize()
    assert kd.device_error(kd.control_block(dev))[0] == 0        # the current stream's: nothing
    with torch.cuda.stream(side):
        assert kd.device_error(kd.control_block(dev)) == (kd._abi.KD_ERR_DEVICE, 2)

    seen = []

    def other():
        kd.token_logprobs_forward(z, tok)
        torch.cuda.synchronize()
        seen.append("called")
        go.wait()
        seen.append(kd.device_error(kd.control_block(dev)))

    go = threading.Event()
    th = threading.Thread(target=other)
    th.start()
    while not seen:
        th.join(0.01)
    assert kd.device_error(kd.control_block(dev))[0] == 0        # not cleared by this thread either
    go.set()
    th.join()
    assert seen[1] == (kd._abi.KD_ERR_DEVICE, 2)


@pytest.mark.parametrize("device", [None, "cuda", "cuda:0", torch.device("cuda"), 0])
def test_any_name_of_the_device(kd, cuda_device, device):
    assert kd.control_block(device) is kd.control_block(torch.device("cuda", 0))


def test_scores_in_a_graph_report(kd, cuda_device):
    z, tok = draw(5, 300, torch.float32, 1), tokens_for(5, 300, 1, 1)
    kd.token_logprobs_forward(z, tok)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kd.token_logprobs_forward(z, tok)
    block = kd.control_block(captured=True)
    graph.replay()
    assert kd.device_error(block)[0] == 0
    tok[4] = 300
    graph.replay()
    assert kd.device_error(block) == (kd._abi.KD_ERR_DEVICE, 4)
    assert kd.device_error(kd.control_block())[0] == 0
