"""Where the error word of a call without a workspace is read, and that nobody else clears it."""
import threading

import pytest
import torch

from test_gpu_logits_kl import case
from test_gpu_logprobs import draw, tokens_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


def kl_with_a_bad_id():
    z, ids, t, _ = case(5, 300, 6, torch.float32)
    ids[3, 2] = 300
    return z, ids, t


def fused_with_a_bad_token(n):
    g = torch.Generator(device="cuda").manual_seed(0)
    H = torch.randn((n, 64), generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randn((500, 64), generator=g, device="cuda").to(torch.bfloat16)
    tok = torch.zeros((n,), dtype=torch.int32, device="cuda")
    tok[n - 1] = 500
    return H, W, tok


def reported(kd, row):
    block = kd.control_block(torch.device("cuda", 0))
    assert kd.device_error(block) == (kd._abi.KD_ERR_DEVICE, row)
    assert kd.device_error(block)[0] == 0


@pytest.fixture(autouse=True)
def clean(kd):
    kd.device_error(kd.control_block(torch.device("cuda", 0)))
    junk = torch.full((1 << 20,), -1, dtype=torch.int32, device="cuda")   # what fresh memory is likely to hold
    del junk


def test_kl_calls_report(kd, cuda_device):
    z, ids, t = kl_with_a_bad_id()
    kd.logits_kl_step(z, ids, t)
    reported(kd, 3)
    kd.logits_kl(z, ids, t)
    reported(kd, 3)
    zr = z.clone().requires_grad_(True)
    loss = kd.logits_kl(zr, ids, t)
    reported(kd, 3)
    loss.backward()
    reported(kd, 3)
    _, stats, ws = kd.logits_kl_forward(z, ids, t)        # hands out its workspace: the error is there
    assert kd.device_error(ws) == (kd._abi.KD_ERR_DEVICE, 3)
    kd.logits_kl_backward(z, ids, t, None, stats, torch.ones(1, device="cuda"))
    reported(kd, 3)


@pytest.mark.parametrize("n", [2, 140])
def test_fused_calls_report(kd, cuda_device, n):
    H, W, tok = fused_with_a_bad_token(n)
    kd.fused_logprobs(H, W, tok)
    reported(kd, n - 1)
    Hr = H.clone().requires_grad_(True)
    logp, _ = kd.fused_logprobs(Hr, W, tok, chunk=128)
    reported(kd, n - 1)
    logp.sum().backward()
    logp, _, _, ws = kd.fused_logprobs_forward(H, W, tok)
    assert kd.device_error(ws) == (kd._abi.KD_ERR_DEVICE, n - 1)


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


def test_calls_in_a_graph_report(kd, cuda_device):
    z, ids, t = kl_with_a_bad_id()
    good = ids.clamp(max=299).contiguous()
    tok = tokens_for(5, 300, 1, 1)
    kd.logits_kl_step(z, good, t)
    kd.token_logprobs_forward(z, tok)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss, _ = kd.logits_kl_step(z, good, t)
        kd.token_logprobs_forward(z, tok)
    block = kd.control_block(torch.device("cuda", 0), captured=True)
    graph.replay()
    assert kd.device_error(block)[0] == 0
    want, _ = kd.logits_kl_step(z, good, t)
    assert torch.equal(loss, want)
    good[1, 1] = -5
    graph.replay()
    assert kd.device_error(block) == (kd._abi.KD_ERR_DEVICE, 1)
    good[1, 1] = 0
    tok[4] = 300
    graph.replay()
    assert kd.device_error(block) == (kd._abi.KD_ERR_DEVICE, 4)
    assert kd.device_error(kd.control_block(torch.device("cuda", 0)))[0] == 0
