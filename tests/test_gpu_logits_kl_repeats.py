"""logits_kl with ids that repeat within a row: the same bits from every run, whichever of an id's entries a
warp comes to first."""
import pytest
import torch

import oracle
from test_gpu_logits_kl import host
from test_gpu_logprobs import check_grad, near

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


@pytest.mark.parametrize("N,V,K", [(200, 700, 128), (40, 4096, 1024), (20, 100000, 300)])
@pytest.mark.parametrize("tail", [False, True])
def test_repeated_ids_in_different_warps(kd, cuda_device, N, V, K, tail):
    g = torch.Generator(device="cuda").manual_seed(K)
    z = torch.randn((N, V), generator=g, device="cuda") * 2
    ids = torch.randint(0, min(V, K), (N, K), generator=g, device="cuda", dtype=torch.int32)   # most repeat
    t = torch.randn((N, K), generator=g, device="cuda")
    t_lse = torch.logsumexp(t, 1) + 0.2 if tail else None
    one = torch.ones(1, device="cuda")

    def go():
        kl = torch.empty((N,), device="cuda")
        _, stats, ws = kd.logits_kl_forward(z, ids, t, None, 1.0, t_lse, kl_out=kl)
        dz = kd.logits_kl_backward(z, ids, t, None, stats, one, 1.0, t_lse, ws=ws)
        kl2 = torch.empty((N,), device="cuda")
        _, dz2 = kd.logits_kl_step(z, ids, t, None, 1.0, t_lse, kl_out=kl2)
        return kl, stats, dz, kl2, dz2

    first = go()
    ref = oracle.logits_kl(host(z), host(ids), host(t), t_lse=host(t_lse))
    for kl, dz in (first[::2][:2], first[3:]):
        near(kl.cpu(), ref.kl, 4e-5 + 4e-7 * (abs(ref.kl) + 40))
        check_grad(dz, ref.grad, torch.float32)
    for _ in range(30):
        for a, b in zip(first, go()):
            assert torch.equal(a, b)
