"""token_logprobs where a thread's groups of vectors share their kept maxima: more than 32 rounds of a
block over its row, which takes fp32 rows of over 131072 logits and rows enough for a block each."""
import pytest
import torch

from test_gpu_logprobs import tokens_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


@pytest.mark.parametrize("V", [140000, 150001, 270000])
@pytest.mark.parametrize("crowded", [False, True])
def test_alternatives_of_shared_groups(kd, cuda_device, V, crowded):
    N, top = 460, 20
    g = torch.Generator(device="cuda").manual_seed(V)
    z = torch.randn((N, V), generator=g, device="cuda") * 2
    if crowded:      # few distinct values, the largest in one stretch, at the end, or everywhere
        z = (z * 2).round() / 2
        z[1, 5000:5400] = 50.0
        z[2, V - 30:] = 60.0 + torch.arange(30, device="cuda") % 3
        z[3] = 1.0
    tok = tokens_for(N, V, 1, 1)
    ws = kd.workspace(256, "cuda")
    r = kd.token_logprobs_forward(z, tok, top=top, entropy=True, ws=ws)
    assert kd.device_error(ws)[0] == 0
    for a in range(0, N, 92):
        rows = z[a:a + 92]
        lp = torch.log_softmax(rows.double(), 1)
        order = torch.sort(rows, dim=1, descending=True, stable=True)[1][:, :top]   # equal values: ascending id
        assert torch.equal(r.top_ids[a:a + 92].long(), order)
        want = lp.gather(1, order)
        assert ((r.top_logp[a:a + 92] - want).abs() <= 4e-5 + 4e-7 * want.abs()).all()
        want = lp.gather(1, tok[a:a + 92].long())
        assert ((r.logp[a:a + 92] - want).abs() <= 4e-5 + 4e-7 * want.abs()).all()
        ent = -(lp.exp() * lp).sum(1)
        assert ((r.entropy[a:a + 92] - ent).abs() <= 4e-5 * (1 + ent)).all()
