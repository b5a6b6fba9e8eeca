"""token_logprobs (forward and backward) against the float64 oracle.

Tolerances.  A row's sum of exponentials is accumulated in fp32: at most V / 512 + 14 sequential
additions (each 2^-24 relative), every term within 2^-22 (ex2) and |t| 2^-23 (rounded exponent) of
its value.  With V <= 201088 and the weight of the sum at |t| < 40 that is below 4e-5 relative:
  logp, lse : 4e-5 absolute plus 4e-7 of the value (its own rounding and m / tau's)
  entropy   : 4e-5 (1 + H) absolute (H times the relative error of each sum)
  gradients : the type's half unit in the last place (bf16 2^-8, fp16 2^-10, fp32 2^-22, one binade
              of slack), 1e-4 of the value, 1e-5 of the row's largest, half a subnormal step
Ids are exact.
"""
import math

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -10, torch.float32: 2.0 ** -22}
TINY = {torch.bfloat16: 1e-38, torch.float16: 6e-8, torch.float32: 1e-38}


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


def draw(N, V, dtype, seed, std=2.0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return (torch.randn((N, V), generator=g, device=device) * std).to(dtype)


def framed(z, lead, pad, fill=float("nan")):
    """z inside a larger buffer: `lead` elements before row 0, `pad` after each row, all of them NaN."""
    N, V = z.shape
    buf = torch.full((lead + N * (V + pad) + 8,), fill, dtype=z.dtype, device=z.device)
    view = buf[lead:lead + N * (V + pad)].view(N, V + pad)[:, :V]
    view.copy_(z)
    return buf, view


def near(got, ref, tol):
    got, ref = np.asarray(got, np.float64), np.asarray(ref, np.float64)
    inf = np.isinf(ref)
    assert np.array_equal(got[inf], ref[inf])
    assert np.isfinite(got[~inf]).all()
    bad = np.abs(got[~inf] - ref[~inf]) - np.broadcast_to(tol, ref.shape)[~inf]
    assert bad.size == 0 or bad.max() <= 0, f"off by {bad.max()} more than allowed"


def check_forward(r, ref, top):
    near(r.logp.double().cpu().reshape(ref.logp.shape), ref.logp, 4e-5 + 4e-7 * np.abs(np.nan_to_num(ref.logp, neginf=0)))
    near(r.lse.double().cpu(), ref.lse, 4e-5 + 4e-7 * np.abs(np.nan_to_num(ref.lse, neginf=0)))
    if r.entropy is not None:
        near(r.entropy.double().cpu(), ref.entropy, 4e-5 * (1 + ref.entropy))
    if top:
        assert np.array_equal(r.top_ids.cpu().numpy(), ref.top_ids)
        near(r.top_logp.double().cpu(), ref.top_logp, 4e-5 + 4e-7 * np.abs(np.nan_to_num(ref.top_logp, neginf=0)))


def check_grad(got, ref, dtype):
    big = np.abs(ref).max(axis=1, keepdims=True)
    near(got.double().cpu(), ref, (EPS[dtype] + 1e-4) * np.abs(ref) + 1e-5 * big + TINY[dtype])


def run_both(kd, z, tokens, mask=None, tau=1.0, top=0, seed=0):
    ws = kd.workspace(kd._abi.kd_token_logprobs_workspace(*z.shape), z.device)
    r = kd.token_logprobs_forward(z, tokens, mask, tau, top, entropy=True, ws=ws)
    g = torch.Generator(device="cuda").manual_seed(seed)
    gl = torch.randn(tokens.shape, generator=g, device="cuda")
    ge = torch.randn((z.shape[0],), generator=g, device="cuda") * 0.1
    dz = kd.token_logprobs_backward(z, tokens, r.lse, gl, mask, tau, r.entropy, ge, ws=ws)
    torch.cuda.synchronize()
    assert kd.device_error(ws)[0] == 0
    return r, dz, gl, ge


def check_both(kd, z, tokens, mask=None, tau=1.0, top=0, seed=0):
    r, dz, gl, ge = run_both(kd, z, tokens, mask, tau, top, seed)
    host = z.double().cpu().numpy()
    m = None if mask is None else mask.cpu().numpy()
    tok = tokens.cpu().numpy()
    check_forward(r, oracle.token_logprobs(host, tok, m, tau, top), top)
    check_grad(dz, oracle.token_logprobs_grad(host, tok, gl.cpu().numpy(), ge.cpu().numpy(), m, tau), z.dtype)
    return r, dz


def tokens_for(N, V, M, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, V, (N, M), generator=g).to(torch.int32).cuda()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("N,V,M,top,tau", [
    (1, 1, 1, 1, 1.0),
    (3, 2, 2, 2, 1.0),
    (5, 7, 1, 7, 0.5),
    (4, 129, 3, 128, 1.0),         # nearly every column is an alternative
    (130, 1000, 2, 20, 1.3),
    (2, 4099, 1, 5, 1.0),
    (7, 32003, 4, 64, 2.0),
    (2, 201088, 1, 20, 1.0),
])
def test_forward_and_backward(kd, cuda_device, dtype, N, V, M, top, tau):
    z = draw(N, V, dtype, 10 * V + N)
    check_both(kd, z, tokens_for(N, V, M, V), None, tau, top)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("lead,pad", [(0, 1), (1, 0), (3, 5), (8, 8), (7, 9)])
def test_any_alignment_and_stride_and_nothing_outside_the_rows(kd, cuda_device, dtype, lead, pad):
    N, V = 9, 2053
    z = draw(N, V, dtype, 5)
    _, zv = framed(z, lead, pad)
    tok = tokens_for(N, V, 2, 1)
    r, dz = check_both(kd, zv, tok, top=11)
    # a gradient buffer of another alignment: its frame keeps every bit
    buf, gv = framed(torch.zeros_like(z), 5, 3, fill=7.0)
    gl, ge = torch.ones(tok.shape, device="cuda"), torch.full((N,), 0.25, device="cuda")
    a = kd.token_logprobs_backward(zv, tok, r.lse, gl, None, 1.0, r.entropy, ge)
    kd.token_logprobs_backward(zv, tok, r.lse, gl, None, 1.0, r.entropy, ge, grad_logits=gv)
    assert torch.equal(gv, a)
    inside = torch.zeros_like(buf, dtype=torch.bool)
    inside[5:5 + N * (V + 3)].view(N, V + 3)[:, :V] = True
    assert (buf[~inside] == 7.0).all()
    # in place: the frame of the logits keeps its NaNs
    buf2, zv2 = framed(z, lead, pad)
    out = kd.token_logprobs_backward(zv2, tok, r.lse, gl, None, 1.0, r.entropy, ge, grad_logits=zv2)
    assert out is zv2 and torch.equal(zv2, a)
    assert int(torch.isnan(buf2).sum()) == buf2.numel() - N * V


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("masked_by", ["inf", "lowest"])
def test_vocabulary_masks_and_empty_rows(kd, cuda_device, dtype, masked_by):
    """Rows with no, one, three and half of their logits left; more alternatives asked for than are left."""
    N, V, top = 6, 6007, 20
    z = draw(N, V, dtype, 8)
    fill = -math.inf if masked_by == "inf" else torch.finfo(dtype).min
    keep = torch.zeros((N, V), dtype=torch.bool, device="cuda")
    keep[1, 4000] = True
    keep[2, [5, 6000, 3001]] = True
    keep[3, ::2] = True
    keep[4] = True
    keep[5, 17] = True
    z = z.masked_fill(~keep, fill)
    z[4, 6001] = fill
    tok = torch.tensor([[3, 9], [4000, 1], [6000, 7], [4, 5], [6001, 2], [16, 17]], dtype=torch.int32, device="cuda")
    check_both(kd, z, tok, top=top)


def test_nan_and_infinity_stay_in_their_rows(kd, cuda_device):
    z = draw(5, 3001, torch.bfloat16, 2)
    z[1, 77] = math.nan
    z[3, 3000] = math.inf
    tok = tokens_for(5, 3001, 1, 0)
    r, dz, gl, ge = run_both(kd, z, tok, top=6)
    for row in (1, 3):
        assert torch.isnan(r.logp[row]).all() and torch.isnan(r.lse[row]) and torch.isnan(r.entropy[row])
        assert torch.isnan(r.top_logp[row]).all() and r.top_ids[row].tolist() == list(range(6))
        assert torch.isnan(dz[row]).any()
    rows = [0, 2, 4]
    ref = oracle.token_logprobs(z[rows].double().cpu().numpy(), tok[rows].cpu().numpy(), top=6)
    check_forward(kd.TokenLogprobs(*(t[rows] for t in r)), ref, 6)
    # a NaN in a padding row is not looked at, nor is its token
    mask = torch.tensor([1, 0, 1, 0, 1], dtype=torch.uint8, device="cuda")
    tok[1], tok[3] = -100, 1 << 30
    r, dz, _, _ = run_both(kd, z, tok, mask, top=6)
    for t in (r.logp, r.lse, r.entropy, r.top_ids, r.top_logp, dz):
        assert not t[[1, 3]].any()
    check_forward(kd.TokenLogprobs(*(t[rows] for t in r)), ref, 6)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_padding(kd, cuda_device, dtype):
    mask = (torch.rand(40, generator=torch.Generator().manual_seed(1)) < 0.6).to(torch.uint8).cuda()
    check_both(kd, draw(40, 515, dtype, 3), tokens_for(40, 515, 3, 2), mask, 0.8, 4)


@pytest.mark.parametrize("V", [40, 1024, 9001, 70001])
@pytest.mark.parametrize("kind", ["constant", "two values", "clustered", "sorted", "periodic"])
def test_ties_and_crowded_rows(kd, cuda_device, V, kind):
    """Alternatives of rows that tie everywhere, or whose largest values crowd into few places."""
    col = torch.arange(V, device="cuda")
    z = {"constant": torch.zeros(V, device="cuda"),
         "two values": (col % 3 == 1).float(),
         "clustered": torch.where((col >= V // 2) & (col < V // 2 + 30), 5.0, 0.0) + (col % 7) * 0.125,
         "sorted": col.float() / V,
         "periodic": torch.where(col % 4096 < 8, 3.0 + (col // 4096) * 0.25, 0.0)}[kind]
    z = z.to(torch.bfloat16).repeat(3, 1)
    z[1] = z[1].flip(0)
    for top in (1, 33, min(V, 128)):
        check_both(kd, z, tokens_for(3, V, 1, 4), top=top)


@pytest.mark.parametrize("N,V", [(1, 201088), (3, 60001)])
@pytest.mark.parametrize("top", [20, 128])
def test_alternatives_of_few_long_rows(kd, cuda_device, N, V, top):
    """Rows that clusters share: the shares' lists are merged; a row whose largest values lie in one share, a
    row of NaNs, a row of few distinct values."""
    z = draw(N, V, torch.bfloat16, 77)
    check_both(kd, z, tokens_for(N, V, 1, 4), top=top)
    z[0, 1000:1300] = 40.0 + (torch.arange(300, device="cuda") % 50)
    check_both(kd, z, tokens_for(N, V, 1, 4), top=top)
    z[0] = (torch.arange(V, device="cuda") % 3).to(torch.bfloat16)
    check_both(kd, z, tokens_for(N, V, 1, 4), top=top)
    z[0] = math.nan
    r = kd.token_logprobs_forward(z, tokens_for(N, V, 1, 4), top=top)
    assert torch.isnan(r.top_logp[0]).all() and r.top_ids[0].tolist() == list(range(top))


def test_signed_zeros_tie(kd, cuda_device):
    z = torch.tensor([[-0.0, 0.0, -1.0, -0.0, 0.0]], device="cuda")
    assert kd.token_logprobs_forward(z, tokens_for(1, 5, 1, 0), top=5).top_ids.tolist() == [[0, 1, 3, 4, 2]]


def test_many_and_repeated_tokens(kd, cuda_device):
    z = draw(3, 300, torch.float32, 6)
    tok = tokens_for(3, 300, 1024, 7)
    tok[0] = 299
    check_both(kd, z, tok)


def test_large_logits(kd, cuda_device):
    """Logits far from zero: differences are formed before they are scaled."""
    z = (draw(4, 2050, torch.float32, 12) + torch.tensor([3e4, -3e4, 1e6, 90.0], device="cuda")[:, None])
    check_both(kd, z, tokens_for(4, 2050, 2, 3), tau=0.9, top=3)


def test_row_offsets_past_32_bits(kd, cuda_device):
    N, V, ld = 1030, 1000, 1 << 21
    buf = torch.empty(((N - 1) * ld + V + 3,), dtype=torch.bfloat16, device="cuda")
    z = buf.as_strided((N, V), (ld, 1), 3)
    z.copy_(draw(N, V, torch.bfloat16, 21))
    tok = tokens_for(N, V, 1, 5)
    r = kd.token_logprobs_forward(z, tok, top=3, entropy=True)
    dense = z.contiguous()
    s = kd.token_logprobs_forward(dense, tok, top=3, entropy=True)
    assert torch.equal(r.top_ids, s.top_ids)
    for a, b in ((r.logp, s.logp), (r.lse, s.lse), (r.entropy, s.entropy)):
        assert (a - b).abs().max() <= 4e-5
    gl, ge = torch.ones_like(s.logp), torch.full((N,), 0.1, device="cuda")
    g = kd.token_logprobs_backward(dense, tok, s.lse, gl, None, 1.0, s.entropy, ge)
    kd.token_logprobs_backward(z, tok, s.lse, gl, None, 1.0, s.entropy, ge, grad_logits=z)
    assert torch.equal(z, g)


@pytest.mark.parametrize("N,V", [(1, 50257), (64, 5000)])
def test_repeats_are_bit_identical_on_any_stream(kd, cuda_device, N, V):
    z, tok = draw(N, V, torch.bfloat16, 1), tokens_for(N, V, 2, 1)
    first = run_both(kd, z, tok, top=8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run_both(kd, z, tok, top=8)
    torch.cuda.synchronize()
    for a, b in zip((*first[0], first[1]), (*again[0], again[1])):
        assert torch.equal(a, b)


def test_graph_capture(kd, cuda_device):
    z, tok = draw(4, 40001, torch.bfloat16, 1), tokens_for(4, 40001, 1, 1)
    ws = kd.workspace(kd._abi.kd_token_logprobs_workspace(4, 40001), "cuda")
    want = kd.token_logprobs_forward(z, tok, top=4, entropy=True, ws=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kd.token_logprobs_forward(z, tok, top=4, entropy=True, ws=ws)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_bad_token_is_reported(kd, cuda_device):
    z, tok = draw(6, 100, torch.float32, 1), tokens_for(6, 100, 2, 1)
    tok[4, 1] = 100
    ws = kd.workspace(kd._abi.kd_token_logprobs_workspace(6, 100), "cuda")
    r = kd.token_logprobs_forward(z, tok, ws=ws)
    assert kd.device_error(ws) == (kd._abi.KD_ERR_DEVICE, 4)
    assert torch.isnan(r.logp[4, 1]) and int(torch.isnan(r.logp).sum()) == 1
    dz = kd.token_logprobs_backward(z, tok, r.lse, torch.ones_like(r.logp), ws=ws)
    assert kd.device_error(ws) == (kd._abi.KD_ERR_DEVICE, 4)
    g = np.ones((6, 2))
    g[4, 1] = 0
    tok[4, 1] = 0
    check_grad(dz, oracle.token_logprobs_grad(z.double().cpu().numpy(), tok.cpu().numpy(), g), torch.float32)


def test_control_block_without_a_workspace(kd, cuda_device):
    z, tok = draw(3, 90, torch.float32, 1), tokens_for(3, 90, 1, 1)
    tok[2] = -1
    block = kd.control_block(z.device)
    assert block is kd.control_block(z.device) and kd.device_error(block)[0] == 0
    kd.token_logprobs_forward(z, tok)
    assert kd.device_error(block) == (kd._abi.KD_ERR_DEVICE, 2)
    assert kd.device_error(block)[0] == 0


def test_gradient_matches_differences(kd, cuda_device):
    """Central differences of the fp32 forward: step 1/16, truncation error (step^2 / 6) |f'''| < 7e-4."""
    z, tok = draw(2, 50, torch.float32, 9), tokens_for(2, 50, 1, 3)
    zr = z.clone().requires_grad_(True)
    logp, ent = kd.token_logprobs(zr, tok[:, 0].contiguous(), tau=1.0)
    (logp.sum() + 0.5 * ent.sum()).backward()

    def f(x):
        r = kd.token_logprobs_forward(x, tok, entropy=True)
        return float(r.logp.double().sum() + 0.5 * r.entropy.double().sum())

    step = 1.0 / 16
    for v in [int(tok[0, 0]), 0, 13, 49]:
        hi, lo = z.clone(), z.clone()
        hi[0, v] += step
        lo[0, v] -= step
        assert abs(float(zr.grad[0, v]) - (f(hi) - f(lo)) / (2 * step)) < 3e-3


def test_autograd_with_either_gradient_alone(kd, cuda_device):
    z, tok = draw(3, 777, torch.float32, 2), tokens_for(3, 777, 1, 2)[:, 0].contiguous()
    host = z.double().cpu().numpy()
    for which in (0, 1):
        zr = z.clone().requires_grad_(True)
        kd.token_logprobs(zr, tok)[which].sum().backward()
        one, none = np.ones((3, 1)), np.zeros((3, 1))
        ref = oracle.token_logprobs_grad(host, tok.cpu().numpy(), none if which else one, one[:, 0] if which else None)
        check_grad(zr.grad, ref, torch.float32)
