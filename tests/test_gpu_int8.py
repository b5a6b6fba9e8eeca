"""quantize_int8, gemm_int8 and teacher_topk_int8 against their definitions.

The integers of quantize_int8 are the exact quotients' nearest whole numbers, so float64 (whose quotient of two
fp32 numbers never rounds onto a tie) gives the same ones; its scale is one fp32 division.  The integer sums
of gemm_int8 are exact below 2^24 in any order, and each rounding after them is fixed: (sum a_scale) b_scale in
fp32, then C's type.  So all comparisons are for equality; only sums past 2^24 have a tolerance, K / 16
roundings (one for each 16-deep step) of at most 2^-23.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module")
def kd(cuda_device):
    from sparse_teacher_kl_gb300.build import build_library
    build_library()
    import sparse_teacher_kl_gb300 as kd
    return kd


def gen(seed=0):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(N, K, g, pad=0, start=0):
    """[N, K] integers over the whole range in rows K + pad apart, the first `start` bytes into its memory."""
    buf = torch.randint(-128, 128, (start + N * (K + pad),), generator=g, device="cuda", dtype=torch.int8)
    return buf[start:].view(N, K + pad)[:, :K]


def scales(N, g):
    return torch.rand((N,), generator=g, device="cuda") * 0.02 + 1e-4


def product(A, sa, B, sb, dtype):
    total = A.double() @ B.double().T
    assert float(total.abs().max()) < 2 ** 24
    return ((total.float() * sa[:, None]) * sb[None, :]).to(dtype)


def check(kd, M, N, K, dtype=torch.bfloat16, pad_a=0, pad_b=0, start=0, seed=0):
    g = gen(seed)
    A, B = ints(M, K, g, pad_a, start), ints(N, K, g, pad_b, start)
    sa, sb = scales(M, g), scales(N, g)
    got = kd.gemm_int8(A, sa, B, sb, out_dtype=dtype)
    assert got.dtype == dtype and torch.equal(got, product(A, sa, B, sb, dtype))
    assert kd.device_error(kd.control_block())[0] == 0


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 128, 16), (1, 129, 128), (3, 257, 144), (7, 1000, 4096), (16, 300, 256), (17, 300, 257),
    (33, 640, 1000), (64, 512, 512), (65, 512, 512), (128, 4096, 256), (129, 1001, 1008), (192, 384, 2880),
    (193, 385, 130), (257, 777, 96), (400, 20000, 64), (1000, 300, 1040)])
def test_sizes(kd, cuda_device, M, N, K):
    check(kd, M, N, K, seed=M + N + K)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("M", [1, 5, 40, 100, 300])
def test_types(kd, cuda_device, M, dtype):
    check(kd, M, 700, 352, dtype)


@pytest.mark.parametrize("pad_a,pad_b,start", [(16, 16, 0), (16, 16, 16), (3, 0, 0), (0, 5, 0), (0, 0, 1), (7, 11, 3),
                                               (0, 16, 8), (1, 4, 4), (8, 2, 2)])
@pytest.mark.parametrize("M,N,K", [(1, 500, 100), (9, 300, 333), (150, 260, 1003)])
def test_rows_anywhere(kd, cuda_device, M, N, K, pad_a, pad_b, start):
    check(kd, M, N, K, torch.float32, pad_a, pad_b, start)


@pytest.mark.parametrize("K", [1, 2, 3, 15, 16, 17, 19, 20, 21, 31, 127, 129])
def test_short_rows_end_where_they_should(kd, cuda_device, K):
    for start in range(4):
        check(kd, 4, 37, K, torch.float32, 0, 0, start, seed=K)
        check(kd, 6, 137, K, torch.float32, 0, 0, start, seed=K)
        check(kd, 70, 300, K, torch.bfloat16, 0, 1, start, seed=K)


@pytest.mark.parametrize("M", [1, 3, 7, 70, 300])
def test_every_start_of_a_row(kd, cuda_device, M):
    """Rows that start at each of the 16 places of a piece, at every row of a tile."""
    for start in range(16):
        check(kd, M, 150, 300, torch.float32, 0, 0, start, seed=start)
        check(kd, M, 150, 272, torch.float32, 0, start, 0, seed=start)


@pytest.mark.parametrize("dtype", TYPES)
def test_output_of_the_callers(kd, cuda_device, dtype):
    g = gen(3)
    for M, pad in ((1, 1), (6, 3), (130, 5)):
        A, B, sa, sb = ints(M, 200, g), ints(333, 200, g), scales(M, g), scales(333, g)
        room = torch.full((M + 2, 333 + pad), 7.0, dtype=dtype, device="cuda")
        out = room[1:M + 1, :333]
        before = room._version
        assert kd.gemm_int8(A, sa, B, sb, out=out) is out and room._version > before
        assert torch.equal(out, product(A, sa, B, sb, dtype))
        assert (room[0] == 7).all() and (room[-1] == 7).all() and (room[:, 333:] == 7).all()


@pytest.mark.parametrize("M", [2, 20, 200])
def test_sums_past_2_24(kd, cuda_device, M):
    K = 4099
    A = torch.full((M, K), 127, dtype=torch.int8, device="cuda")
    B = torch.full((300, K), -128, dtype=torch.int8, device="cuda")
    A[:, ::7] = 113
    one = lambda n: torch.ones((n,), device="cuda")
    got = kd.gemm_int8(A, one(M), B, one(300), out_dtype=torch.float32).double()
    want = A.double() @ B.double().T
    assert ((got - want).abs() <= want.abs() * (K / 16 + 1) * 2.0 ** -23).all()


def test_scales_pass_through(kd, cuda_device):
    g = gen(5)
    for M in (3, 100):
        A, B, sa, sb = ints(M, 64, g), ints(200, 64, g), scales(M, g), scales(200, g)
        sa[1], sb[2] = float("nan"), 0.0
        got = kd.gemm_int8(A, sa, B, sb, out_dtype=torch.float32)
        assert torch.isnan(got[1]).all() and not got[0, 2] and torch.isfinite(got[0]).all()


def quantized(x):
    x = x.double()
    most = x.abs().amax(dim=1)
    scale = (most / torch.full_like(most, 127.0)).float()
    s = scale.double()[:, None]
    q = torch.where(s > 0, x / s, torch.zeros_like(x)).round().clamp(-127, 127)
    return q.to(torch.int8), scale


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("N,d,pad", [(1, 1, 0), (1, 2880, 0), (3, 7, 1), (5, 1003, 3), (700, 4096, 0), (64, 8192, 8),
                                     (3, 40001, 0), (2000, 16, 0), (33, 256, 5), (4, 12000, 4)])
def test_quantize(kd, cuda_device, N, d, pad, dtype):
    x = torch.empty((N, d + pad), dtype=dtype, device="cuda")[:, :d]
    x.copy_(torch.randn((N, d), generator=gen(d), device="cuda") * 3)
    q, scale = kd.quantize_int8(x)
    rq, rs = quantized(x)
    assert torch.equal(scale, rs) and torch.equal(q, rq)


def test_quantize_ties(kd, cuda_device):
    """With a largest value of 127 * 2^e the scale is 2^e: halves are ties, and their fp32 neighbours are not."""
    steps = torch.arange(-254, 255, device="cuda", dtype=torch.float32) / 2
    for e in (-126, -30, 0, 5, 100):
        x = torch.stack([steps, torch.nextafter(steps, steps + 1), torch.nextafter(steps, steps - 1)])
        x[:, 0], x[:, -1] = -127, 127
        x = x * 2.0 ** e
        q, scale = kd.quantize_int8(x)
        rq, rs = quantized(x)
        assert torch.equal(scale, rs) and torch.equal(q, rq)
    # scales that are no powers of two, where x / s rounds onto a half now and then
    g = gen(9)
    x = torch.randn((4000, 300), generator=g, device="cuda")
    s = x.abs().amax(1, keepdim=True) / 127
    x[:, 1:] = ((torch.randint(-126, 127, (4000, 299), generator=g, device="cuda") + 0.5) * s).clamp(-s * 127, s * 127)
    q, scale = kd.quantize_int8(x)
    rq, rs = quantized(x)
    assert torch.equal(scale, rs) and torch.equal(q, rq)


def test_quantize_odd_rows(kd, cuda_device):
    x = torch.randn((8, 300), generator=gen(1), device="cuda")
    x[0] = 0
    x[1, 299] = float("inf")
    x[2, 0] = float("nan")
    x[3, 5] = -float("inf")
    x[4] = 0
    x[4, 7] = -2.0 ** -149     # its scale rounds to 0
    x[5] *= 1e-40              # subnormal
    x[6] *= 3e37
    q, scale = kd.quantize_int8(x)
    rq, rs = quantized(x[4:])
    assert not scale[0] and not q[0].any()
    assert torch.isnan(scale[1:4]).all() and not q[1:4].any()
    assert torch.equal(scale[4:], rs) and torch.equal(q[4:], rq)


def test_quantize_into_the_callers(kd, cuda_device):
    x = torch.randn((9, 100), generator=gen(2), device="cuda").to(torch.bfloat16)
    room = torch.full((9, 107), 5, dtype=torch.int8, device="cuda")
    scale = torch.empty((9,), device="cuda")
    q, s = kd.quantize_int8(x, q=room[:, :100], scale=scale)
    rq, rs = quantized(x)
    assert s is scale and torch.equal(q, rq) and torch.equal(scale, rs) and (room[:, 100:] == 5).all()


@pytest.mark.parametrize("N,d,V,K,chunk", [(1, 64, 1000, 10, 1024), (70, 96, 3000, 100, 32), (130, 200, 1111, 33, 1024),
                                           (67, 101, 700, 20, 32), (9, 64, 500, 7, 4), (5, 33, 400, 5, 2)])
@pytest.mark.parametrize("pad", [0, 3])
def test_teacher(kd, cuda_device, N, d, V, K, chunk, pad):
    """Quantised states and head to a cache: the top-K of the bf16 logits that the product's definition gives."""
    g = gen(N)
    H = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
    W = (torch.randn((V, d), generator=g, device="cuda") * 0.1).to(torch.bfloat16)
    h8, hs = kd.quantize_int8(H)
    w8 = torch.empty((V, d + pad), dtype=torch.int8, device="cuda")[:, :d]
    w8, ws = kd.quantize_int8(W, q=w8)
    z = torch.full((N, (V + 7) // 8 * 8), float("-inf"), dtype=torch.bfloat16, device="cuda")
    z[:, :V] = product(h8, hs, w8, ws, torch.bfloat16)
    ids, vals, lse, dropped = kd.teacher_topk_int8(h8, hs, w8, ws, K, chunk=chunk, with_lse=True, with_dropped=True)
    want, wid = torch.sort(z, dim=1, descending=True, stable=True)
    assert torch.equal(vals, want[:, :K].float()) and torch.equal(ids.long(), wid[:, :K])
    ref = z.double().logsumexp(1)
    assert ((lse.double() - ref).abs() < 1e-5 * (1 + ref.abs())).all()
    rest = 1 - (vals.double() - ref[:, None]).exp().sum(1)
    assert ((dropped.double() - rest).abs() < 1e-5).all()
    a, b = kd.teacher_topk_int8(h8, hs, w8, ws, K, chunk=chunk)
    assert torch.equal(a, ids) and torch.equal(b, vals)


def test_quantised_teacher_then_distillation(kd, cuda_device):
    """As used together: a quantised teacher's cache, the student's KL term against it and the hard-label term."""
    g = gen(11)
    N, d, V = 200, 128, 900
    Ht = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
    Wt = (torch.randn((V, d), generator=g, device="cuda") * 0.2).to(torch.bfloat16)
    ids, vals = kd.teacher_topk_int8(*kd.quantize_int8(Ht), *kd.quantize_int8(Wt), K=50)
    H, W = Ht.clone().requires_grad_(), Wt.clone().requires_grad_()
    labels = ids[:, 0].contiguous()
    labels[::5] = -100
    kl = kd.fused_kl(H, W, ids, vals, chunk=128)
    ce = kd.fused_cross_entropy(H, W, labels, chunk=256)
    loss = 0.5 * kl + 0.5 * ce
    gH, gW = torch.autograd.grad(loss, (H, W))
    z = (Ht.double() @ Wt.double().T)
    z.requires_grad_()
    lp = z.log_softmax(1)
    t = vals.double().log_softmax(1)
    kl_r = (t.exp() * (t - lp.gather(1, ids.long()))).sum(1).mean()
    keep = labels >= 0
    ce_r = -lp.gather(1, labels.clamp(min=0).long()[:, None])[keep].mean()
    assert abs(float(kl) - float(kl_r)) < 5e-4 and abs(float(ce) - float(ce_r)) < 5e-4
    (dz,) = torch.autograd.grad(0.5 * kl_r + 0.5 * ce_r, z)
    for got, ref in ((gH, dz @ Wt.double()), (gW, dz.T @ Ht.double())):
        assert float((got.double() - ref).abs().max()) <= 1e-2 * float(ref.abs().max())


@pytest.mark.parametrize("M", [1, 30, 300])
def test_captured_and_replayed(kd, cuda_device, M):
    g = gen(M)
    x = torch.randn((M, 300), generator=g, device="cuda").to(torch.bfloat16)
    B, sb = ints(500, 300, g), scales(500, g)
    call = lambda: kd.gemm_int8(*kd.quantize_int8(x), B, sb, out_dtype=torch.float32)
    call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        call()
    torch.cuda.current_stream().wait_stream(s)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    outs = []
    for graph in graphs:
        with torch.cuda.graph(graph):
            outs.append(call())
    for _ in range(2):
        x.copy_(torch.randn((M, 300), generator=g, device="cuda"))
        want = product(*quantized(x), B, sb, torch.float32)
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)


def test_two_streams(kd, cuda_device):
    g = gen(8)
    args = [(ints(M, 515, g), scales(M, g), ints(2000, 515, g), scales(2000, g)) for M in (200, 5)]
    want = [product(*a, torch.float32) for a in args]
    streams = [torch.cuda.Stream() for _ in args]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for a, s in zip(args, streams):
            with torch.cuda.stream(s):
                got.append(kd.gemm_int8(*a, out_dtype=torch.float32))
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_offsets_past_32_bits(kd, cuda_device):
    """An output of more than 2^32 elements, and weights of more than 2^32 bytes, checked where they end."""
    g = gen(4)
    M, N, K = 4000, 1100000, 32
    A, B, sa, sb = ints(M, K, g), ints(N, K, g), scales(M, g), scales(N, g)
    out = kd.gemm_int8(A, sa, B, sb)
    for rows, cols in ((slice(M - 40, M), slice(N - 1000, N)), (slice(0, 40), slice(0, 1000))):
        assert torch.equal(out[rows, cols], product(A[rows], sa[rows], B[cols], sb[cols], torch.bfloat16))
    del out
    wide = torch.empty((70000, 65536), dtype=torch.int8, device="cuda")
    tail = ints(1000, 65536, g)
    wide[-1000:] = tail >> 6
    sb = scales(70000, g)
    A = ints(3, 65536, g) >> 2
    out = kd.gemm_int8(A, sa[:3].contiguous(), wide, sb, out_dtype=torch.float32)
    assert torch.equal(out[:, -1000:], product(A, sa[:3], wide[-1000:], sb[-1000:], torch.float32))
