"""What the cross entropy and the 8-bit products are measured on: cases, inputs, plain forms, 64-bit values.

Three operators around a language model's output head:

  ce_eval / ce_step / ce_train   fused_cross_entropy: softmax cross entropy against hard labels straight from
                       hidden states and the head (label smoothing, z-loss, softcap, ignored labels), the [N, V]
                       logits never kept; its loss alone, loss and gradients in one call, and under autograd
  quantize             quantize_int8: rows to 8-bit integers with one scale each
  gemm8 / project8     gemm_int8: the product of 8-bit integers with a scale for each token and channel;
                       project8 is the pair as a quantised head runs it, from bf16 hidden states

``own`` chooses the side that ``run`` takes: the plain torch form below, or the package.
"""
import math

import torch

own = False

F32 = torch.float32
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CHUNK = 8192      # positions per chunk of the fused operator: one chunk, so that grad_W is stored once
IGNORED = -100    # label of a position without a loss


# ------------------------------------------------------------------------- cases

def listed():
    ce = dict(valid=1.0, smooth=0.0, z_loss=0.0, cap=0.0)
    return [
        # the smallest training step: latency
        dict(ce, name="ce_step_tiny", op="ce_step", N=128, d=256, V=4096),
        # held-out loss of a model with capped logits and smoothed labels, odd sizes, padding
        dict(ce, name="ce_eval_odd", op="ce_eval", N=509, d=1000, V=50257, valid=0.9, smooth=0.1, cap=30.0),
        # the small language model's step with padding, smoothed labels and a z-loss
        dict(ce, name="ce_step_small", op="ce_step", N=8192, d=2048, V=32000, valid=0.95, smooth=0.1, z_loss=1e-4),
        # instruction tuning: the labels of the prompt's positions are ignored
        dict(ce, name="ce_step_prompt", op="ce_step", N=4096, d=4096, V=151936, valid=0.35),
        # forward and backward as an autograd graph runs them, the largest head
        dict(ce, name="ce_train_large", op="ce_train", N=4096, d=2880, V=201088, z_loss=1e-4),
        # one token's hidden state quantised: latency
        dict(name="quantize_token", op="quantize", type="bf16", N=1, d=2880, pad=0),
        # a batch of prompts' hidden states
        dict(name="quantize_batch", op="quantize", type="bf16", N=8192, d=4096, pad=0),
        # one generated token projected by a quantised head, its activations quantised on the way
        dict(name="project8_token", op="project8", type="bf16", M=1, K=2880, N=201088, pad=0),
        # a handful of sequences decoded together
        dict(name="gemm8_few", op="gemm8", type="fp16", M=7, K=4096, N=151936, pad=0),
        # odd sizes throughout (rows start unaligned), fp32 logits
        dict(name="gemm8_odd", op="gemm8", type="fp32", M=257, K=1003, N=50257, pad=0),
        # the small language model's head over a prompt
        dict(name="gemm8_small", op="gemm8", type="bf16", M=2048, K=2048, N=32000, pad=0),
        # a chunk of a teacher's positions projected by its quantised head
        dict(name="project8_prompt", op="project8", type="bf16", M=4096, K=2880, N=201088, pad=0),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["ce_eval", "ce_step", "ce_step", "ce_train", "quantize", "gemm8", "gemm8", "project8"])
    if op == "quantize":
        d = spread(1, 8192) if rng.random() < 0.6 else 8 * spread(8, 1024)
        return dict(op=op, type=rng.choice(["bf16", "bf16", "fp16", "fp32"]), N=spread(1, max(2, min(16384, int(3e7 / d)))),
                    d=d, pad=rng.choice([0, 0, 3, 16]))
    V = spread(1000, 201088) if rng.random() < 0.75 else rng.choice([4096, 32000, 151936, 201088])
    if op in ("gemm8", "project8"):
        K = 16 * spread(4, 256) if rng.random() < 0.7 else spread(64, 4096)
        most = 4096 * 2880 * 201088
        M = spread(1, max(2, min(4096, int(most / (K * V)))))
        return dict(op=op, type=rng.choice(["bf16", "bf16", "fp16", "fp32"]), M=M, K=K, N=V, pad=rng.choice([0, 0, 5, 16]))
    d = 8 * spread(8, 512)
    most = 4096 * 2880 * 201088 / (1 if op != "ce_eval" else 1.5)
    N = spread(1 if op == "ce_eval" else 16, max(17, min(8192, int(most / (d * V)))))
    return dict(op=op, N=N, d=d, V=V, valid=rng.choice([1.0, round(rng.uniform(0.2, 0.98), 2)]),
                smooth=rng.choice([0.0, 0.0, 0.1]), z_loss=rng.choice([0.0, 1e-4]), cap=rng.choice([0.0, 0.0, 30.0]))


# ------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 29)
    return g


def _rows(N, d, pad, dtype):
    """An [N, d] matrix whose rows are `pad` elements further apart than they are long."""
    return torch.empty((N, d + pad), dtype=dtype, device="cuda")[:, :d]


def prepare(case, seed):
    g = _gen(seed)
    op, N = case["op"], case["N"]
    if op.startswith("ce"):
        d, V = case["d"], case["V"]
        H = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
        W = torch.empty((V, d), dtype=torch.bfloat16, device="cuda").normal_(0.0, 1.5 / math.sqrt(d), generator=g)
        labels = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
        # a model in training has learnt something: two thirds of the hidden states lean towards their label
        lean = (torch.rand((N,), generator=g, device="cuda") < 0.67).float() * 4.0
        H = (H.float() + lean[:, None] * W[labels.long()].float()).to(torch.bfloat16)
        drop = torch.rand((N,), generator=g, device="cuda") >= case["valid"]
        labels.masked_fill_(drop, IGNORED)
        return dict(op=op, H=H, W=W, labels=labels, smooth=case["smooth"], z_loss=case["z_loss"], cap=case["cap"])
    dtype = TYPES[case["type"]]
    if op == "quantize":
        # hidden states: normal, with a few channels far larger than the rest
        x = _rows(N, case["d"], case["pad"], dtype)
        far = 1.0 + 15.0 * (torch.rand((case["d"],), generator=g, device="cuda") < 0.01).float()
        x.copy_(torch.randn((N, case["d"]), generator=g, device="cuda") * far)
        return dict(op=op, x=x)
    M, K = case["M"], case["K"]
    w = torch.empty((N, K), dtype=torch.bfloat16, device="cuda").normal_(0.0, 1.5 / math.sqrt(K), generator=g)
    B = _rows(N, K, case["pad"], torch.int8)
    b_scale = torch.empty((N,), dtype=F32, device="cuda")
    step = max(1, int(1e8 // K))
    for a in range(0, N, step):
        q, b_scale[a:a + step] = _quantized(w[a:a + step])
        B[a:a + step] = q
    del w
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    s = dict(op=op, B=B, b_scale=b_scale, dtype=dtype)
    if op == "project8":
        s["x"] = x
    else:
        s["A"] = _rows(M, K, case["pad"], torch.int8)
        q, s["a_scale"] = _quantized(x)
        s["A"].copy_(q)
    return s


# ------------------------------------------------------------------------- the operators

def run(s):
    return (_package if own else _plain)[s["op"]](s)


# ---- plain forms: 32 bits throughout (64 where a rounding to whole numbers is decided), one rounding at the end

def _capped(z, cap):
    return cap * torch.tanh(z / cap) if cap else z


def _losses(s):
    """Capped logits, logsumexp, log softmax and the loss of every position (0 where the label is ignored)."""
    z = _capped(s["H"].float() @ s["W"].float().T, s["cap"])
    m = z.amax(dim=1)
    lp = z - m[:, None]
    log_sum = torch.log(torch.exp(lp).sum(dim=1))
    lp -= log_sum[:, None]
    lse = m + log_sum
    on = s["labels"] != IGNORED
    at = torch.where(on, s["labels"], 0).long()[:, None]
    nll = -lp.gather(1, at)[:, 0]
    if s["smooth"]:
        nll = (1.0 - s["smooth"]) * nll - s["smooth"] * lp.mean(dim=1)
    each = nll + s["z_loss"] * lse * lse
    n = on.sum().clamp(min=1)
    each = torch.where(on, each, torch.zeros_like(each))
    return z, lse, lp, on, at, n, each


def _plain_eval(s):
    _, _, _, _, _, n, each = _losses(s)
    return dict(loss=each.sum() / n, losses=each)


def _plain_train(s):
    z, lse, lp, on, at, n, each = _losses(s)
    dz = torch.exp(lp) * (1.0 + 2.0 * s["z_loss"] * lse)[:, None]
    if s["smooth"]:
        dz -= s["smooth"] / z.shape[1]
    dz.scatter_add_(1, at, torch.full_like(lse, -(1.0 - s["smooth"]))[:, None])
    if s["cap"]:
        dz *= 1.0 - (z / s["cap"]) ** 2
    dz = torch.where(on[:, None], dz / n, torch.zeros_like(dz))
    out = dict(loss=each.sum() / n, grad_H=(dz @ s["W"].float()).to(torch.bfloat16),
               grad_W=(dz.T @ s["H"].float()).to(torch.bfloat16))
    if s["op"] == "ce_step":
        out["losses"] = each
    return out


def _quantized(x):
    """(8-bit integers, scales): x / scale to the nearest whole number, ties to even, of the exact quotient."""
    most = x.abs().amax(dim=1).float()
    scale = most / torch.full_like(most, 127.0)   # by a tensor: by a number it would be a product with 1 / 127
    quotient = x.double() / torch.where(scale > 0, scale, torch.ones_like(scale)).double()[:, None]
    return torch.round(quotient).clamp(-127, 127).to(torch.int8), scale


def _product(A, a_scale, B, b_scale, dtype):
    """Whole numbers below 2^24 are exact in 32-bit floating point: the sums of these products are too."""
    return ((A.float() @ B.float().T) * a_scale[:, None] * b_scale[None, :]).to(dtype)


def _plain_quantize(s):
    q, scale = _quantized(s["x"])
    return dict(q=q, scale=scale)


def _plain_gemm8(s):
    return dict(out=_product(s["A"], s["a_scale"], s["B"], s["b_scale"], s["dtype"]))


def _plain_project8(s):
    return dict(out=_product(*_quantized(s["x"]), s["B"], s["b_scale"], s["dtype"]))


_plain = dict(ce_eval=_plain_eval, ce_step=_plain_train, ce_train=_plain_train, quantize=_plain_quantize,
              gemm8=_plain_gemm8, project8=_plain_project8)


# ---- the package's operators, as a user calls them

def _options(s):
    return dict(chunk=CHUNK, label_smoothing=s["smooth"], z_loss=s["z_loss"], softcap=s["cap"], ignore_index=IGNORED)


def _package_eval(s):
    import sparse_teacher_kl_gb300 as kd
    each = torch.empty((s["H"].shape[0],), dtype=F32, device=s["H"].device)
    loss, _, _ = kd.fused_cross_entropy_forward(s["H"], s["W"], s["labels"], **_options(s), loss_out=each)
    return dict(loss=loss[0], losses=each)


def _package_step(s):
    import sparse_teacher_kl_gb300 as kd
    each = torch.empty((s["H"].shape[0],), dtype=F32, device=s["H"].device)
    loss, gH, gW = kd.fused_cross_entropy_step(s["H"], s["W"], s["labels"], **_options(s), loss_out=each,
                                               grad_W_bf16=True)
    return dict(loss=loss[0], grad_H=gH, grad_W=gW, losses=each)


def _package_train(s):
    import sparse_teacher_kl_gb300 as kd
    H, W = s["H"].detach().requires_grad_(True), s["W"].detach().requires_grad_(True)
    loss = kd.fused_cross_entropy(H, W, s["labels"], **_options(s))
    gH, gW = torch.autograd.grad(loss, (H, W))
    return dict(loss=loss.detach(), grad_H=gH, grad_W=gW)


def _package_quantize(s):
    import sparse_teacher_kl_gb300 as kd
    q, scale = kd.quantize_int8(s["x"])
    return dict(q=q, scale=scale)


def _package_gemm8(s):
    import sparse_teacher_kl_gb300 as kd
    return dict(out=kd.gemm_int8(s["A"], s["a_scale"], s["B"], s["b_scale"], out_dtype=s["dtype"]))


def _package_project8(s):
    import sparse_teacher_kl_gb300 as kd
    q, scale = kd.quantize_int8(s["x"])
    return dict(out=kd.gemm_int8(q, scale, s["B"], s["b_scale"], out_dtype=s["dtype"]))


_package = dict(ce_eval=_package_eval, ce_step=_package_step, ce_train=_package_train, quantize=_package_quantize,
                gemm8=_package_gemm8, project8=_package_project8)


# ------------------------------------------------------------------------- the work of one pass

def work(case):
    """Each input read once (ignored positions' hidden states are not needed), each output written once."""
    op, N = case["op"], case["N"]
    if op.startswith("ce"):
        d, V, rows = case["d"], case["V"], case["N"] * case["valid"]
        train = op != "ce_eval"
        return dict(bytes=2.0 * (rows + V) * d + N * 8.0 + (2.0 * (N + V) * d if train else 0.0),
                    flops=2.0 * rows * d * V * (3 if train else 1))
    size = 4 if case["type"] == "fp32" else 2
    if op == "quantize":
        return dict(bytes=N * case["d"] * (size + 1.0) + 4.0 * N, flops=3.0 * N * case["d"])
    M, K = case["M"], case["K"]
    read = M * K * (2.0 if op == "project8" else 1.0) + float(N) * K + 4.0 * N + (0.0 if op == "project8" else 4.0 * M)
    return dict(bytes=read + float(M) * N * size, flops=2.0 * M * N * K)


# ------------------------------------------------------------------------- values in 64 bits

def exact(case, seed):
    """The definitions in float64, written out row block by row block from the inputs alone."""
    s = prepare(case, seed)
    if case["op"].startswith("ce"):
        return _exact_ce(s)
    if case["op"] == "quantize":
        q, scale = _exact_quantize(s["x"])
        return dict(q=q.to(torch.int8), scale=scale)
    A, a = (s["A"].double(), s["a_scale"].double()) if case["op"] == "gemm8" else _exact_quantize(s["x"])
    b = s["b_scale"].double()
    N = b.shape[0]
    out = torch.empty((A.shape[0], N), dtype=torch.float64, device="cuda")
    step = max(1, int(2e8 // A.shape[1]))
    for lo in range(0, N, step):
        out[:, lo:lo + step] = (A @ s["B"][lo:lo + step].double().T) * (a[:, None] * b[lo:lo + step])
    return dict(out=out)


def _exact_quantize(x):
    """The scale is a 32-bit number (it is what the integers are multiples of)."""
    x = x.double()
    most = x.abs().max(dim=1).values
    scale = (most / torch.full_like(most, 127.0)).float().double()
    q = torch.where(scale[:, None] > 0, x / scale[:, None], torch.zeros_like(x)).round()
    return q.clamp(-127.0, 127.0), scale


def _exact_ce(s):
    labels, W = s["labels"].long(), s["W"].double()
    N, V, e, c = labels.shape[0], W.shape[0], s["smooth"], s["cap"]
    live = (labels != IGNORED).nonzero()[:, 0]
    n = max(1, live.shape[0])
    train = s["op"] != "ce_eval"
    losses = torch.zeros(N, dtype=torch.float64, device="cuda")
    gH = torch.zeros((N, W.shape[1]), dtype=torch.float64, device="cuda") if train else None
    gW = torch.zeros_like(W) if train else None
    for rows in live.split(max(1, int(1e8 // V))):
        h, y = s["H"][rows].double(), labels[rows][:, None]
        z = h @ W.T
        slope = None
        if c:
            t = (z / c).tanh()
            z, slope = c * t, 1.0 - t * t
        lse = z.logsumexp(dim=1)
        losses[rows] = lse - (1.0 - e) * z.gather(1, y)[:, 0] - e * z.mean(dim=1) + s["z_loss"] * lse ** 2
        if train:
            g = (z - lse[:, None]).exp() * (1.0 + 2.0 * s["z_loss"] * lse[:, None]) - e / V
            g.scatter_add_(1, y, torch.full(y.shape, e - 1.0, dtype=torch.float64, device="cuda"))
            if slope is not None:
                g *= slope
            g /= n
            gH[rows] = g @ W
            gW += g.T @ h
    out = dict(loss=losses.sum() / n)
    if s["op"] != "ce_train":
        out["losses"] = losses
    if train:
        out.update(grad_H=gH, grad_W=gW)
    return out
