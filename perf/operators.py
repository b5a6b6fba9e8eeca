"""What the scoring and distillation operators are measured on: cases, inputs, plain forms, 64-bit values.

Three operators that read a language model's output layer, each in both directions:

  score / score_grad   token_logprobs: from dense logits [N, V], the log probabilities of given
                       tokens, the entropy and the top alternatives; the gradient of the logits
  kl_step / kl_grads   logits_kl: KL against a teacher's cached top logits on dense student
                       logits, optionally with the teacher's remaining mass as one more class
  fused / fused_train  fused_logprobs: log probability of the target and entropy straight from
                       hidden states and the LM head, the [N, V] logits never stored

``own`` chooses the side that ``run`` takes: the plain torch form below, or the package.
"""
import math

import torch

own = False

F32 = torch.float32
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
CHUNK = 4096   # positions per chunk of the fused operator


# ------------------------------------------------------------------------- cases

def listed():
    dense = dict(type="bf16", M=1, top=0, tau=1.0, valid=1.0, banned=0.0)
    kl = dict(type="bf16", K=100, tau=1.0, valid=1.0, tail=False)
    fused = dict(tau=1.0, valid=1.0)
    return [
        # one sampled token reported with its log probability and 20 alternatives: latency
        dict(dense, name="score_token", op="score", N=1, V=201088, top=20),
        # a prompt scored in one call, five alternatives for each position
        dict(dense, name="score_prompt", op="score", N=4096, V=151936, top=5),
        # four candidate answers per position from fp32 logits, odd vocabulary (rows start unaligned),
        # padding, and an eighth of the vocabulary banned
        dict(dense, name="score_odd", op="score", type="fp32", N=509, V=50257, M=4, tau=0.7, valid=0.9,
             banned=0.125),
        # policy-gradient backward with an entropy bonus, the forward pass's logsumexp and entropy kept
        dict(dense, name="policy_grad", op="score_grad", N=4096, V=151936),
        # the same for fp16 logits of an odd vocabulary, three scored tokens per position
        dict(dense, name="policy_grad_odd", op="score_grad", type="fp16", N=257, V=32003, M=3, tau=1.3, valid=0.8),
        # the smallest distillation step: loss and gradient in one call
        dict(kl, name="kl_step_tiny", op="kl_step", N=128, V=4096, K=16),
        # the small language model's step with padding
        dict(kl, name="kl_step_small", op="kl_step", N=8192, V=32000, valid=0.95),
        # a large vocabulary, the teacher's mass outside its cached logits kept as one class
        dict(kl, name="kl_step_tail", op="kl_step", N=4096, V=201088, tail=True),
        # forward and backward as an autograd graph runs them: fp32, odd sizes, a temperature
        dict(kl, name="kl_grads_odd", op="kl_grads", type="fp32", N=300, V=50257, K=33, tau=2.0, tail=True,
             valid=0.9),
        # one generated token scored from its hidden state: the head's weights are read once
        dict(fused, name="fused_token", op="fused", N=1, d=2880, V=201088),
        # a prompt scored from hidden states
        dict(fused, name="fused_score", op="fused", N=4096, d=2880, V=201088),
        # the hard-label term of the small language model's step, with padding
        dict(fused, name="fused_train", op="fused_train", N=8192, d=2048, V=32000, valid=0.95),
    ]


def draw(rng):
    def spread(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["score", "score", "score_grad", "kl_step", "kl_step", "kl_grads", "fused", "fused_train"])
    V = spread(1000, 201088) if rng.random() < 0.75 else rng.choice([4096, 32000, 151936, 201088])
    tau = rng.choice([1.0, 1.0, round(rng.uniform(0.5, 2.0), 2)])
    valid = rng.choice([1.0, round(rng.uniform(0.5, 0.98), 2)])
    if op in ("fused", "fused_train"):
        d = 8 * spread(8, 512)
        most = 4096 * 2880 * 201088 / (1 if op == "fused" else 6)
        N = spread(1 if op == "fused" else 16, max(17, min(8192, int(most / (d * V)))))
        return dict(op=op, N=N, d=d, V=V, tau=tau, valid=valid)
    kind = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    N = spread(1, max(2, min(8192, int(2.5e8 / V))))
    if op in ("score", "score_grad"):
        top = rng.choice([0, 1, 5, 20, spread(1, 64)]) if op == "score" else 0
        return dict(op=op, type=kind, N=N, V=V, M=rng.choice([1, 1, 2, spread(1, 16)]), top=top, tau=tau,
                    valid=valid, banned=rng.choice([0.0, 0.0, 0.5]))
    return dict(op=op, type=kind, N=N, V=V, K=min(V, rng.choice([100, spread(1, 256)])), tau=tau, valid=valid,
                tail=rng.random() < 0.5)


# ------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _mask(case, g):
    if case["valid"] >= 1.0:
        return None
    return (torch.rand((case["N"],), generator=g, device="cuda") < case["valid"]).to(torch.uint8)


def _distinct(N, K, V, g):
    """K distinct ids per row: one in each of K equal ranges of the vocabulary, in random order."""
    lo = torch.arange(K, device="cuda") * V // K
    hi = torch.arange(1, K + 1, device="cuda") * V // K
    ids = lo + (torch.rand((N, K), generator=g, device="cuda") * (hi - lo)).long().clamp(max=hi - lo - 1)
    at = torch.argsort(torch.rand((N, K), generator=g, device="cuda"), dim=1)
    return ids.gather(1, at).to(torch.int32).contiguous()


def _logits(N, V, dtype, g):
    """Dense logits N(0, 2) with a handful of likely tokens per row, as a model emits them."""
    z = torch.randn((N, V), generator=g, device="cuda", dtype=torch.bfloat16 if dtype == torch.bfloat16 else F32)
    z *= math.sqrt(2.0)
    likely = torch.randint(0, V, (N, 8), generator=g, device="cuda")
    z.scatter_(1, likely, (torch.randn((N, 8), generator=g, device="cuda") * 2.0 + 9.0).to(z.dtype))
    return z.to(dtype), likely


def prepare(case, seed):
    g = _gen(seed)
    op, N, V = case["op"], case["N"], case["V"]
    s = dict(op=op, tau=case["tau"], mask=_mask(case, g))
    if op in ("fused", "fused_train"):
        d = case["d"]
        s["H"] = torch.randn((N, d), generator=g, device="cuda").to(torch.bfloat16)
        s["W"] = torch.empty((V, d), dtype=torch.bfloat16, device="cuda").normal_(0.0, 1.5 / math.sqrt(d), generator=g)
        s["tokens"] = torch.randint(0, V, (N,), generator=g, device="cuda", dtype=torch.int32)
        if op == "fused_train":
            s["g_logp"] = torch.randn((N,), generator=g, device="cuda") * 0.5 - 1.0
            s["g_ent"] = torch.randn((N,), generator=g, device="cuda") * 0.01
        return s
    dtype = TYPES[case["type"]]
    s["z"], likely = _logits(N, V, dtype, g)
    if op in ("score", "score_grad"):
        M = case["M"]
        other = torch.randint(0, V, (N, M), generator=g, device="cuda")
        pick = torch.rand((N, M), generator=g, device="cuda") < 0.7
        s["tokens"] = torch.where(pick, likely[:, torch.arange(M, device="cuda") % 8], other).to(torch.int32)
        s["top"] = case["top"]
        if case["banned"] > 0:
            out = torch.rand((V,), generator=g, device="cuda") < case["banned"]
            s["z"].masked_fill_(out[None, :], -math.inf)
            s["z"][:, 0] = 0.5
        if op == "score_grad":
            s["g_logp"] = torch.randn((N, M), generator=g, device="cuda") * 0.5 - 1.0
            s["g_ent"] = torch.randn((N,), generator=g, device="cuda") * 0.01
            s["lse"], s["entropy"] = _lse_entropy(s["z"].float() / s["tau"])
        return s
    K = case["K"]
    s["ids"] = _distinct(N, K, V, g)
    r = torch.arange(1, K + 1, device="cuda", dtype=F32)
    noise = torch.randn((N, K), generator=g, device="cuda") * math.sqrt(0.5)
    s["tlog"] = torch.sort(8.0 - 1.5 * torch.log(r) + noise, dim=1, descending=True)[0].contiguous()
    near = s["tlog"] + torch.randn((N, K), generator=g, device="cuda")
    s["z"].scatter_(1, s["ids"].long(), near.to(dtype))
    s["t_lse"] = None
    if case["tail"]:
        rest = 0.01 + 0.3 * torch.rand((N,), generator=g, device="cuda")
        s["t_lse"] = _lse(s["tlog"] / s["tau"]) - torch.log1p(-rest)
    s["grad"] = torch.full((1,), 0.5, dtype=F32, device="cuda")
    return s


# ------------------------------------------------------------------------- the operators

def run(s):
    return (_package if own else _plain)[s["op"]](s)


def _keep(**out):
    return {k: v for k, v in out.items() if v is not None}


# ---- plain forms: 32 bits throughout, one rounding at the end

def _lse(x):
    m = x.amax(dim=1)
    return m + torch.log(torch.exp(x - m[:, None]).sum(dim=1))


def _lse_entropy(x):
    lse = _lse(x)
    lp = x - lse[:, None]
    p = torch.exp(lp)
    return lse, -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(dim=1)


def _rows(x, mask):
    if mask is None:
        return x
    keep = mask.bool()
    return torch.where(keep if x.dim() == 1 else keep[:, None], x, torch.zeros_like(x))


def _top(z, n):
    """The n largest of each row, equal ones by ascending column."""
    bits = (z + 0.0).view(torch.int32).long()
    order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits)
    column = torch.arange(z.shape[1], device=z.device)
    key = torch.topk(order * (1 << 32) + (0xFFFFFFFF - column), n, dim=1)[0]
    ids = 0xFFFFFFFF - (key & 0xFFFFFFFF)
    return ids.to(torch.int32), z.gather(1, ids)


def _plain_score(s):
    z, mask = s["z"].float(), s["mask"]
    x = z / s["tau"]
    lse, ent = _lse_entropy(x)
    logp = x.gather(1, s["tokens"].long()) - lse[:, None]
    ids = top = None
    if s["top"]:
        ids, vals = _top(z, s["top"])
        top = _rows(vals / s["tau"] - lse[:, None], mask)
        ids = _rows(ids, mask)
    return _keep(logp=_rows(logp, mask), entropy=_rows(ent, mask), top_ids=ids, top_logp=top)


def _plain_score_grad(s):
    x = s["z"].float() / s["tau"]
    lp = x - s["lse"][:, None]
    p = torch.exp(lp)
    slope = torch.where(p > 0, p * (lp + s["entropy"][:, None]), torch.zeros_like(p))
    dz = -p * s["g_logp"].sum(dim=1, keepdim=True) - s["g_ent"][:, None] * slope
    dz.scatter_add_(1, s["tokens"].long(), s["g_logp"])
    return dict(grad=_rows(dz / s["tau"], s["mask"]).to(s["z"].dtype))


def _plain_kl(s):
    x, ids, mask = s["z"].float() / s["tau"], s["ids"].long(), s["mask"]
    t = s["tlog"] / s["tau"]
    lse = _lse(x)
    logq = x.gather(1, ids) - lse[:, None]
    logp = t - (_lse(t) if s["t_lse"] is None else s["t_lse"])[:, None]
    p = torch.exp(logp)
    kl = (p * (logp - logq)).sum(dim=1)
    lp = x - lse[:, None]
    dz = torch.exp(lp)
    if s["t_lse"] is not None:
        lse_rest = _lse(x.scatter(1, ids, -math.inf))
        p_rest = (1.0 - p.sum(dim=1)).clamp(min=0.0)
        log_q = lse_rest - lse
        kl = kl + torch.where(p_rest > 0, p_rest * (torch.log(p_rest) - log_q), torch.zeros_like(kl))
        scale = torch.exp(log_q) - p_rest
        dz = torch.exp(x - lse_rest[:, None]) * scale[:, None]
    dz.scatter_(1, ids, torch.exp(logq) - p)
    n = s["z"].shape[0] if mask is None else mask.sum().clamp(min=1)
    loss = _rows(kl, mask).sum() / n
    dz = _rows(dz * (s["grad"] / (n * s["tau"])), mask)
    return dict(loss=loss, kl=kl if mask is None else _rows(kl, mask), grad=dz.to(s["z"].dtype))


def _plain_fused(s):
    x = (s["H"].float() @ s["W"].float().T) / s["tau"]
    lse, ent = _lse_entropy(x)
    logp = x.gather(1, s["tokens"].long()[:, None])[:, 0] - lse
    return dict(logp=_rows(logp, s["mask"]), entropy=_rows(ent, s["mask"]))


def _plain_fused_train(s):
    H, W = s["H"].float(), s["W"].float()
    x = (H @ W.T) / s["tau"]
    lse, ent = _lse_entropy(x)
    at = s["tokens"].long()[:, None]
    lp = x - lse[:, None]
    p = torch.exp(lp)
    logp = lp.gather(1, at)[:, 0]
    dz = -p * (s["g_logp"][:, None] + s["g_ent"][:, None] * (lp + ent[:, None]))
    dz.scatter_add_(1, at, s["g_logp"][:, None])
    dz = _rows(dz / s["tau"], s["mask"])
    return dict(logp=_rows(logp, s["mask"]), entropy=_rows(ent, s["mask"]),
                grad_H=(dz @ W).to(torch.bfloat16), grad_W=(dz.T @ H).to(torch.bfloat16))


_plain = dict(score=_plain_score, score_grad=_plain_score_grad, kl_step=_plain_kl, kl_grads=_plain_kl,
              fused=_plain_fused, fused_train=_plain_fused_train)


# ---- the package's operators, as a user calls them

def _package_score(s):
    import sparse_teacher_kl_gb300 as kd
    r = kd.token_logprobs_forward(s["z"], s["tokens"], s["mask"], tau=s["tau"], top=s["top"], entropy=True)
    return _keep(logp=r.logp, entropy=r.entropy, top_ids=r.top_ids, top_logp=r.top_logp)


def _package_score_grad(s):
    import sparse_teacher_kl_gb300 as kd
    return dict(grad=kd.token_logprobs_backward(s["z"], s["tokens"], s["lse"], s["g_logp"], s["mask"], tau=s["tau"],
                                                entropy=s["entropy"], grad_entropy=s["g_ent"]))


def _package_kl_step(s):
    import sparse_teacher_kl_gb300 as kd
    kl = torch.empty((s["z"].shape[0],), dtype=F32, device=s["z"].device)
    loss, grad = kd.logits_kl_step(s["z"], s["ids"], s["tlog"], s["mask"], tau=s["tau"], t_lse=s["t_lse"],
                                   grad_loss=s["grad"], kl_out=kl)
    return dict(loss=loss[0], kl=kl, grad=grad)


def _package_kl_grads(s):
    import sparse_teacher_kl_gb300 as kd
    kl = torch.empty((s["z"].shape[0],), dtype=F32, device=s["z"].device)
    loss, stats, ws = kd.logits_kl_forward(s["z"], s["ids"], s["tlog"], s["mask"], tau=s["tau"], t_lse=s["t_lse"],
                                           kl_out=kl)
    grad = kd.logits_kl_backward(s["z"], s["ids"], s["tlog"], s["mask"], stats, s["grad"], tau=s["tau"],
                                 t_lse=s["t_lse"], ws=ws)
    return dict(loss=loss[0], kl=kl, grad=grad)


def _package_fused(s):
    import sparse_teacher_kl_gb300 as kd
    logp, _, ent, _ = kd.fused_logprobs_forward(s["H"], s["W"], s["tokens"], s["mask"], chunk=CHUNK, tau=s["tau"],
                                                entropy=True)
    return dict(logp=logp, entropy=ent)


def _package_fused_train(s):
    import sparse_teacher_kl_gb300 as kd
    H, W = s["H"].detach().requires_grad_(True), s["W"].detach().requires_grad_(True)
    logp, ent = kd.fused_logprobs(H, W, s["tokens"], s["mask"], chunk=CHUNK, tau=s["tau"])
    gH, gW = torch.autograd.grad((logp, ent), (H, W), (s["g_logp"], s["g_ent"]))
    return dict(logp=logp, entropy=ent, grad_H=gH, grad_W=gW)


_package = dict(score=_package_score, score_grad=_package_score_grad, kl_step=_package_kl_step,
                kl_grads=_package_kl_grads, fused=_package_fused, fused_train=_package_fused_train)


# ------------------------------------------------------------------------- the work of one pass

def work(case):
    """Each input read once (padding rows' logits are not needed), each output written once."""
    op, N, V = case["op"], case["N"], case["V"]
    rows = N * case["valid"]
    if op in ("fused", "fused_train"):
        d = case["d"]
        train = op == "fused_train"
        return dict(bytes=2.0 * (rows + V) * d * (2 if train else 1) + N * (20.0 if train else 12.0),
                    flops=2.0 * rows * d * V * (3 if train else 1))
    size = 4 if case["type"] == "fp32" else 2
    if op == "score":
        return dict(bytes=rows * V * size + N * (8.0 * case["M"] + 4 + 8.0 * case["top"]), flops=6.0 * rows * V)
    if op == "score_grad":
        return dict(bytes=(rows + N) * V * size + N * (8.0 * case["M"] + 12), flops=6.0 * rows * V)
    return dict(bytes=(rows + N) * V * size + N * (8.0 * case["K"] + 4 + (4 if case["tail"] else 0)),
                flops=8.0 * rows * V)


# ------------------------------------------------------------------------- values in 64 bits

def exact(case, seed):
    """The definitions in float64, written out row block by row block from the inputs alone."""
    s = prepare(case, seed)
    return _exact_fused(s) if case["op"] in ("fused", "fused_train") else _exact_dense(case, s)


def _blocks(N, V):
    step = max(1, int(1e8 // V))
    return [(a, min(N, a + step)) for a in range(0, N, step)]


def _log_softmax64(x):
    m = x.max(dim=1, keepdim=True).values
    shifted = x - m
    return shifted - shifted.exp().sum(dim=1, keepdim=True).log()


def _entropy64(lp):
    p = lp.exp()
    return -(p * lp.clamp(min=-1e300)).sum(dim=1), p


def _exact_dense(case, s):
    op, N, V, tau = case["op"], case["N"], case["V"], float(s["tau"])
    on = torch.ones(N, dtype=torch.float64, device="cuda") if s["mask"] is None else s["mask"].double()
    parts = []
    for a, b in _blocks(N, V):
        keep, live = on[a:b], on[a:b] > 0
        x = s["z"][a:b].double() / tau
        lp = _log_softmax64(x)
        if op in ("score", "score_grad"):
            at = s["tokens"][a:b].long()
            ent, p = _entropy64(lp)
        if op == "score":
            part = dict(logp=torch.where(live[:, None], lp.gather(1, at), 0.0), entropy=ent * keep)
            if case["top"]:
                order = torch.sort(s["z"][a:b], dim=1, descending=True, stable=True)[1][:, :case["top"]]
                part["top_ids"] = torch.where(live[:, None], order, 0).to(torch.int32)
                part["top_logp"] = torch.where(live[:, None], lp.gather(1, order), 0.0)
        elif op == "score_grad":
            g, h = s["g_logp"][a:b].double(), s["g_ent"][a:b].double()[:, None]
            d = -p * (g.sum(dim=1, keepdim=True) + h * (lp.clamp(min=-1e300) + ent[:, None]))
            d.scatter_add_(1, at, g)
            part = dict(grad=d * keep[:, None] / tau)
        else:
            ids = s["ids"][a:b].long()
            t = s["tlog"][a:b].double() / tau
            logq = lp.gather(1, ids)
            q = lp.exp()
            if s["t_lse"] is None:
                logt = _log_softmax64(t)
                pt = logt.exp()
                kl = (pt * (logt - logq)).sum(dim=1)
                d = q
                d.scatter_add_(1, ids, -pt)
            else:
                logt = t - s["t_lse"][a:b].double()[:, None]
                pt = logt.exp()
                p_rest = (1.0 - pt.sum(dim=1)).clamp(min=0.0)
                outside = q.scatter(1, ids, 0.0)
                q_rest = outside.sum(dim=1)
                kl = (pt * (logt - logq)).sum(dim=1) + p_rest * (p_rest / q_rest).log()
                d = outside * (1.0 - p_rest / q_rest)[:, None]
                d.scatter_(1, ids, logq.exp() - pt)
            part = dict(kl=kl * keep, grad=d * keep[:, None])
        parts.append(part)
    out = {k: torch.cat([q[k] for q in parts]) for k in parts[0]}
    if op in ("kl_step", "kl_grads"):
        n = on.sum().clamp(min=1.0)
        out["loss"] = out["kl"].sum() / n
        out["grad"] *= float(s["grad"]) / (float(n) * tau)
    return out


def _exact_fused(s):
    H, W, tau = s["H"].double(), s["W"].double(), float(s["tau"])
    N = H.shape[0]
    on = torch.ones(N, dtype=torch.float64, device="cuda") if s["mask"] is None else s["mask"].double()
    train = "g_logp" in s
    logp, ent, gH = [], [], []
    gW = torch.zeros_like(W) if train else None
    for a, b in _blocks(N, W.shape[0]):
        lp = _log_softmax64(H[a:b] @ W.T / tau)
        h, p = _entropy64(lp)
        at = s["tokens"][a:b].long()[:, None]
        logp.append(lp.gather(1, at)[:, 0] * on[a:b])
        ent.append(h * on[a:b])
        if train:
            g, e = s["g_logp"][a:b].double()[:, None], s["g_ent"][a:b].double()[:, None]
            d = -p * (g + e * (lp + h[:, None]))
            d.scatter_add_(1, at, g)
            d *= on[a:b, None] / tau
            gH.append(d @ W)
            gW += d.T @ H[a:b]
    out = dict(logp=torch.cat(logp), entropy=torch.cat(ent))
    if train:
        out.update(grad_H=torch.cat(gH), grad_W=gW)
    return out
