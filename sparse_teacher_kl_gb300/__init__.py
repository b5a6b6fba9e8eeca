"""Fused chunked KL distillation against an offline top-K teacher cache, on GB300.

PyTorch supplies device memory and the current stream; every step of the path
runs in the CUDA kernels of ``libkdkl.so`` (see ``include/kdkl.h``).

    from sparse_teacher_kl_gb300 import topk_cache, fused_kl
    ids, vals = topk_cache(teacher_logits_bf16, K=100)          # offline cache
    loss = fused_kl(H, W, ids, vals, mask, chunk=4096)          # drop-in KL term
    loss.backward()                                             # recompute per chunk
"""
from __future__ import annotations

import ctypes
import functools
import threading
from typing import NamedTuple, Optional

import torch

from . import _abi
from ._abi import KDError, KD_MAX_K, KD_MAX_TOP

__all__ = [
    "topk_cache",
    "teacher_topk",
    "fused_kl",
    "fused_kl_forward",
    "fused_kl_backward",
    "chunked_kl_forward",
    "chunked_kl_backward",
    "TokenLogprobs",
    "token_logprobs",
    "token_logprobs_forward",
    "token_logprobs_backward",
    "logits_kl",
    "logits_kl_forward",
    "logits_kl_backward",
    "logits_kl_step",
    "fused_logprobs",
    "fused_logprobs_forward",
    "fused_logprobs_backward",
    "fused_cross_entropy",
    "fused_cross_entropy_forward",
    "fused_cross_entropy_step",
    "gemm_bf16",
    "quantize_int8",
    "gemm_int8",
    "teacher_topk_int8",
    "cache_write",
    "cache_info",
    "cache_read",
    "CacheReader",
    "device_error",
    "Profile",
    "KDError",
    "KD_MAX_K",
    "KD_MAX_TOP",
    "workspace",
    "control_block",
]


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(device) -> int:
    # the raw handle of the current stream, without a Stream object around it (2 us less per call)
    return torch._C._cuda_getCurrentRawStream(device.index)


def _on_its_device(f):
    """f with its first tensor's device made the current one, where it is another."""
    @functools.wraps(f)
    def call(*args, **kw):
        t = args[0] if args else next((v for v in kw.values() if isinstance(v, torch.Tensor)), None)
        if t is None or not t.is_cuda or torch.cuda.current_device() == t.device.index:
            return f(*args, **kw)
        with torch.cuda.device(t.device):
            return f(*args, **kw)
    return call


def workspace(nbytes: int, device) -> torch.Tensor:
    """A 256-byte aligned uint8 device buffer of at least ``nbytes`` (zeroed control block)."""
    buf = torch.zeros(int(nbytes) + 256, dtype=torch.uint8, device=device)
    off = (-buf.data_ptr()) % 256
    return buf[off:off + int(nbytes)]


def _require_cuda(*ts):
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("all tensors must be CUDA tensors")
        if t is not None and not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")


def topk_cache(logits: torch.Tensor, K: int, ws: Optional[torch.Tensor] = None, with_lse: bool = False,
               with_dropped: bool = False):
    """Top-K teacher cache of a dense bf16 [N, V] logits tensor: (ids int32 [N, K], vals fp32 [N, K]), then,
    when asked, the full-row logsumexp [N] (``with_lse``) and the teacher probability outside the K kept
    logits [N] (``with_dropped``), both computed by the kernel in the same pass."""
    _require_cuda(logits)
    if logits.dtype != torch.bfloat16 or logits.dim() != 2:
        raise ValueError("logits must be a 2-D bf16 tensor")
    N, V = logits.shape
    dev = logits.device
    ids = torch.empty((N, K), dtype=torch.int32, device=dev)
    vals = torch.empty((N, K), dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(_abi.kd_topk_cache_workspace(N, V, K), dev)
    lse = torch.empty((N,), dtype=torch.float32, device=dev) if with_lse else None
    dropped = torch.empty((N,), dtype=torch.float32, device=dev) if with_dropped else None
    st = _abi.kd_topk_cache(_ptr(logits), N, V, logits.stride(0), K, _ptr(ids), _ptr(vals), _ptr(lse), _ptr(dropped),
                            _ptr(ws), ws.numel(), _stream(dev))
    _abi.check(st, "kd_topk_cache")
    return (ids, vals) + ((lse,) if with_lse else ()) + ((dropped,) if with_dropped else ())


def teacher_topk(Ht: torch.Tensor, Wt: torch.Tensor, K: int, chunk: int = 1024, with_lse: bool = False,
                 with_dropped: bool = False, ws: Optional[torch.Tensor] = None):
    """Top-K cache straight from teacher hidden states Ht [N, dt] and LM-head Wt [V, dt] (bf16): the
    teacher logits exist only one chunk at a time (see kd_teacher_topk).  Returns as topk_cache."""
    _require_cuda(Ht, Wt)
    N, dt = Ht.shape
    V = Wt.shape[0]
    dev = Ht.device
    ids = torch.empty((N, K), dtype=torch.int32, device=dev)
    vals = torch.empty((N, K), dtype=torch.float32, device=dev)
    lse = torch.empty((N,), dtype=torch.float32, device=dev) if with_lse else None
    dropped = torch.empty((N,), dtype=torch.float32, device=dev) if with_dropped else None
    if ws is None:
        ws = workspace(_abi.kd_teacher_topk_workspace(N, dt, V, K, chunk), dev)
    st = _abi.kd_teacher_topk(_ptr(Ht), _ptr(Wt), N, dt, V, K, chunk, _ptr(ids), _ptr(vals), _ptr(lse), _ptr(dropped),
                              _ptr(ws), ws.numel(), _stream(dev))
    _abi.check(st, "kd_teacher_topk")
    return (ids, vals) + ((lse,) if with_lse else ()) + ((dropped,) if with_dropped else ())


def fused_kl_forward(H, W, ids, tlog, mask=None, chunk=4096, tau=1.0, ws=None, kl_out=None):
    """kd_fused_kl_fwd: returns (loss [1] fp32, lse [N] fp32, ws)."""
    _require_cuda(H, W, ids, tlog, mask)
    N, d = H.shape
    V = W.shape[0]
    K = ids.shape[1]
    if ws is None:
        ws = workspace(_abi.kd_fused_kl_workspace(N, d, V, K, chunk), H.device)
    loss = torch.empty((1,), dtype=torch.float32, device=H.device)
    lse = torch.empty((N,), dtype=torch.float32, device=H.device)
    st = _abi.kd_fused_kl_fwd(_ptr(H), _ptr(W), _ptr(ids), _ptr(tlog), _ptr(mask), N, d, V, K, chunk, float(tau),
                              _ptr(loss), _ptr(lse), _ptr(kl_out), _ptr(ws), ws.numel(), _stream(H.device))
    _abi.check(st, "kd_fused_kl_fwd")
    return loss, lse, ws


def fused_kl_backward(H, W, ids, tlog, mask, lse, grad_loss, chunk=4096, tau=1.0, ws=None, grad_H=None,
                      grad_W=None, grad_H_fp32=False):
    """kd_fused_kl_bwd: returns (grad_H [N, d] bf16 or fp32, grad_W [V, d] fp32 accumulated)."""
    _require_cuda(H, W, ids, tlog, mask, lse, grad_loss)
    N, d = H.shape
    V = W.shape[0]
    K = ids.shape[1]
    if ws is None:
        ws = workspace(_abi.kd_fused_kl_workspace(N, d, V, K, chunk), H.device)
    if grad_H is None:
        grad_H = torch.empty((N, d), dtype=torch.float32 if grad_H_fp32 else torch.bfloat16, device=H.device)
    if grad_W is None:
        grad_W = torch.zeros((V, d), dtype=torch.float32, device=H.device)
    st = _abi.kd_fused_kl_bwd(_ptr(H), _ptr(W), _ptr(ids), _ptr(tlog), _ptr(mask), N, d, V, K, chunk, float(tau),
                              _ptr(lse), _ptr(grad_loss), _ptr(grad_H), 1 if grad_H.dtype == torch.float32 else 0,
                              _ptr(grad_W), _ptr(ws), ws.numel(), _stream(H.device))
    _abi.check(st, "kd_fused_kl_bwd")
    return grad_H, grad_W


def chunked_kl_forward(H, W, ids, tlog, mask=None, chunk=4096, tau=1.0, ws=None, kl_out=None, z_store=None):
    """kd_chunked_kl_fwd (forward-chunked mode): returns (loss, lse, ws, z_store); z_store keeps the logits."""
    _require_cuda(H, W, ids, tlog, mask)
    N, d = H.shape
    V = W.shape[0]
    K = ids.shape[1]
    if ws is None:
        ws = workspace(_abi.kd_fused_kl_workspace(N, d, V, K, chunk), H.device)
    zb = _abi.kd_chunked_kl_logits_bytes(N, V)
    if z_store is None:
        z_store = torch.empty((zb,), dtype=torch.uint8, device=H.device)
    loss = torch.empty((1,), dtype=torch.float32, device=H.device)
    lse = torch.empty((N,), dtype=torch.float32, device=H.device)
    st = _abi.kd_chunked_kl_fwd(_ptr(H), _ptr(W), _ptr(ids), _ptr(tlog), _ptr(mask), N, d, V, K, chunk, float(tau),
                                _ptr(loss), _ptr(lse), _ptr(kl_out), _ptr(z_store), z_store.numel(), _ptr(ws),
                                ws.numel(), _stream(H.device))
    _abi.check(st, "kd_chunked_kl_fwd")
    return loss, lse, ws, z_store


def chunked_kl_backward(H, W, ids, tlog, mask, lse, grad_loss, z_store, chunk=4096, tau=1.0, ws=None, grad_H=None,
                        grad_W=None, grad_H_fp32=False):
    """kd_chunked_kl_bwd: gradients from the logits kept by chunked_kl_forward (no recompute)."""
    _require_cuda(H, W, ids, tlog, mask, lse, grad_loss, z_store)
    N, d = H.shape
    V = W.shape[0]
    K = ids.shape[1]
    if ws is None:
        ws = workspace(_abi.kd_fused_kl_workspace(N, d, V, K, chunk), H.device)
    if grad_H is None:
        grad_H = torch.empty((N, d), dtype=torch.float32 if grad_H_fp32 else torch.bfloat16, device=H.device)
    if grad_W is None:
        grad_W = torch.zeros((V, d), dtype=torch.float32, device=H.device)
    st = _abi.kd_chunked_kl_bwd(_ptr(H), _ptr(W), _ptr(ids), _ptr(tlog), _ptr(mask), N, d, V, K, chunk, float(tau),
                                _ptr(lse), _ptr(grad_loss), _ptr(z_store), z_store.numel(), _ptr(grad_H),
                                1 if grad_H.dtype == torch.float32 else 0, _ptr(grad_W), _ptr(ws), ws.numel(),
                                _stream(H.device))
    _abi.check(st, "kd_chunked_kl_bwd")
    return grad_H, grad_W


class _FusedKL(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, ids, tlog, mask, chunk, tau):
        loss, lse, ws = fused_kl_forward(H, W, ids, tlog, mask, chunk, tau)
        ctx.save_for_backward(H, W, ids, tlog, lse)
        ctx.mask = mask
        ctx.chunk, ctx.tau, ctx.ws = chunk, tau, ws
        return loss[0]

    @staticmethod
    def backward(ctx, grad_out):
        H, W, ids, tlog, lse = ctx.saved_tensors
        g = grad_out.reshape(1).to(torch.float32).contiguous()
        grad_H, grad_W = fused_kl_backward(H, W, ids, tlog, ctx.mask, lse, g, ctx.chunk, ctx.tau, ws=ctx.ws)
        return grad_H.to(H.dtype), grad_W.to(W.dtype), None, None, None, None, None


def fused_kl(H, W, ids, tlog, mask=None, chunk=4096, tau=1.0):
    """Differentiable fused chunked KL(p_teacher || q_student) token mean (scalar tensor)."""
    return _FusedKL.apply(H, W, ids, tlog, mask, int(chunk), float(tau))


# ------------------------------------------------------------- dense logits

_DTYPES = {torch.bfloat16: _abi.KD_BF16, torch.float16: _abi.KD_F16, torch.float32: _abi.KD_F32}


def _check(t: Optional[torch.Tensor], name: str, dtype, shape, device):
    """A contiguous tensor of this type and shape on this device (or None)."""
    if t is None:
        return
    if t.device != device or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")


def _check_logits(z: torch.Tensor, name: str = "logits"):
    """(type code, N, V, row stride) of a 2-D CUDA matrix whose rows are contiguous."""
    if not z.is_cuda or z.dim() != 2 or z.dtype not in _DTYPES:
        raise ValueError(f"{name} must be a 2-D bf16, fp16 or fp32 CUDA tensor")
    N, V = z.shape
    if N < 1 or V < 1:
        raise ValueError(f"{name} must not be empty")
    ld = z.stride(0) if N > 1 else V
    if (z.stride(1) != 1 and V > 1) or ld < V:
        raise ValueError(f"the rows of {name} must be contiguous and must not overlap")
    return _DTYPES[z.dtype], N, V, ld


def _grad_like(z: torch.Tensor, grad: Optional[torch.Tensor]):
    """(gradient matrix, its row stride): a new one, or the caller's (the logits themselves included)."""
    if grad is None:
        grad = torch.empty(z.shape, dtype=z.dtype, device=z.device)
        return grad, z.shape[1]
    if grad.shape != z.shape or grad.dtype != z.dtype or grad.device != z.device:
        raise ValueError("grad_logits must have the logits' shape, type and device")
    return grad, _check_logits(grad, "grad_logits")[3]


def _written(*ts):
    """Tells autograd that a kernel wrote to these tensors of the caller's: where one of them was saved for a backward
    pass, that pass raises in place of reading what took its values' place."""
    for t in ts:
        if t is not None and not t.is_inference():
            torch.autograd.graph.increment_version(t)


def _fresh_ws(nbytes: int, device) -> torch.Tensor:
    """A workspace with its control block zeroed and the rest left as it is (the allocator's blocks are aligned)."""
    ws = _scratch(nbytes, device)
    _abi.check(_abi.kd_workspace_clear(ws.data_ptr(), ws.numel(), _stream(device)), "kd_workspace_clear")
    return ws


def _scratch(nbytes: int, device) -> torch.Tensor:
    """A workspace of any content, for calls that report to a control block of its own."""
    return torch.empty((int(nbytes),), dtype=torch.uint8, device=device)


class _Blocks(threading.local):
    """A thread's control blocks, by device index and stream."""

    def __init__(self):
        self.by_stream = {}


_blocks = _Blocks()
_captured = {}  # device index -> the control block of calls captured into graphs


def _cleared(device: torch.device) -> torch.Tensor:
    ws = _fresh_ws(256, device)
    torch.cuda.current_stream(device).synchronize()  # cleared before another stream uses it
    return ws


def _control(device: torch.device) -> torch.Tensor:
    """The control block of a call without a workspace, on the current stream."""
    if torch.cuda.is_current_stream_capturing():
        ws = _captured.get(device.index)
        # memory of a capture belongs to its graph: without an earlier call outside, nobody can read it
        return _fresh_ws(256, device) if ws is None else ws
    key = (device.index, _stream(device))
    ws = _blocks.by_stream.get(key)
    if ws is None:
        ws = _blocks.by_stream[key] = _cleared(device)
        if device.index not in _captured:
            _captured.setdefault(device.index, _cleared(device))
    return ws


def control_block(device=None, captured: bool = False) -> torch.Tensor:
    """The control block that calls on dense logits, and the differentiable calls, report to when they are given no
    workspace: its only content is the error word, which ``device_error(control_block(device))`` reads and clears.
    Each thread has one for every device and stream (this is the current stream's; a backward pass reports to the
    block of its forward pass).  With ``captured``, the one that calls captured into graphs on the device share,
    where a call outside a capture (a warm-up) came first."""
    device = torch.device("cuda" if device is None else device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    block = _control(device)
    return _captured[device.index] if captured else block


class TokenLogprobs(NamedTuple):
    """What token_logprobs_forward returns (None for what was not asked for)."""
    logp: torch.Tensor                      # [N, M] (or [N]) log probabilities of the given tokens
    lse: torch.Tensor                       # [N] logsumexp of logits / tau
    entropy: Optional[torch.Tensor]         # [N]
    top_ids: Optional[torch.Tensor]         # [N, top] int32, most probable first
    top_logp: Optional[torch.Tensor]        # [N, top]


def token_logprobs_forward(logits, tokens, mask=None, tau=1.0, top=0, entropy=False, ws=None) -> TokenLogprobs:
    """kd_token_logprobs_fwd: log probabilities of ``tokens`` (int32 [N] or [N, M]) under softmax(logits / tau),
    with the ``top`` most probable alternatives and the entropy when asked.  ``logits``: [N, V] bf16, fp16 or
    fp32 with contiguous rows (any row stride)."""
    dt, N, V, ld = _check_logits(logits)
    dev = logits.device
    M = tokens.shape[1] if tokens.dim() == 2 else 1
    _check(tokens, "tokens", torch.int32, (N, M) if tokens.dim() == 2 else (N,), dev)
    _check(mask, "mask", torch.uint8, (N,), dev)
    f32 = dict(dtype=torch.float32, device=dev)
    logp = torch.empty(tokens.shape, **f32)
    lse = torch.empty((N,), **f32)
    ent = torch.empty((N,), **f32) if entropy else None
    top_ids = torch.empty((N, top), dtype=torch.int32, device=dev) if top else None
    top_logp = torch.empty((N, top), **f32) if top else None
    if ws is None:
        ws = _control(dev)
    st = _abi.kd_token_logprobs_fwd(_ptr(logits), dt, N, V, ld, _ptr(tokens), M, _ptr(mask), float(tau), int(top),
                                    _ptr(logp), _ptr(lse), _ptr(ent), _ptr(top_ids), _ptr(top_logp), _ptr(ws),
                                    ws.numel(), _stream(dev))
    _abi.check(st, "kd_token_logprobs_fwd")
    return TokenLogprobs(logp, lse, ent, top_ids, top_logp)


def token_logprobs_backward(logits, tokens, lse, grad_logp, mask=None, tau=1.0, entropy=None, grad_entropy=None,
                            ws=None, grad_logits=None):
    """kd_token_logprobs_bwd: the gradient of the logits, in their type.  ``grad_logits`` may be the logits
    themselves (their memory is then reused)."""
    dt, N, V, ld = _check_logits(logits)
    dev = logits.device
    M = tokens.shape[1] if tokens.dim() == 2 else 1
    _check(tokens, "tokens", torch.int32, (N, M) if tokens.dim() == 2 else (N,), dev)
    _check(grad_logp, "grad_logp", torch.float32, tokens.shape, dev)
    for t, name in ((lse, "lse"), (entropy, "entropy"), (grad_entropy, "grad_entropy")):
        _check(t, name, torch.float32, (N,), dev)
    _check(mask, "mask", torch.uint8, (N,), dev)
    given = grad_logits
    grad_logits, ldg = _grad_like(logits, grad_logits)
    if ws is None:
        ws = _control(dev)
    st = _abi.kd_token_logprobs_bwd(_ptr(logits), dt, N, V, ld, _ptr(tokens), M, _ptr(mask), float(tau), _ptr(lse),
                                    _ptr(entropy), _ptr(grad_logp), _ptr(grad_entropy), _ptr(grad_logits), ldg,
                                    _ptr(ws), ws.numel(), _stream(dev))
    _abi.check(st, "kd_token_logprobs_bwd")
    _written(given)
    return grad_logits


def _f32c(g):
    return None if g is None else g.to(torch.float32).contiguous()


class _NoSecondDerivative(torch.autograd.Function):
    @staticmethod
    def forward(ctx, g):
        return g.view_as(g)

    @staticmethod
    def backward(ctx, g):
        raise RuntimeError("trying to differentiate twice a function that is once_differentiable")


def _once_differentiable(backward):
    """A backward pass whose gradients, under create_graph, raise when they are differentiated in turn, by the inputs
    as by the incoming gradients (torch's own decorator sees the latter alone)."""
    @functools.wraps(backward)
    def run(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        return tuple(None if g is None else _NoSecondDerivative.apply(g.detach().requires_grad_()) for g in out)
    return run


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, mask, tau):
        _check_logits(logits)
        ctx.control = _control(logits.device)
        r = token_logprobs_forward(logits, tokens, mask, tau, entropy=True, ws=ctx.control)
        ctx.save_for_backward(logits, tokens, mask, r.lse, r.entropy)
        ctx.tau = tau
        ctx.set_materialize_grads(False)
        return r.logp, r.entropy

    @staticmethod
    @_once_differentiable
    def backward(ctx, g_logp, g_entropy):
        logits, tokens, mask, lse, ent = ctx.saved_tensors
        if g_logp is None and g_entropy is None:
            return None, None, None, None
        if g_logp is None:
            g_logp = torch.zeros(tokens.shape, dtype=torch.float32, device=logits.device)
        g = token_logprobs_backward(logits, tokens, lse, _f32c(g_logp), mask, ctx.tau, ent, _f32c(g_entropy),
                                    ws=ctx.control)
        return g, None, None, None


def token_logprobs(logits, tokens, mask=None, tau=1.0):
    """Differentiable (log probabilities of ``tokens``, entropy [N]) of softmax(logits / tau)."""
    return _TokenLogprobs.apply(logits, tokens, mask, float(tau))


def _check_kl(logits, ids, tlog, mask, t_lse, kl_out=None):
    dt, N, V, ld = _check_logits(logits)
    dev = logits.device
    if ids.dim() != 2:
        raise ValueError("ids must be an int32 [N, K] tensor")
    K = ids.shape[1]
    _check(ids, "ids", torch.int32, (N, K), dev)
    _check(tlog, "tlog", torch.float32, (N, K), dev)
    _check(t_lse, "t_lse", torch.float32, (N,), dev)
    _check(mask, "mask", torch.uint8, (N,), dev)
    _check(kl_out, "kl_out", torch.float32, (N,), dev)
    return dt, N, V, ld, K, dev


def _kl_forward(logits, ids, tlog, mask, tau, t_lse, ws, control, kl_out=None):
    dt, N, V, ld, K, dev = _check_kl(logits, ids, tlog, mask, t_lse, kl_out)
    if ws is None:
        ws = (_fresh_ws if control is None else _scratch)(_abi.kd_logits_kl_workspace(N, V, K), dev)
    if control is None:
        control = ws
    loss = torch.empty((1,), dtype=torch.float32, device=dev)
    stats = torch.empty((N, 4), dtype=torch.float32, device=dev)
    st = _abi.kd_logits_kl_fwd_ctl(_ptr(logits), dt, N, V, ld, _ptr(ids), _ptr(tlog), K, _ptr(t_lse), _ptr(mask),
                                   float(tau), _ptr(loss), _ptr(stats), _ptr(kl_out), _ptr(ws), ws.numel(),
                                   _ptr(control), _stream(dev))
    _abi.check(st, "kd_logits_kl_fwd")
    _written(kl_out)
    return loss, stats, ws


def logits_kl_forward(logits, ids, tlog, mask=None, tau=1.0, t_lse=None, ws=None, kl_out=None):
    """kd_logits_kl_fwd: KL of the cached teacher (``ids`` int32, ``tlog`` fp32 [N, K]; with ``t_lse`` its mass
    outside the cache as one more class) against softmax(logits / tau): (loss [1], stats [N, 4], ws)."""
    return _kl_forward(logits, ids, tlog, mask, tau, t_lse, ws, None, kl_out)


def _kl_backward(logits, ids, tlog, mask, stats, grad_loss, tau, t_lse, ws, control, grad_logits=None):
    dt, N, V, ld, K, dev = _check_kl(logits, ids, tlog, mask, t_lse)
    _check(stats, "stats", torch.float32, (N, 4), dev)
    _check(grad_loss, "grad_loss", torch.float32, (1,), dev)
    given = grad_logits
    grad_logits, ldg = _grad_like(logits, grad_logits)
    if control is None:
        control = _control(dev) if ws is None else ws
    if ws is None:
        ws = _scratch(_abi.kd_logits_kl_workspace(N, V, K), dev)
    st = _abi.kd_logits_kl_bwd_ctl(_ptr(logits), dt, N, V, ld, _ptr(ids), _ptr(tlog), K, _ptr(t_lse), _ptr(mask),
                                   float(tau), _ptr(stats), _ptr(grad_loss), _ptr(grad_logits), ldg, _ptr(ws),
                                   ws.numel(), _ptr(control), _stream(dev))
    _abi.check(st, "kd_logits_kl_bwd")
    _written(given)
    return grad_logits


def logits_kl_backward(logits, ids, tlog, mask, stats, grad_loss, tau=1.0, t_lse=None, ws=None, grad_logits=None):
    """kd_logits_kl_bwd: the gradient of the logits, in their type (``grad_logits`` may be the logits themselves).
    Without a workspace errors go to the stream's control_block."""
    return _kl_backward(logits, ids, tlog, mask, stats, grad_loss, tau, t_lse, ws, None, grad_logits)


def logits_kl_step(logits, ids, tlog, mask=None, tau=1.0, t_lse=None, grad_loss=None, ws=None, kl_out=None,
                   grad_logits=None):
    """kd_logits_kl_step: loss and gradient in one pass over the logits, for a ``grad_loss`` ([1] fp32, default 1)
    known beforehand: (loss [1], grad_logits).  ``grad_logits`` may be the logits themselves.  Without a workspace
    errors go to the stream's control_block."""
    dt, N, V, ld, K, dev = _check_kl(logits, ids, tlog, mask, t_lse, kl_out)
    if grad_loss is None:
        grad_loss = torch.ones((1,), dtype=torch.float32, device=dev)
    _check(grad_loss, "grad_loss", torch.float32, (1,), dev)
    given = grad_logits
    grad_logits, ldg = _grad_like(logits, grad_logits)
    control = ws
    if ws is None:
        control = _control(dev)
        ws = _scratch(_abi.kd_logits_kl_workspace(N, V, K), dev)
    loss = torch.empty((1,), dtype=torch.float32, device=dev)
    st = _abi.kd_logits_kl_step_ctl(_ptr(logits), dt, N, V, ld, _ptr(ids), _ptr(tlog), K, _ptr(t_lse), _ptr(mask),
                                    float(tau), _ptr(grad_loss), _ptr(loss), _ptr(kl_out), _ptr(grad_logits), ldg,
                                    _ptr(ws), ws.numel(), _ptr(control), _stream(dev))
    _abi.check(st, "kd_logits_kl_step")
    _written(given, kl_out)
    return loss, grad_logits


class _LogitsKL(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, tlog, mask, tau, t_lse):
        _check_logits(logits)
        ctx.control = _control(logits.device)
        loss, stats, ws = _kl_forward(logits, ids, tlog, mask, tau, t_lse, None, ctx.control)
        ctx.save_for_backward(logits, ids, tlog, mask, t_lse, stats)
        ctx.tau, ctx.ws = tau, ws
        return loss[0]

    @staticmethod
    @_once_differentiable
    def backward(ctx, grad_out):
        logits, ids, tlog, mask, t_lse, stats = ctx.saved_tensors
        g = _kl_backward(logits, ids, tlog, mask, stats, _f32c(grad_out.reshape(1)), ctx.tau, t_lse, ctx.ws,
                         ctx.control)
        return g, None, None, None, None, None


def logits_kl(logits, ids, tlog, mask=None, tau=1.0, t_lse=None):
    """Differentiable KL(p_teacher || q_student) token mean on dense student logits (scalar tensor)."""
    return _LogitsKL.apply(logits, ids, tlog, mask, float(tau), t_lse)


def _check_projection(H, W, tokens, mask, name="tokens"):
    for t, which in ((H, "H"), (W, "W")):
        if not t.is_cuda or t.dim() != 2 or t.dtype != torch.bfloat16 or not t.is_contiguous():
            raise ValueError(f"{which} must be a contiguous 2-D bf16 CUDA tensor")
    N, d = H.shape
    if W.shape[1] != d or W.device != H.device:
        raise ValueError("W must be [V, d] on the device of H [N, d]")
    _check(tokens, name, torch.int32, (N,), H.device)
    _check(mask, "mask", torch.uint8, (N,), H.device)
    return N, d, W.shape[0], H.device


def _fused_forward(H, W, tokens, mask, chunk, tau, entropy, ws, control):
    N, d, V, dev = _check_projection(H, W, tokens, mask)
    if ws is None:
        ws = (_fresh_ws if control is None else _scratch)(_abi.kd_fused_logprobs_workspace(N, d, V, chunk, 0), dev)
    if control is None:
        control = ws
    logp = torch.empty((N,), dtype=torch.float32, device=dev)
    lse = torch.empty((N,), dtype=torch.float32, device=dev)
    ent = torch.empty((N,), dtype=torch.float32, device=dev) if entropy else None
    st = _abi.kd_fused_logprobs_fwd_ctl(_ptr(H), _ptr(W), _ptr(tokens), _ptr(mask), N, d, V, chunk, float(tau),
                                        _ptr(logp), _ptr(lse), _ptr(ent), _ptr(ws), ws.numel(), _ptr(control),
                                        _stream(dev))
    _abi.check(st, "kd_fused_logprobs_fwd")
    return logp, lse, ent, ws


def fused_logprobs_forward(H, W, tokens, mask=None, chunk=4096, tau=1.0, entropy=False, ws=None):
    """kd_fused_logprobs_fwd: (logp [N], lse [N], entropy [N] or None, ws) of ``tokens`` (int32 [N]) under
    softmax(H W^T / tau), the logits never stored."""
    return _fused_forward(H, W, tokens, mask, chunk, tau, entropy, ws, None)


def _fused_backward(H, W, tokens, lse, grad_logp, mask, chunk, tau, entropy, grad_entropy, ws, control, grad_H=None,
                    grad_W=None, grad_H_fp32=False, grad_W_bf16=False):
    N, d, V, dev = _check_projection(H, W, tokens, mask)
    for t, name in ((lse, "lse"), (grad_logp, "grad_logp"), (entropy, "entropy"), (grad_entropy, "grad_entropy")):
        _check(t, name, torch.float32, (N,), dev)
    if control is None:
        control = _control(dev) if ws is None else ws
    if ws is None:
        ws = _scratch(_abi.kd_fused_logprobs_workspace(N, d, V, chunk, 1), dev)
    given = grad_H, grad_W
    if grad_H is None:
        grad_H = torch.empty((N, d), dtype=torch.float32 if grad_H_fp32 else torch.bfloat16, device=dev)
    kind = _abi.KD_GRAD_ADD_F32
    if grad_W is None:
        kind = _abi.KD_GRAD_STORE_BF16 if grad_W_bf16 else _abi.KD_GRAD_STORE_F32
        grad_W = torch.empty((V, d), dtype=torch.bfloat16 if grad_W_bf16 else torch.float32, device=dev)
    else:
        _check(grad_W, "grad_W", torch.float32, (V, d), dev)
    _check(grad_H, "grad_H", torch.float32 if grad_H.dtype == torch.float32 else torch.bfloat16, (N, d), dev)
    st = _abi.kd_fused_logprobs_bwd_ctl(_ptr(H), _ptr(W), _ptr(tokens), _ptr(mask), N, d, V, chunk, float(tau),
                                        _ptr(lse), _ptr(entropy), _ptr(grad_logp), _ptr(grad_entropy), _ptr(grad_H),
                                        1 if grad_H.dtype == torch.float32 else 0, _ptr(grad_W), kind, _ptr(ws),
                                        ws.numel(), _ptr(control), _stream(dev))
    _abi.check(st, "kd_fused_logprobs_bwd")
    _written(*given)
    return grad_H, grad_W


def fused_logprobs_backward(H, W, tokens, lse, grad_logp, mask=None, chunk=4096, tau=1.0, entropy=None,
                            grad_entropy=None, ws=None, grad_H=None, grad_W=None, grad_H_fp32=False, grad_W_bf16=False):
    """kd_fused_logprobs_bwd: (grad_H [N, d] bf16 or fp32, grad_W [V, d]).  A ``grad_W`` of the caller's (fp32) is
    added into; without one it is a new tensor, fp32 or with ``grad_W_bf16`` (one chunk only) bf16.  Without a
    workspace errors go to the stream's control_block."""
    return _fused_backward(H, W, tokens, lse, grad_logp, mask, chunk, tau, entropy, grad_entropy, ws, None, grad_H,
                           grad_W, grad_H_fp32, grad_W_bf16)


class _FusedLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, H, W, tokens, mask, chunk, tau):
        _check_projection(H, W, tokens, mask)
        ctx.control = _control(H.device)
        logp, lse, ent, _ = _fused_forward(H, W, tokens, mask, chunk, tau, True, None, ctx.control)
        ctx.save_for_backward(H, W, tokens, mask, lse, ent)
        ctx.chunk, ctx.tau = chunk, tau
        ctx.set_materialize_grads(False)
        return logp, ent

    @staticmethod
    @_once_differentiable
    def backward(ctx, g_logp, g_entropy):
        H, W, tokens, mask, lse, ent = ctx.saved_tensors
        if g_logp is None and g_entropy is None:
            return None, None, None, None, None, None
        if g_logp is None:
            g_logp = torch.zeros_like(lse)
        grad_H, grad_W = _fused_backward(H, W, tokens, lse, _f32c(g_logp), mask, ctx.chunk, ctx.tau, ent,
                                         _f32c(g_entropy), None, ctx.control, grad_W_bf16=H.shape[0] <= ctx.chunk)
        return grad_H, grad_W.to(W.dtype), None, None, None, None


def fused_logprobs(H, W, tokens, mask=None, chunk=4096, tau=1.0):
    """Differentiable (log probability of ``tokens`` [N], entropy [N]) of softmax(H W^T / tau)."""
    return _FusedLogprobs.apply(H, W, tokens, mask, int(chunk), float(tau))


def _ce_options(label_smoothing, z_loss, softcap, ignore_index):
    if not -2 ** 31 <= int(ignore_index) < 2 ** 31:
        raise ValueError("ignore_index must be an int32 number")
    return float(label_smoothing), float(z_loss), float(softcap), int(ignore_index)


def _ce_step(H, W, labels, mask, chunk, options, grad_loss, ws, control, loss_out=None, grad_H=None, grad_W=None,
             grad_H_fp32=False, grad_W_bf16=False):
    N, d, V, dev = _check_projection(H, W, labels, mask, "labels")
    _check(loss_out, "loss_out", torch.float32, (N,), dev)
    _check(grad_loss, "grad_loss", torch.float32, (1,), dev)
    if ws is None:
        ws = _scratch(_abi.kd_fused_cross_entropy_workspace(N, d, V, chunk, 1), dev)
    given = loss_out, grad_H, grad_W
    if grad_H is None:
        grad_H = torch.empty((N, d), dtype=torch.float32 if grad_H_fp32 else torch.bfloat16, device=dev)
    kind = _abi.KD_GRAD_ADD_F32
    if grad_W is None:
        kind = _abi.KD_GRAD_STORE_BF16 if grad_W_bf16 else _abi.KD_GRAD_STORE_F32
        grad_W = torch.empty((V, d), dtype=torch.bfloat16 if grad_W_bf16 else torch.float32, device=dev)
    else:
        _check(grad_W, "grad_W", torch.float32, (V, d), dev)
    _check(grad_H, "grad_H", torch.float32 if grad_H.dtype == torch.float32 else torch.bfloat16, (N, d), dev)
    loss = torch.empty((1,), dtype=torch.float32, device=dev)
    lse = torch.empty((N,), dtype=torch.float32, device=dev)
    st = _abi.kd_fused_cross_entropy_step(_ptr(H), _ptr(W), _ptr(labels), _ptr(mask), N, d, V, chunk, *options,
                                          _ptr(grad_loss), _ptr(loss), _ptr(lse), _ptr(loss_out), _ptr(grad_H),
                                          1 if grad_H.dtype == torch.float32 else 0, _ptr(grad_W), kind, _ptr(ws),
                                          ws.numel(), _ptr(control), _stream(dev))
    _abi.check(st, "kd_fused_cross_entropy_step")
    _written(*given)
    return loss, grad_H, grad_W


def _ce_forward(H, W, labels, mask, chunk, options, ws, control, loss_out=None):
    N, d, V, dev = _check_projection(H, W, labels, mask, "labels")
    _check(loss_out, "loss_out", torch.float32, (N,), dev)
    if ws is None:
        ws = (_fresh_ws if control is None else _scratch)(_abi.kd_fused_cross_entropy_workspace(N, d, V, chunk, 0), dev)
    if control is None:
        control = ws
    loss = torch.empty((1,), dtype=torch.float32, device=dev)
    lse = torch.empty((N,), dtype=torch.float32, device=dev)
    st = _abi.kd_fused_cross_entropy_fwd(_ptr(H), _ptr(W), _ptr(labels), _ptr(mask), N, d, V, chunk, *options,
                                         _ptr(loss), _ptr(lse), _ptr(loss_out), _ptr(ws), ws.numel(), _ptr(control),
                                         _stream(dev))
    _abi.check(st, "kd_fused_cross_entropy_fwd")
    _written(loss_out)
    return loss, lse, ws


@_on_its_device
def fused_cross_entropy_forward(H, W, labels, mask=None, chunk=4096, label_smoothing=0.0, z_loss=0.0, softcap=0.0,
                                ignore_index=-100, ws=None, loss_out=None):
    """kd_fused_cross_entropy_fwd: (loss [1], lse [N], ws).  Cross entropy of ``labels`` (int32 [N]) against
    softmax(H W^T), the logits never stored: the mean over the positions whose label is not ``ignore_index`` and
    whose ``mask`` is not 0; each position's own loss goes to ``loss_out`` ([N] fp32) when given."""
    return _ce_forward(H, W, labels, mask, chunk, _ce_options(label_smoothing, z_loss, softcap, ignore_index), ws, None,
                       loss_out)


@_on_its_device
def fused_cross_entropy_step(H, W, labels, mask=None, chunk=4096, label_smoothing=0.0, z_loss=0.0, softcap=0.0,
                             ignore_index=-100, grad_loss=None, ws=None, loss_out=None, grad_H=None, grad_W=None,
                             grad_H_fp32=False, grad_W_bf16=False):
    """kd_fused_cross_entropy_step: loss and gradients in one call, for a ``grad_loss`` ([1] fp32, default 1) known
    beforehand: (loss [1], grad_H [N, d] bf16 or fp32, grad_W [V, d]).  A ``grad_W`` of the caller's (fp32) is added
    into; without one it is a new tensor, fp32 or with ``grad_W_bf16`` (one chunk only) bf16.  Without a workspace
    errors go to the stream's control_block."""
    options = _ce_options(label_smoothing, z_loss, softcap, ignore_index)
    _check_projection(H, W, labels, mask, "labels")
    control = _control(H.device) if ws is None else ws
    return _ce_step(H, W, labels, mask, chunk, options, grad_loss, ws, control, loss_out, grad_H, grad_W, grad_H_fp32,
                    grad_W_bf16)


class _FusedCrossEntropy(torch.autograd.Function):
    """The factor that arrives joins the gradients before they are rounded to their type.  Positions of one chunk: the
    forward pass keeps the logits in 16 bits and the backward pass takes both gradients from them (one projection in
    place of two).  Of more chunks: the forward pass takes the gradients of a factor 1 in fp32, the backward pass
    multiplies and rounds them."""

    @staticmethod
    def forward(ctx, H, W, labels, mask, chunk, options, wanted):
        N, d, V, dev = _check_projection(H, W, labels, mask, "labels")
        ctx.control = _control(dev)
        ctx.chunk, ctx.options, ctx.spent = chunk, options, False
        if not wanted:
            return _ce_forward(H, W, labels, mask, chunk, options, None, ctx.control)[0][0]
        if N <= chunk:
            if chunk % 128:  # refused as by the calls that take it
                _abi.check(_abi.KD_ERR_INVALID_ARG, "kd_fused_cross_entropy_keep")
            kept = (_scratch(_abi.kd_fused_cross_entropy_kept(N, d, V), dev),)
            loss = torch.empty((1,), dtype=torch.float32, device=dev)
            lse = torch.empty((N,), dtype=torch.float32, device=dev)
            st = _abi.kd_fused_cross_entropy_keep(_ptr(H), _ptr(W), _ptr(labels), _ptr(mask), N, d, V, *options,
                                                  _ptr(loss), _ptr(lse), None, _ptr(kept[0]), kept[0].numel(),
                                                  _ptr(ctx.control), _stream(dev))
            _abi.check(st, "kd_fused_cross_entropy_keep")
        else:
            loss, *kept = _ce_step(H, W, labels, mask, chunk, options, None, None, ctx.control, grad_H_fp32=True)
        ctx.save_for_backward(H, W, labels, mask, *kept)
        return loss[0]

    @staticmethod
    @_once_differentiable
    def backward(ctx, grad_out):
        H, W, labels, mask, *kept = ctx.saved_tensors
        (N, d), V, dev = H.shape, W.shape[0], H.device
        one, g = N <= ctx.chunk, _f32c(grad_out.reshape(1))
        if ctx.spent:
            # what was kept has become the first pass's gradients: a second one takes them anew
            _, gH, gW = _ce_step(H, W, labels, mask, ctx.chunk, ctx.options, g, None, ctx.control, grad_H_fp32=not one,
                                 grad_W_bf16=one)
            return gH.to(H.dtype), gW.to(W.dtype), None, None, None, None, None
        ctx.spent = True
        if one:
            gH, gW = torch.empty_like(H), torch.empty_like(W)
            ws = _scratch(_abi.kd_fused_cross_entropy_bwd_workspace(N, d, V), dev)
            st = _abi.kd_fused_cross_entropy_bwd(_ptr(W), N, d, V, ctx.options[0], ctx.options[2], _ptr(g), _ptr(gH), 0,
                                                 _ptr(gW), _abi.KD_GRAD_STORE_BF16, _ptr(kept[0]), kept[0].numel(),
                                                 _ptr(ws), ws.numel(), _ptr(ctx.control), _stream(dev))
            _abi.check(st, "kd_fused_cross_entropy_bwd")
            return gH, gW, None, None, None, None, None
        for t in kept:
            _abi.check(_abi.kd_scale_gradient(_ptr(t), t.numel(), 1, _ptr(g), _stream(dev)), "kd_scale_gradient")
        return kept[0].to(H.dtype), kept[1].to(W.dtype), None, None, None, None, None


@_on_its_device
def fused_cross_entropy(H, W, labels, mask=None, chunk=4096, label_smoothing=0.0, z_loss=0.0, softcap=0.0,
                        ignore_index=-100):
    """Differentiable cross entropy of ``labels`` (int32 [N]) against softmax(H W^T): the mean over the positions
    whose label is not ``ignore_index`` and whose ``mask`` is not 0 (scalar tensor).  Up to ``chunk`` positions the
    graph keeps their logits in 16 bits until the backward pass (2 N V bytes); of more, the forward pass takes both
    gradients already, in fp32 (4 V d bytes), so a loss that is not differentiated belongs under ``no_grad``."""
    wanted = torch.is_grad_enabled() and (H.requires_grad or W.requires_grad)
    return _FusedCrossEntropy.apply(H, W, labels, mask, int(chunk),
                                    _ce_options(label_smoothing, z_loss, softcap, ignore_index), wanted)


def gemm_bf16(A, B, M, N, K, a_mn_major=False, b_mn_major=False, C=None):
    """The projection engine on its own: C[M, N] fp32 = A·B (see kd_gemm_bf16)."""
    _require_cuda(A, B)
    if C is None:
        C = torch.empty((M, N), dtype=torch.float32, device=A.device)
        acc = 0
    else:
        acc = 1
    ws = workspace(_abi.kd_gemm_workspace(), A.device)
    st = _abi.kd_gemm_bf16(_ptr(A), _ptr(B), _ptr(C), M, N, K, int(a_mn_major), int(b_mn_major), acc, _ptr(ws),
                           ws.numel(), _stream(A.device))
    _abi.check(st, "kd_gemm_bf16")
    return C, ws


# ------------------------------------------------------------------ 8 bits

@_on_its_device
def quantize_int8(x, q=None, scale=None):
    """kd_quantize_int8: (q int8 [N, d], scale fp32 [N]) of the rows of ``x`` ([N, d] bf16, fp16 or fp32, any row
    stride): scale = max |x| / 127, q = x / scale to the nearest whole number."""
    dt, N, d, ld = _check_logits(x, "x")
    given = q, scale
    if q is None:
        q, ldq = torch.empty((N, d), dtype=torch.int8, device=x.device), d
    else:
        ldq = _check_int8(q, "q", x.device)
        if q.shape != x.shape:
            raise ValueError("q must have the shape of x")
    if scale is None:
        scale = torch.empty((N,), dtype=torch.float32, device=x.device)
    else:
        _check(scale, "scale", torch.float32, (N,), x.device)
    st = _abi.kd_quantize_int8(_ptr(x), dt, N, d, ld, _ptr(q), ldq, _ptr(scale), _stream(x.device))
    _abi.check(st, "kd_quantize_int8")
    _written(*given)
    return q, scale


def _check_int8(t, name: str, device=None) -> int:
    """The row stride of a 2-D int8 CUDA matrix whose rows are contiguous."""
    if not t.is_cuda or t.dim() != 2 or t.dtype != torch.int8 or (device is not None and t.device != device):
        raise ValueError(f"{name} must be a 2-D int8 CUDA tensor" + ("" if device is None else f" on {device}"))
    if t.shape[0] < 1 or t.shape[1] < 1:
        raise ValueError(f"{name} must not be empty")
    ld = t.stride(0) if t.shape[0] > 1 else t.shape[1]
    if (t.stride(1) != 1 and t.shape[1] > 1) or ld < t.shape[1]:
        raise ValueError(f"the rows of {name} must be contiguous and must not overlap")
    return ld


def _rows_aligned(t, ld: int) -> int:
    return int(t.data_ptr() % 16 == 0 and ld % 16 == 0)


@_on_its_device
def gemm_int8(A, a_scale, B, b_scale, out_dtype=torch.bfloat16, out=None, ws=None):
    """kd_gemm_int8: [M, N] = (A B^T) a_scale[:, None] b_scale of int8 matrices A [M, K] (tokens) and B [N, K]
    (channels), rows of any stride, in bf16, fp16 or fp32 (``out_dtype``, or that of a given ``out``).  Weights
    B whose rows start on 16-byte boundaries are read in place.  Without a workspace errors go to the stream's
    control_block."""
    lda, ldb = _check_int8(A, "A"), _check_int8(B, "B", A.device)
    (M, K), N, dev = A.shape, B.shape[0], A.device
    if B.shape[1] != K:
        raise ValueError("A and B must have the same number of columns")
    _check(a_scale, "a_scale", torch.float32, (M,), dev)
    _check(b_scale, "b_scale", torch.float32, (N,), dev)
    given = out
    if out is None:
        if out_dtype not in _DTYPES:
            raise ValueError("out_dtype must be bf16, fp16 or fp32")
        out, dt, ldc = torch.empty((M, N), dtype=out_dtype, device=dev), _DTYPES[out_dtype], N
    else:
        if out.device != dev or out.shape != (M, N):
            raise ValueError(f"out must be [{M}, {N}] on {dev}")
        dt, _, _, ldc = _check_logits(out, "out")
    control = ws
    if ws is None:
        ws = control = _control(dev)
        need = _abi.kd_gemm_int8_workspace(M, N, K, _rows_aligned(B, ldb))
        if need > ws.numel():  # few tokens need the control block alone
            ws = _scratch(need, dev)
    st = _abi.kd_gemm_int8(_ptr(A), lda, _ptr(a_scale), _ptr(B), ldb, _ptr(b_scale), _ptr(out), dt, ldc, M, N, K,
                           _ptr(ws), ws.numel(), _ptr(control), _stream(dev))
    _abi.check(st, "kd_gemm_int8")
    _written(given)
    return out


@_on_its_device
def teacher_topk_int8(Ht, h_scale, Wt, w_scale, K: int, chunk: int = 1024, with_lse: bool = False,
                      with_dropped: bool = False, ws: Optional[torch.Tensor] = None):
    """Top-K cache from quantised teacher hidden states Ht [N, dt] and LM-head Wt [V, dt] (int8 with their rows'
    scales, see quantize_int8): the teacher logits exist only one chunk at a time, in bf16.  Returns as topk_cache."""
    ld_h, ld_w = _check_int8(Ht, "Ht"), _check_int8(Wt, "Wt", Ht.device)
    (N, dt), V, dev = Ht.shape, Wt.shape[0], Ht.device
    if Wt.shape[1] != dt:
        raise ValueError("Ht and Wt must have the same number of columns")
    _check(h_scale, "h_scale", torch.float32, (N,), dev)
    _check(w_scale, "w_scale", torch.float32, (V,), dev)
    ids = torch.empty((N, K), dtype=torch.int32, device=dev)
    vals = torch.empty((N, K), dtype=torch.float32, device=dev)
    lse = torch.empty((N,), dtype=torch.float32, device=dev) if with_lse else None
    dropped = torch.empty((N,), dtype=torch.float32, device=dev) if with_dropped else None
    control = ws
    if ws is None:
        control = _control(dev)
        ws = _scratch(_abi.kd_teacher_topk_int8_workspace(N, dt, V, K, chunk, _rows_aligned(Wt, ld_w)), dev)
    st = _abi.kd_teacher_topk_int8(_ptr(Ht), ld_h, _ptr(h_scale), _ptr(Wt), ld_w, _ptr(w_scale), N, dt, V, K, chunk,
                                   _ptr(ids), _ptr(vals), _ptr(lse), _ptr(dropped), _ptr(ws), ws.numel(),
                                   _ptr(control), _stream(dev))
    _abi.check(st, "kd_teacher_topk_int8")
    return (ids, vals) + ((lse,) if with_lse else ()) + ((dropped,) if with_dropped else ())


def device_error(ws: torch.Tensor):
    """(status, detail) of a workspace's device error word; synchronises the current stream."""
    detail = ctypes.c_int64(0)
    st = _abi.kd_get_device_error(_ptr(ws), _stream(ws.device), ctypes.byref(detail))
    return st, detail.value


# ---------------------------------------------------------------- disk cache

def _host_c(t, dtype):
    t = torch.as_tensor(t)
    if t.is_cuda:
        t = t.cpu()
    return t.to(dtype).contiguous()


def cache_write(path: str, ids, vals, V: int, lse=None, row0: int = 0, bf16: bool = False):
    """Write a top-K cache shard (host copies of ids [N, K] int32, vals [N, K] fp32, lse [N] or None)."""
    ids = _host_c(ids, torch.int32)
    vals = _host_c(vals, torch.float32)
    N, K = ids.shape
    lse_t = None if lse is None else _host_c(lse, torch.float32)
    st = _abi.kd_cache_write(str(path).encode(), ids.data_ptr(), vals.data_ptr(), _ptr(lse_t), N, K, int(V),
                             int(row0), int(bool(bf16)))
    _abi.check(st, "kd_cache_write")


def cache_info(path: str) -> dict:
    N, K, V, row0, bf, hl = (ctypes.c_int64(), ctypes.c_int(), ctypes.c_int64(), ctypes.c_int64(), ctypes.c_int(),
                             ctypes.c_int())
    st = _abi.kd_cache_info(str(path).encode(), ctypes.byref(N), ctypes.byref(K), ctypes.byref(V), ctypes.byref(row0),
                            ctypes.byref(bf), ctypes.byref(hl))
    _abi.check(st, "kd_cache_info")
    return dict(N=N.value, K=K.value, V=V.value, row0=row0.value, bf16=bool(bf.value), has_lse=bool(hl.value))


def cache_read(path: str, first: int = 0, count: Optional[int] = None, with_lse: bool = False, pin: bool = False):
    """Read positions [first, first + count) of a shard into (pinned, if asked) host tensors."""
    info = cache_info(path)
    if count is None:
        count = info["N"] - first
    K = info["K"]
    ids = torch.empty((count, K), dtype=torch.int32, pin_memory=pin)
    vals = torch.empty((count, K), dtype=torch.float32, pin_memory=pin)
    lse = torch.empty((count,), dtype=torch.float32, pin_memory=pin) if with_lse else None
    st = _abi.kd_cache_read(str(path).encode(), int(first), int(count), ids.data_ptr(), vals.data_ptr(), _ptr(lse))
    _abi.check(st, "kd_cache_read")
    return (ids, vals, lse) if with_lse else (ids, vals)


class CacheReader:
    """Iterate a shard in batches of consecutive positions; the next batch is read from disk on a
    background thread (native) while the current one is in use.  Yields (ids, vals) host tensors."""

    def __init__(self, path: str, rows_per_batch: int, pin: bool = False):
        self.info = cache_info(path)
        self.rows = int(rows_per_batch)
        self.pin = pin
        self._h = ctypes.c_void_p()
        _abi.check(_abi.kd_cache_reader_open(str(path).encode(), self.rows, ctypes.byref(self._h)),
                   "kd_cache_reader_open")

    def __iter__(self):
        K = self.info["K"]
        while True:
            ids = torch.empty((self.rows, K), dtype=torch.int32, pin_memory=self.pin)
            vals = torch.empty((self.rows, K), dtype=torch.float32, pin_memory=self.pin)
            n = ctypes.c_int64(0)
            _abi.check(_abi.kd_cache_reader_next(self._h, ids.data_ptr(), vals.data_ptr(), ctypes.byref(n)),
                       "kd_cache_reader_next")
            if n.value == 0:
                return
            yield ids[:n.value], vals[:n.value]

    def close(self):
        if self._h:
            _abi.kd_cache_reader_close(self._h)
            self._h = ctypes.c_void_p()

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
        return False

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class Profile:
    """Per-launch CUDA-event timing of the library's kernels while the context is open."""

    def __init__(self, capacity: int = 4096):
        self.capacity = capacity
        self.records = []

    def __enter__(self):
        _abi.check(_abi.kd_profile_begin(self.capacity), "kd_profile_begin")
        return self

    def __exit__(self, *exc):
        _abi.kd_profile_end()
        n = self.capacity
        names = (ctypes.c_char_p * n)()
        ms = (ctypes.c_float * n)()
        got = _abi.kd_profile_read(names, ms, n)
        if got < 0:
            raise KDError(-got, "kd_profile_read")
        self.records = [(names[i].decode(), ms[i]) for i in range(min(got, n))]
        return False

    def summary(self):
        out = {}
        for name, t in self.records:
            c, tot = out.get(name, (0, 0.0))
            out[name] = (c + 1, tot + t)
        return out
