"""Log probabilities, entropy, alternatives and the dense-logits KL, in float64.

TEST INFRASTRUCTURE (see the package docstring): the definitions written out row by row
in numpy float64, with hand-written gradients.  Logits arrive as any float array and are
widened exactly.  A row whose logits are all -inf has logsumexp -inf, log probabilities
-inf, entropy 0 and zero gradients; padding rows give zeros.
"""
from __future__ import annotations

import dataclasses
from typing import Optional

import numpy as np

F64 = np.float64
REST_RESOLUTION = 2.0 ** -21  # of 1 + |t_lse|


def _log_softmax(x: np.ndarray):
    """(log_softmax, logsumexp) of one row; an all -inf row gives -inf everywhere."""
    m = np.max(x)
    if m == -np.inf:
        return np.full_like(x, -np.inf), -np.inf
    ln_s = np.log(np.sum(np.exp(x - m)))
    return x - m - ln_s, m + ln_s


def _entropy(lp: np.ndarray, p: np.ndarray) -> float:
    on = p > 0
    return float(-np.sum(p[on] * lp[on]))


@dataclasses.dataclass
class Scores:
    logp: np.ndarray
    lse: np.ndarray
    entropy: np.ndarray
    top_ids: Optional[np.ndarray] = None
    top_logp: Optional[np.ndarray] = None


def token_logprobs(logits, tokens, mask=None, tau=1.0, top=0) -> Scores:
    """Log probabilities of tokens [N, M], entropy and the top alternatives of softmax(logits / tau)."""
    z = np.asarray(logits, dtype=F64)
    N, V = z.shape
    tokens = np.asarray(tokens).reshape(N, -1)
    out = Scores(np.zeros(tokens.shape), np.zeros(N), np.zeros(N),
                 np.zeros((N, top), np.int64) if top else None, np.zeros((N, top)) if top else None)
    for r in range(N):
        if mask is not None and not mask[r]:
            continue
        lp, out.lse[r] = _log_softmax(z[r] / tau)
        out.logp[r] = lp[tokens[r]]
        out.entropy[r] = _entropy(lp, np.exp(lp))
        if top:
            order = np.lexsort((np.arange(V), -z[r]))[:top]  # value descending, then id ascending
            out.top_ids[r], out.top_logp[r] = order, lp[order]
    return out


def token_logprobs_grad(logits, tokens, g_logp, g_entropy=None, mask=None, tau=1.0) -> np.ndarray:
    """dL/dlogits for L = sum g_logp * logp + sum g_entropy * entropy."""
    z = np.asarray(logits, dtype=F64)
    N, V = z.shape
    tokens = np.asarray(tokens).reshape(N, -1)
    g_logp = np.asarray(g_logp, dtype=F64).reshape(N, -1)
    dz = np.zeros((N, V))
    for r in range(N):
        if mask is not None and not mask[r]:
            continue
        lp, lse = _log_softmax(z[r] / tau)
        if lse == -np.inf:
            continue
        p = np.exp(lp)
        d = -p * g_logp[r].sum()
        if g_entropy is not None:
            on = p > 0
            d[on] -= float(g_entropy[r]) * p[on] * (lp[on] + _entropy(lp, p))
        np.add.at(d, tokens[r], g_logp[r])
        dz[r] = d / tau
    return dz


@dataclasses.dataclass
class DenseKL:
    loss: float
    kl: np.ndarray
    grad: np.ndarray


def logits_kl(logits, ids, tlog, mask=None, tau=1.0, t_lse=None, grad_loss=1.0) -> DenseKL:
    """KL of a cached top-K teacher (with t_lse: its remaining mass as one class) against dense student logits.

    A teacher entry of logit -inf is absent; entries that share an id add up; a row without
    entries (and without t_lse) has KL 0 and no gradient; entries that cover the whole
    vocabulary leave no rest class, and a remainder below the resolution of an fp32 t_lse has
    no mass.
    """
    z = np.asarray(logits, dtype=F64)
    N, V = z.shape
    kl, grad = np.zeros(N), np.zeros((N, V))
    valid = np.ones(N, bool) if mask is None else np.asarray(mask).astype(bool)
    c = grad_loss / (max(int(valid.sum()), 1) * tau)
    for r in np.flatnonzero(valid):
        t = np.asarray(tlog[r], dtype=F64) / tau
        have = t != -np.inf
        t, at = t[have], np.asarray(ids[r])[have]
        lq, lse = _log_softmax(z[r] / tau)
        q = np.exp(lq)
        if t_lse is None:
            if not len(t):
                continue
            lp = t - (np.max(t) + np.log(np.sum(np.exp(t - np.max(t)))))
        else:
            lp = t - F64(t_lse[r])
        p = np.exp(lp)
        on = p > 0
        kl[r] = np.sum(p[on] * (lp[on] - lq[at[on]]))
        d = q.copy()
        if t_lse is not None:
            outside = np.ones(V, bool)
            outside[at] = False
            p_rest = 1.0 - float(p.sum())
            least = 0.0 if t_lse[r] == -np.inf else REST_RESOLUTION * (1.0 + abs(float(t_lse[r])))
            if not outside.any() or p_rest < least:
                p_rest = 0.0
            lq_out, lq_rest = _log_softmax(lq[outside]) if outside.any() else (None, -np.inf)
            if p_rest > 0:
                kl[r] += p_rest * (np.log(p_rest) - lq_rest)
            if lq_rest > -np.inf:
                d[outside] = (np.exp(lq_rest) - p_rest) * np.exp(lq_out)
        np.add.at(d, at, -p)
        if lse != -np.inf:
            grad[r] = c * d
    loss = float(kl[valid].sum() / valid.sum()) if valid.any() else 0.0
    return DenseKL(loss, kl, grad)
