"""Pins of oracle/scores.py (CPU): torch's float64 log_softmax and autograd, central
differences, hand-worked rows and limits; none of them re-types the oracle."""
import numpy as np
import pytest
import torch

import oracle


def _case(N=4, V=37, M=3, seed=0):
    rng = np.random.default_rng(seed)
    z = rng.normal(0, 2, (N, V))
    tokens = rng.integers(0, V, (N, M))
    return rng, z, tokens


@pytest.mark.parametrize("tau", [1.0, 0.7, 2.5])
def test_logprobs_match_torch(tau):
    _, z, tokens = _case()
    lp = torch.log_softmax(torch.from_numpy(z) / tau, dim=1)
    got = oracle.token_logprobs(z, tokens, tau=tau, top=5)
    assert np.allclose(got.logp, lp.gather(1, torch.from_numpy(tokens)).numpy(), atol=1e-12)
    assert np.allclose(got.lse, torch.logsumexp(torch.from_numpy(z) / tau, 1).numpy(), atol=1e-12)
    assert np.allclose(got.entropy, torch.distributions.Categorical(logits=lp).entropy().numpy(), atol=1e-12)
    v, i = lp.topk(5, dim=1)
    assert np.array_equal(got.top_ids, i.numpy()) and np.allclose(got.top_logp, v.numpy(), atol=1e-12)


def test_ties_and_empty_rows():
    z = np.array([[1.0, 3.0, 3.0, -np.inf], [-np.inf] * 4, [0.0, -0.0, 0.0, -0.0]])
    got = oracle.token_logprobs(z, np.array([[3], [0], [2]]), top=3)
    assert got.top_ids.tolist() == [[1, 2, 0], [0, 1, 2], [0, 1, 2]]
    assert got.logp[0, 0] == -np.inf and got.logp[1, 0] == -np.inf and got.lse[1] == -np.inf
    assert got.entropy[1] == 0.0 and np.isclose(got.entropy[2], np.log(4))
    assert not oracle.token_logprobs_grad(z, np.array([[3], [0], [2]]), np.ones((3, 1)))[1].any()


@pytest.mark.parametrize("tau", [1.0, 1.7])
def test_logprobs_gradient_matches_autograd(tau):
    rng, z, tokens = _case(seed=3)
    tokens[0, 1] = tokens[0, 0]  # a repeated token adds up
    g, h = rng.normal(size=tokens.shape), rng.normal(size=4)
    mask = np.array([1, 1, 0, 1])
    zt = torch.from_numpy(z).requires_grad_(True)
    lp = torch.log_softmax(zt / tau, dim=1)
    loss = (lp.gather(1, torch.from_numpy(tokens)) * torch.from_numpy(g)).sum(1)
    loss = loss - (lp.exp() * lp).sum(1) * torch.from_numpy(h)
    (loss * torch.from_numpy(mask)).sum().backward()
    assert np.allclose(oracle.token_logprobs_grad(z, tokens, g, h, mask, tau), zt.grad.numpy(), atol=1e-12)


def _kl_case(N=5, V=41, K=6, seed=1):
    rng = np.random.default_rng(seed)
    z = rng.normal(0, 2, (N, V))
    ids = np.stack([rng.permutation(V)[:K] for _ in range(N)])
    t = rng.normal(0, 2, (N, K))
    rest = np.log(np.exp(t).sum(1)) - np.log1p(-rng.uniform(0.05, 0.6, N))
    return rng, z, ids, t, rest


@pytest.mark.parametrize("tau", [1.0, 2.0])
@pytest.mark.parametrize("tail", [False, True])
def test_kl_gradient_matches_differences(tau, tail):
    rng, z, ids, t, _ = _kl_case()
    t_lse = np.log(np.exp(t / tau).sum(1)) + 0.3 if tail else None
    mask = np.array([1, 0, 1, 1, 1])
    got = oracle.logits_kl(z, ids, t, mask, tau, t_lse, grad_loss=0.7)
    eps = 1e-5
    for r, v in [(0, int(ids[0, 0])), (0, 7), (1, 3), (3, int(ids[3, 2])), (4, 11)]:
        lo, hi = z.copy(), z.copy()
        lo[r, v] -= eps
        hi[r, v] += eps
        slope = (oracle.logits_kl(hi, ids, t, mask, tau, t_lse).loss
                 - oracle.logits_kl(lo, ids, t, mask, tau, t_lse).loss) / (2 * eps)
        assert abs(got.grad[r, v] - 0.7 * slope) < 1e-9


def test_kl_without_rest_is_the_dense_oracle():
    """With H = z and W = I the fused loss's dense formulation sees the same logits."""
    _, z, ids, t, _ = _kl_case(V=16)
    z = torch.from_numpy(z).to(torch.bfloat16)
    bits = z.view(torch.int16).numpy().view(np.uint16)
    eye = torch.eye(16, dtype=torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
    ref = oracle.dense_kl(bits, eye, ids.astype(np.int32), t.astype(np.float32), None, 1.0)
    got = oracle.logits_kl(z.double().numpy(), ids, t.astype(np.float32))
    assert abs(got.loss - ref.loss) < 1e-12 and np.allclose(got.kl, ref.kl, atol=1e-12)
    assert np.allclose(got.grad, ref.grad_H, atol=1e-12)  # W = I: grad_H is dL/dz


def test_kl_with_rest_is_the_kl_of_the_merged_classes():
    _, z, ids, t, t_lse = _kl_case()
    got = oracle.logits_kl(z, ids, t, t_lse=t_lse)
    p = np.exp(t - t_lse[:, None])
    lq = torch.log_softmax(torch.from_numpy(z), 1)
    qk = lq.exp().gather(1, torch.from_numpy(ids)).numpy()
    P = np.concatenate([p, 1 - p.sum(1, keepdims=True)], 1)
    Q = np.concatenate([qk, 1 - qk.sum(1, keepdims=True)], 1)
    ref = torch.nn.functional.kl_div(torch.from_numpy(Q).log(), torch.from_numpy(P), reduction="none").sum(1).numpy()
    assert np.allclose(got.kl, ref, atol=1e-10) and (got.kl >= 0).all()
    assert np.allclose(got.grad.sum(1), 0, atol=1e-12)  # each row of a softmax gradient sums to 0


def test_kl_absent_repeated_and_empty_entries():
    _, z, ids, t, t_lse = _kl_case(N=3)
    t2, ids2 = t.copy(), ids.copy()
    t2[0, 4:] = -np.inf          # absent: as if the cache were shorter
    a = oracle.logits_kl(z[:1], ids[:1, :4], t[:1, :4])
    b = oracle.logits_kl(z[:1], ids2[:1], t2[:1])
    assert np.isclose(a.kl[0], b.kl[0]) and np.allclose(a.grad, b.grad)
    ids2[1, 3] = ids2[1, 0]      # repeated: one entry of the summed probability in the gradient
    g = oracle.logits_kl(z[1:2], ids2[1:2], t[1:2]).grad[0]
    p = np.exp(t[1]) / np.exp(t[1]).sum()
    q = np.exp(z[1]) / np.exp(z[1]).sum()
    at = ids2[1, 0]
    assert np.isclose(g[at], q[at] - p[0] - p[3])
    t2[2] = -np.inf              # nothing cached
    e = oracle.logits_kl(z[2:3], ids[2:3], t2[2:3])
    assert e.kl[0] == 0 and not e.grad.any()


def test_planted_slips_are_caught():
    """The pins above see a wrong sign, a missing temperature, an unnormalised rest class."""
    rng, z, ids, t, t_lse = _kl_case()
    got = oracle.logits_kl(z, ids, t, t_lse=t_lse)
    p = np.exp(t - t_lse[:, None])
    wrong = oracle.logits_kl(z, ids, t).grad  # teacher renormalised although the rest is kept
    assert not np.allclose(got.grad, wrong, atol=1e-6)
    tok = ids[:, :1]
    g = np.ones(tok.shape)
    assert not np.allclose(oracle.token_logprobs_grad(z, tok, g, tau=2.0), oracle.token_logprobs_grad(z, tok, g), atol=1e-3)
    assert (oracle.token_logprobs_grad(z, tok, g)[np.arange(5), tok[:, 0]] > 0).all()
    assert (p.sum(1) < 1).all()
