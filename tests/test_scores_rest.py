"""The oracle's rest class (CPU), where its masses are at the end of a type's range."""
import numpy as np
import pytest

import oracle


def test_a_students_rest_below_the_range_of_a_double():
    """The student's mass outside the cache is e^-2000 of the cached: its logarithm is what the KL takes."""
    rng = np.random.default_rng(5)
    z = rng.normal(0, 1, (3, 30))
    ids = np.stack([rng.permutation(30)[:4] for _ in range(3)])
    t = rng.normal(0, 1, (3, 4))
    np.put_along_axis(z, ids, np.take_along_axis(z, ids, 1) + 2000.0, 1)
    t_lse = np.log(np.exp(t).sum(1)) + 0.25
    got = oracle.logits_kl(z, ids, t, t_lse=t_lse)
    for r in range(3):
        out = np.setdiff1d(np.arange(30), ids[r])
        p = np.exp(t[r] - t_lse[r])
        p_rest = 1 - p.sum()
        zs = z[r][ids[r]]
        lse = zs.max() + np.log(np.exp(zs - zs.max()).sum())          # the others add nothing
        rest = np.exp(z[r][out])
        kl = (p * (np.log(p) - zs + lse)).sum() + p_rest * (np.log(p_rest) + lse - np.log(rest.sum()))
        assert np.isclose(got.kl[r], kl, rtol=1e-12)
        assert np.allclose(got.grad[r][out], -p_rest * rest / rest.sum() / 3, rtol=1e-12)


@pytest.mark.parametrize("shift", [0.0, 17.0, -40.0])
def test_a_cache_that_holds_all_of_the_teachers_mass(shift):
    rng = np.random.default_rng(3)
    N, V, K = 200, 60, 20
    ids = np.stack([rng.permutation(V)[:K] for _ in range(N)])
    t = (rng.normal(0, 3, (N, K)) + shift).astype(np.float32)
    exact = np.log(np.exp(t.astype(np.float64)).sum(1))
    z = np.full((N, V), -np.inf)
    np.put_along_axis(z, ids, rng.normal(0, 2, (N, K)), 1)
    want = oracle.logits_kl(z, ids, t)
    assert np.isfinite(want.kl).all()
    for off in (-1, 0, 1):     # the fp32 logsumexp, and its neighbours
        t_lse = np.float32(exact)
        if off:
            t_lse = np.nextafter(t_lse, np.float32(np.inf * off), dtype=np.float32)
        got = oracle.logits_kl(z, ids, t, t_lse=t_lse)
        assert np.allclose(got.kl, want.kl, rtol=0, atol=1e-4)
        assert np.allclose(got.grad, want.grad, atol=1e-6)


def test_a_rest_above_the_resolution_is_kept():
    rng = np.random.default_rng(4)
    N, V, K = 20, 60, 20
    ids = np.stack([rng.permutation(V)[:K] for _ in range(N)])
    t, z = rng.normal(0, 1, (N, K)), rng.normal(0, 1, (N, V))
    full = np.log(np.exp(t).sum(1))
    for rest in (1e-4, 0.1, 0.9):
        got = oracle.logits_kl(z, ids, t, t_lse=full - np.log1p(-rest))
        p = np.exp(t - full[:, None]) * (1 - rest)
        lq = z - np.log(np.exp(z).sum(1, keepdims=True))
        q_s = np.take_along_axis(np.exp(lq), ids, 1)
        kl = (p * (np.log(p) - np.log(q_s))).sum(1) + rest * (np.log(rest) - np.log(1 - q_s.sum(1)))
        assert np.allclose(got.kl, kl, atol=1e-10)


def test_a_teacher_row_of_nothing():
    """Every teacher logit -inf, its logsumexp too: no divergence, no gradient."""
    rng = np.random.default_rng(6)
    z = rng.normal(0, 1, (2, 20))
    ids = np.stack([rng.permutation(20)[:3] for _ in range(2)])
    t = np.full((2, 3), -np.inf)
    for t_lse in (np.full(2, -np.inf), None):
        got = oracle.logits_kl(z, ids, t, t_lse=t_lse)
        assert np.allclose(got.kl, 0, atol=1e-12) and np.allclose(got.grad, 0, atol=1e-12)
