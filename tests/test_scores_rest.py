"""The oracle's rest class (CPU), where its masses are at the end of a type's range."""
import numpy as np

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
