"""The float64 sampling oracle against closed forms."""
import numpy as np

from oracle import sampling


def test_pick():
    w = np.array([0.0, 0.25, 0.0, 0.5, 0.25, 0.0])
    assert [sampling.pick(w, u) for u in (-1, 0, 0.2499, 0.25, 0.7499, 0.75, 0.9999, 1.0, 5.0)] == [1, 1, 1, 3, 3, 4, 4, 4, 4]
    assert sampling.pick(np.zeros(3), 0.5) == -1
    assert sampling.distance(w, 0.3, 3) == 0 and np.isclose(sampling.distance(w, 0.2, 3), 0.05)


def test_emitted_tokens_have_the_targets_distribution():
    """One draft: sum over drafts and uniforms of what is emitted is the target's row."""
    rng = np.random.default_rng(0)
    p, after, q = (w / w.sum() for w in rng.random((3, 5)))
    emitted = np.zeros(5)
    for x in range(5):
        taken = min(1.0, p[x] / q[x])
        emitted[x] += q[x] * taken
        if taken < 1:
            u = (taken + 1) / 2
            counts, weights = sampling.verify(np.stack([p, after]), q[None], [x], [1], [u], [q[x]])
            assert counts[0] == 0
            emitted += q[x] * (1 - taken) * weights[0] / weights[0].sum()
        counts, weights = sampling.verify(np.stack([p, after]), q[None], [x], [1], [taken * 0.999], [q[x]])
        assert counts[0] == 1 and (weights[0] == after).all()
    np.testing.assert_allclose(emitted, p, atol=1e-12)


def test_nothing_left_and_no_probabilities():
    p = sampling.probabilities([[0.0, 1.0, 2.0]] * 2)
    _, w = sampling.verify(p, p[:1], [1], [1], [1.0], [p[0, 1]])
    assert (w[0] == p[0]).all()
    bad = sampling.probabilities([[0.0, np.inf], [np.nan, 1.0]])
    assert np.isnan(bad).all()
