"""Sampling and draft verification from given uniform numbers, in float64 numpy (test
infrastructure only)."""
import numpy as np


def probabilities(z, temperature=1.0):
    """softmax of each row of z / temperature; NaN throughout in a row that has none."""
    z = np.asarray(z, np.float64) / temperature
    with np.errstate(invalid="ignore"):
        e = np.exp(z - z.max(1, keepdims=True))
        return e / e.sum(1, keepdims=True)


def pick(weights, u):
    """The first index whose cumulated weight exceeds u times their sum, else the last of
    positive weight; -1 without weights."""
    total = weights.sum()
    if not total > 0:
        return -1
    over = np.nonzero((np.cumsum(weights) > max(u, 0.0) * total) & (weights > 0))[0]
    return int(over[0]) if len(over) else int(np.nonzero(weights > 0)[0][-1])


def distance(weights, u, token):
    """How far u lies outside the token's share of [0, 1) (0: inside)."""
    ends = np.cumsum(weights) / weights.sum()
    low = ends[token - 1] if token else 0.0
    return max(low - u, u - ends[token], 0.0)


def verify(p, q, drafts, lengths, accept_u, draft_q):
    """(counts, weights of the drawn token for each sequence).  p: the target's rows, q: the
    draft model's, draft_q: q at the drafts."""
    counts, weights, d, row = [], [], 0, 0
    for n in lengths:
        taken = 0
        while taken < n:
            x = drafts[d + taken]
            inside = 0 <= x < p.shape[1]
            if not (inside and accept_u[d + taken] * draft_q[d + taken] < p[row + taken, x]):
                break
            taken += 1
        w = p[row + taken]
        if taken < n:
            left = w - q[d + taken]
            left = np.where(left > 0, left, 0.0 if np.isfinite(left).all() else np.nan)
            w = left if not left.sum() == 0 else w
        counts.append(taken)
        weights.append(w)
        d += n
        row += n + 1
    return np.array(counts), weights
