"""Losses on token log-probabilities and clipping by the global norm, in plain fp64 numpy.

Test infrastructure only; written from the formulas in include/muon.h and sharing no
code with the kernels.  Arrays are any float type on the way in and float64 inside.
"""
from __future__ import annotations

import numpy as np


def grad_norm(grads) -> float:
    total = np.float64(0.0)
    with np.errstate(over="ignore", invalid="ignore"):
        for g in grads:
            x = np.asarray(g, np.float64).ravel()
            total += np.dot(x, x)
    return float(np.sqrt(total))


def clip_factor(norm: float, max_norm: float, eps: float, zero_nonfinite: bool = False) -> float:
    if not np.isfinite(norm):
        return 0.0 if zero_nonfinite else 1.0
    den = norm + eps
    return 1.0 if den <= max_norm else max_norm / den


def log_softmax(logits, temperature=1.0):
    z = np.asarray(logits, np.float64) / temperature
    m = z.max(axis=-1, keepdims=True)
    return z - m - np.log(np.exp(z - m).sum(axis=-1, keepdims=True))


def token_logprobs(logits, targets, mask=None, temperature=1.0):
    out = np.zeros(len(targets))
    for t in range(len(targets)):
        if mask is None or mask[t]:
            out[t] = log_softmax(logits[t], temperature)[targets[t]]
    return out


def logits_gradient(logits, targets, slope, mask=None, temperature=1.0):
    """slope_t / temperature (1[j = y_t] - softmax(z_t)_j), zero rows where masked."""
    g = np.zeros(np.shape(logits))
    for t in range(len(targets)):
        if mask is None or mask[t]:
            row = -np.exp(log_softmax(logits[t], temperature))
            # 1 - p without its cancellation
            row[targets[t]] = -np.expm1(log_softmax(logits[t], temperature)[targets[t]])
            g[t] = slope[t] / temperature * row
    return g


def position_weights(n, mask, reduction, offsets=None):
    live = np.ones(n) if mask is None else np.asarray(mask).astype(np.float64)
    if reduction == "sum":
        return live
    if reduction == "token":
        return live / max(1.0, live.sum())
    w = np.zeros(n)
    seqs = len(offsets) - 1
    for q in range(seqs):
        part = slice(offsets[q], offsets[q + 1])
        w[part] = live[part] / (seqs * max(1.0, live[part].sum()))
    return w


def policy_loss(logits, targets, old_logp, adv, *, mask=None, ref_logp=None, offsets=None, temperature=1.0,
                clip_low=0.2, clip_high=0.2, kl_beta=0.0, reduction="token", logp=None):
    """Returns a dict: stats (loss, policy term, KL term, clipped share), logp, slope
    (dL/dlogp), weights, and scale, the sum of the slope's terms' magnitudes."""
    n = len(targets)
    if logp is None:
        logp = token_logprobs(logits, targets, mask, temperature)
    w = position_weights(n, mask, reduction, offsets)
    stats, slope, scale = np.zeros(4), np.zeros(n), np.zeros(n)
    for t in range(n):
        if w[t] == 0:
            continue
        r, a = np.exp(logp[t] - old_logp[t]), np.float64(adv[t])
        plain, held = r * a, min(max(r, 1 - clip_low), 1 + clip_high) * a
        clipped = held < plain
        kl, dkl = 0.0, 0.0
        if kl_beta:
            d = np.float64(ref_logp[t]) - logp[t]
            kl, dkl = np.expm1(d) - d, -np.expm1(d)
        s = min(plain, held)
        stats += w[t] * np.array([-s + kl_beta * kl, -s, kl, float(clipped)])
        slope[t] = w[t] * ((0.0 if clipped else -plain) + kl_beta * dkl)
        scale[t] = w[t] * (abs(plain) + abs(kl_beta) * (1 + np.exp(0.0 if not kl_beta else d)))
    return dict(stats=stats, logp=logp, slope=slope, weights=w, scale=scale)


def preference_loss(logits, targets, offsets, ref, *, mask=None, temperature=1.0, beta=0.1, smooth=0.0, mean=False,
                    logp=None):
    """Returns a dict: loss, margins, seq_logp, logp, slope (dL/dlogp)."""
    n, pairs = len(targets), (len(offsets) - 1) // 2
    if logp is None:
        logp = token_logprobs(logits, targets, mask, temperature)
    live = np.ones(n) if mask is None else np.asarray(mask).astype(np.float64)
    sums, per = np.zeros(2 * pairs), np.ones(2 * pairs)
    for q in range(2 * pairs):
        part = slice(offsets[q], offsets[q + 1])
        per[q] = max(1.0, live[part].sum()) if mean else 1.0
        sums[q] = (logp[part] * live[part]).sum() / per[q]
    gain = sums - np.asarray(ref, np.float64)
    margins = beta * (gain[:pairs] - gain[pairs:])
    log_sig = lambda h: -np.logaddexp(0.0, -h)  # noqa: E731
    term = lambda weight, h: weight * log_sig(h) if weight else np.zeros(pairs)  # noqa: E731  (0, not 0 * inf)
    loss = -np.mean(term(1 - smooth, margins) + term(smooth, -margins)) if pairs else 0.0
    slope = np.zeros(n)
    for i in range(pairs):
        sig = np.exp(log_sig(margins[i]))
        d = beta / pairs * (smooth * sig - (1 - smooth) * (1 - sig))
        for q, sign in ((i, 1.0), (pairs + i, -1.0)):
            part = slice(offsets[q], offsets[q + 1])
            slope[part] = sign * d / per[q] * live[part]
    return dict(loss=float(loss), margins=margins, seq_logp=sums, logp=logp, slope=slope)
