"""Token log-probabilities, the policy loss and the preference loss against the fp64 oracle.

Tolerances, derived before the first run.  A row's sum of exponentials: each term is
within a few units of 2^-23 and at most about 1100 of them are added one after the
other in fp32 for the rows used here; rounding errors of a sum of positive terms grow
like the square root, sqrt(1100) 2^-24 = 2e-6, of which five times is allowed:
  logp       |error| <= LP_ABS + LP_REL |logp|, LP_ABS = 1e-5, LP_REL = 4e-7 (3 roundings)
  terms      a relative error of logp's absolute one: 2e-5 of the sum of the magnitudes
  gradient   slope and softmax each relatively 2e-5: 4e-5 (|dL/dlogp| scale) (p + 1[j = y]),
             and half a unit of bf16, 2^-9 (2^-8 with a tie's neighbour), where it is bf16
"""
import math

import numpy as np
import pytest

from gpu_util import nsm
from oracle import losses

pytestmark = pytest.mark.gpu
LP_ABS, LP_REL = 1e-5, 4e-7
CLIP = dict(clip_low=0.2, clip_high=0.28)


@pytest.fixture(scope="module")
def m():
    return nsm()


def _dev(x, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dtype is None else t.to(dtype)


def _f64(t):
    return t.detach().double().cpu().numpy()


class Batch:
    """Seeded logits with a likely token a row, on the device and as the float64 values the device holds."""

    def __init__(self, n, v, dtype="float32", pad=0, lead=0, drop=0.25, temperature=1.0, scale=2.5, seed=0):
        import torch
        rng = np.random.default_rng([n, v, seed])
        z = rng.normal(0, scale * temperature, (n, v))
        self.targets = rng.integers(0, v, n)
        z[np.arange(n), self.targets] += rng.uniform(0, 6, n) * temperature
        dt = getattr(torch, dtype)
        buffer = torch.full((lead + n * (v + pad),), 300.0, device="cuda").to(dt)
        self.logits = buffer[lead:].view(n, v + pad)[:, :v]
        self.logits.copy_(_dev(z.astype(np.float32)))
        self.z = _f64(self.logits)
        self.y = _dev(self.targets)
        self.mask = None if drop is None else rng.random(n) >= drop
        self.dmask = None if drop is None else _dev(self.mask)
        self.temperature = temperature
        self.rng, self.n, self.v = rng, n, v
        self.eps = 2.0 ** -8 if dtype == "bfloat16" else 0.0
        self.logp = losses.token_logprobs(self.z, self.targets, self.mask, temperature)

    def offsets(self, seqs):
        cut = np.sort(self.rng.integers(0, self.n + 1, seqs - 1))
        return np.concatenate([[0], cut, [self.n]]).astype(np.int64)

    def policy_inputs(self, beta):
        """Ratios on both sides of the limits and none within 1e-3 of one."""
        delta = self.rng.normal(0, 0.3, self.n)
        for lim in (math.log(0.8), math.log(1.28)):
            delta = np.where(abs(delta - lim) < 2e-3, delta + 5e-3, delta)
        old = (self.logp - delta).astype(np.float32)
        adv = self.rng.normal(0, 1, self.n).astype(np.float32)
        ref = (self.logp + self.rng.normal(0, 0.4, self.n)).astype(np.float32) if beta else None
        return old, adv, ref

    def check_logp(self, got):
        err = np.abs(_f64(got) - self.logp)
        assert (err <= LP_ABS + LP_REL * np.abs(self.logp)).all(), err.max()

    def check_grad(self, grad, slope, scale):
        assert grad.dtype == self.logits.dtype and tuple(grad.shape) == (self.n, self.v)
        want = losses.logits_gradient(self.z, self.targets, slope, self.mask, self.temperature)
        p = np.exp(losses.log_softmax(self.z, self.temperature))
        p[np.arange(self.n), self.targets] += 1
        bound = 4e-5 * np.abs(scale)[:, None] / self.temperature * p + self.eps * np.abs(want) + 1e-37
        got = _f64(grad)
        assert np.isfinite(got).all()
        worst = np.abs(got - want) / bound
        assert worst.max() <= 1, (worst.max(), np.unravel_index(worst.argmax(), worst.shape))
        if self.mask is not None:
            assert (got[~self.mask] == 0).all()


SHAPES = [(1, 1), (1, 2), (3, 7), (2, 8), (5, 33), (9, 1000), (4, 1024), (17, 4099), (300, 515), (3, 19001),
          (2, 50001), (3, 131072), (1, 160003), (2, 400009)]
LAYOUTS = [(0, 0), (3, 0), (64, 1)]


@pytest.mark.parametrize("n,v", SHAPES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("pad,lead", LAYOUTS)
def test_logprobs(m, n, v, dtype, pad, lead):
    b = Batch(n, v, dtype, pad, lead, drop=None if n < 3 else 0.25, temperature=1.0 if pad else 0.7)
    b.check_logp(m.muon_token_logprobs(b.logits, b.y, mask=b.dmask, temperature=b.temperature))


@pytest.mark.parametrize("n,v", SHAPES)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("pad,lead", LAYOUTS)
def test_policy_shapes(m, n, v, dtype, pad, lead):
    _policy(m, Batch(n, v, dtype, pad, lead, drop=None if n < 3 else 0.25), 0.1, "token")


@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
@pytest.mark.parametrize("beta", [0.0, 0.3])
@pytest.mark.parametrize("temperature", [1.0, 0.6])
@pytest.mark.parametrize("seqs", [1, 5, 60])
def test_policy_options(m, reduction, beta, temperature, seqs):
    _policy(m, Batch(41, 700, drop=0.4, temperature=temperature, seed=seqs), beta, reduction, seqs=seqs, grad_scale=3.0)


def _policy(m, b, beta, reduction, seqs=4, grad_scale=1.0, **call):
    old, adv, ref = b.policy_inputs(beta)
    offsets = b.offsets(seqs)
    want = losses.policy_loss(b.z, b.targets, old, adv, mask=b.mask, ref_logp=ref, offsets=offsets,
                              temperature=b.temperature, kl_beta=beta, reduction=reduction, logp=b.logp,
                              clip_low=float(np.float32(0.2)), clip_high=float(np.float32(0.28)))
    cfg = m.muon_policy_config_default(
        kl_beta=beta, grad_scale=grad_scale, **CLIP,
        reduction={"token": m.MUON_REDUCE_TOKEN_MEAN, "sequence": m.MUON_REDUCE_SEQUENCE_MEAN,
                   "sum": m.MUON_REDUCE_SUM}[reduction])
    stats, logp, grad = m.muon_policy_loss(b.logits, b.y, _dev(old), _dev(adv), mask=b.dmask,
                                           ref_logp=None if ref is None else _dev(ref), seq_offsets=_dev(offsets),
                                           temperature=b.temperature, config=cfg, **call)
    b.check_logp(logp)
    size = want["scale"].sum() + want["weights"].sum() * 2 * (1 + beta)
    assert np.abs(_f64(stats) - want["stats"]).max() <= 2e-5 * size
    if grad is not None:
        b.check_grad(grad, want["slope"] * grad_scale, want["scale"] * grad_scale)
    return stats, logp, grad


@pytest.mark.parametrize("drop", [0.0, 1.0])
@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
def test_policy_masks_that_keep_or_leave_nothing(m, drop, reduction):
    b = Batch(23, 300, drop=drop)
    stats, logp, grad = _policy(m, b, 0.2, reduction)
    if drop == 1.0:
        assert (stats == 0).all() and (logp == 0).all() and (grad == 0).all()


def test_policy_without_gradient_and_in_place(m):
    import torch
    b = Batch(37, 1003, "bfloat16", pad=5)
    first = _policy(m, b, 0.1, "token")
    assert _policy(m, Batch(37, 1003, "bfloat16", pad=5), 0.1, "token", with_grad=False)[2] is None
    c = Batch(37, 1003, "bfloat16", pad=5)
    edge = c.logits.as_strided((37, 5), (1008, 1), c.logits.storage_offset() + 1003).clone()
    out = _policy(m, c, 0.1, "token", grad=c.logits)
    assert out[2].data_ptr() == c.logits.data_ptr() and torch.equal(out[2], first[2])
    assert torch.equal(c.logits.as_strided((37, 5), (1008, 1), c.logits.storage_offset() + 1003), edge)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("v", [7, 1003, 70001])
@pytest.mark.parametrize("lead,pad", [(0, 0), (1, 2), (3, 5)])
def test_gradient_buffers_of_any_alignment(m, dtype, v, lead, pad):
    import torch
    b = Batch(6, v, dtype, pad=1, lead=2)
    flat = torch.full((lead + 6 * (v + pad) + 9,), 77.0, device="cuda").to(b.logits.dtype)
    grad = flat[lead:lead + 6 * (v + pad)].view(6, v + pad)[:, :v]
    _policy(m, b, 0.1, "token", grad=grad)
    rest = torch.ones(flat.numel(), dtype=torch.bool, device="cuda")
    rest[lead:lead + 6 * (v + pad)].view(6, v + pad)[:, :v] = False
    assert (flat[rest] == 77).all()


def test_policy_of_no_tokens(m):
    import torch
    z = torch.empty(0, 50, device="cuda")
    e = torch.empty(0, device="cuda")
    stats, logp, grad = m.muon_policy_loss(z, e.long(), e, e)
    assert (stats == 0).all() and logp.numel() == 0 and grad.shape == (0, 50)
    off = torch.zeros(5, dtype=torch.int64, device="cuda")
    loss, margins, sums, grad = m.muon_preference_loss(z, e.long(), off, torch.zeros(4, device="cuda"))
    assert loss.item() == pytest.approx(math.log(2), rel=1e-6) and (sums == 0).all() and (margins == 0).all()
    loss = m.muon_preference_loss(z, e.long(), off[:1], e)[0]
    assert loss.item() == 0.0
    assert m.muon_token_logprobs(z, e.long()).numel() == 0


def test_gaps_around_the_sequences_have_no_weight(m):
    b = Batch(30, 200, drop=0.2)
    old, adv, _ = b.policy_inputs(0)
    offsets = np.array([4, 9, 9, 22], np.int64)
    want = losses.policy_loss(b.z, b.targets, old, adv, mask=b.mask, offsets=offsets, reduction="sequence", logp=b.logp)
    cfg = m.muon_policy_config_default(reduction=m.MUON_REDUCE_SEQUENCE_MEAN)
    stats, _, grad = m.muon_policy_loss(b.logits, b.y, _dev(old), _dev(adv), mask=b.dmask, seq_offsets=_dev(offsets),
                                        config=cfg)
    assert np.abs(_f64(stats) - want["stats"]).max() <= 2e-5 * (want["scale"].sum() + 2)
    b.check_grad(grad, want["slope"], want["scale"])
    assert (grad[:4] == 0).all() and (grad[22:] == 0).all()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("v", [200, 5003, 131072, 500009])
def test_rows_that_move_nothing_have_zero_gradients(m, dtype, v):
    """Positions of no sequence take no part, whatever their logits; a clipped position's row is zero."""
    import torch
    b = Batch(8, v, dtype, pad=1, drop=None)
    b.logits[:2] = math.nan
    b.logits[7, 1:] = math.inf
    one = torch.ones(8, device="cuda")
    off = torch.tensor([2, 4, 7], device="cuda")
    cfg = m.muon_policy_config_default(reduction=m.MUON_REDUCE_SEQUENCE_MEAN)
    for args in (dict(), dict(grad=torch.empty(8, v, device="cuda", dtype=b.logits.dtype))):
        stats, _, grad = m.muon_policy_loss(b.logits, b.y, one * -50, one, seq_offsets=off, config=cfg, **args)
        assert stats.tolist() == pytest.approx([-1.2, -1.2, 0.0, 1.0], rel=1e-6)     # every ratio is above the limit
        assert (grad == 0).all()
        out = m.muon_preference_loss(b.logits, b.y, off, one[:2], **args)
        assert torch.isfinite(out[0]).all() and torch.isfinite(out[3]).all()
        assert (out[3][:2] == 0).all() and (out[3][7] == 0).all() and (out[3][2:7] != 0).any(1).all()


def test_offsets_out_of_range_stay_inside(m):
    # offsets beyond the batch are cut to it: nothing outside the buffers is touched
    b = Batch(12, 100, drop=None)
    old, adv, _ = b.policy_inputs(0)
    cfg = m.muon_policy_config_default(reduction=m.MUON_REDUCE_SEQUENCE_MEAN)
    offsets = np.array([-5, 6, 1 << 40], np.int64)
    stats, _, grad = m.muon_policy_loss(b.logits, b.y, _dev(old), _dev(adv), seq_offsets=_dev(offsets), config=cfg)
    want = losses.policy_loss(b.z, b.targets, old, adv, offsets=[0, 6, 12], reduction="sequence", logp=b.logp)
    assert np.abs(_f64(stats) - want["stats"]).max() <= 2e-5 * (want["scale"].sum() + 2)
    b.check_grad(grad, want["slope"], want["scale"])


PAIRS = [(2, 1, 5), (9, 1, 33), (40, 3, 1000), (64, 8, 4099), (12, 2, 50001), (700, 40, 64)]


@pytest.mark.parametrize("n,pairs,v", PAIRS)
@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("mean,smooth,temperature", [(False, 0.0, 1.0), (True, 0.1, 0.7)])
def test_preference(m, n, pairs, v, dtype, mean, smooth, temperature):
    _preference(m, Batch(n, v, dtype, pad=3, drop=0.3, temperature=temperature), pairs, mean, smooth, grad_scale=2.0)


def _preference(m, b, pairs, mean=False, smooth=0.0, beta=0.5, grad_scale=1.0, offsets=None, **call):
    offsets = b.offsets(2 * pairs) if offsets is None else offsets
    base = losses.preference_loss(b.z, b.targets, offsets, np.zeros(2 * pairs), mask=b.mask, mean=mean, logp=b.logp)
    ref = (base["seq_logp"] + b.rng.normal(0, 1, 2 * pairs)).astype(np.float32)
    beta = float(np.float32(beta))
    want = losses.preference_loss(b.z, b.targets, offsets, ref, mask=b.mask, beta=beta, smooth=float(np.float32(smooth)),
                                  mean=mean, logp=b.logp)
    cfg = m.muon_preference_config_default(beta=beta, label_smoothing=smooth, length_normalize=int(mean),
                                           grad_scale=grad_scale)
    loss, margins, sums, grad = m.muon_preference_loss(b.logits, b.y, _dev(offsets), _dev(ref), mask=b.dmask,
                                                       temperature=b.temperature, config=cfg, **call)
    # every position may be LP_ABS + LP_REL |logp| off; a mean divides by its length again
    off = np.array([(LP_ABS + LP_REL * np.abs(b.logp[s:e])).sum() for s, e in zip(offsets[:-1], offsets[1:])])
    if mean:
        live = np.ones(b.n) if b.mask is None else b.mask
        off = off / [max(1.0, live[s:e].sum()) for s, e in zip(offsets[:-1], offsets[1:])]
    assert (np.abs(_f64(sums) - want["seq_logp"]) <= off + 1e-6 + 2 ** -23 * np.abs(want["seq_logp"])).all()
    moff = beta * (off[:pairs] + off[pairs:]) + 2 ** -22 * (1 + np.abs(want["margins"]))
    assert (np.abs(_f64(margins) - want["margins"]) <= moff).all()
    # |d loss / d margin| <= 1, |d slope / d margin| <= 1/4 of beta / P
    assert abs(loss.item() - want["loss"]) <= moff.max() + 2e-6 * (1 + want["loss"])
    if grad is not None:
        scale = np.abs(want["slope"]) * (1 + 1e4 * 0.25 * moff.max()) + 1e-12
        b.check_grad(grad, want["slope"] * grad_scale, np.maximum(scale, np.abs(want["slope"]) * 2) * grad_scale)
    return loss, margins, sums, grad


def test_preference_empty_answers_and_gaps(m):
    b = Batch(20, 90, drop=0.3)
    # pair 0: both empty; pair 1: the preferred one empty; positions 0-1 and 15-19 in no sequence
    offsets = np.array([2, 2, 2, 9, 9, 15, 15], np.int64)
    loss, margins, sums, grad = _preference(m, b, 3, offsets=offsets)
    assert (grad[:2] == 0).all() and (grad[15:] == 0).all()
    assert (sums[[0, 1, 3, 5]] == 0).all()
    b = Batch(20, 90, drop=1.0)
    assert (_preference(m, b, 2)[3] == 0).all()


def test_preference_without_gradient_and_in_place(m):
    import torch
    args = dict(dtype="bfloat16", pad=1)
    first = _preference(m, Batch(24, 5001, **args), 2)
    none = _preference(m, Batch(24, 5001, **args), 2, with_grad=False)
    assert none[3] is None and torch.equal(none[0], first[0]) and torch.equal(none[1], first[1])
    b = Batch(24, 5001, **args)
    assert torch.equal(_preference(m, b, 2, grad=b.logits)[3], first[3])


def test_impossible_tokens(m):
    """Logits of -inf: probability and gradient 0; a whole row of them, or a target among them, is what the formula gives."""
    import torch
    b = Batch(8, 2053, drop=None)
    hide = b.rng.random((8, 2053)) < 0.5
    hide[np.arange(8), b.targets] = False
    hide[0] = True
    hide[0, b.targets[0]] = False                 # one possible token: logp 0
    b.logits.masked_fill_(_dev(hide), -math.inf)
    b.z = _f64(b.logits)
    b.logp = losses.token_logprobs(b.z, b.targets)
    b.check_logp(m.muon_token_logprobs(b.logits, b.y))
    _, _, grad = _policy(m, b, 0.1, "token")
    assert (grad[_dev(hide)] == 0).all()
    low = torch.finfo(torch.float32).min          # the type's lowest value instead of -inf
    b.logits.masked_fill_(_dev(hide), low)
    _policy(m, b, 0.1, "token")
    z = torch.full((3, 700), -math.inf, device="cuda")
    z[1:, 5] = 1.0
    z[2, 600] = math.nan
    lp = m.muon_token_logprobs(z, torch.tensor([3, 9, 5], device="cuda")).tolist()
    assert math.isnan(lp[0]) and lp[1] == -math.inf and math.isnan(lp[2])


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("v", [5, 700, 20011])
def test_rows_of_the_types_lowest_value(m, dtype, v):
    """Equal logits are equally likely, also where log2(e) times them leaves fp32's range."""
    import torch
    dt = getattr(torch, dtype)
    low = torch.finfo(dt).min
    z = torch.full((3, v), low, device="cuda", dtype=dt)
    z[1] = -low
    z[2, 1:] = -math.inf
    y = torch.tensor([v - 1, 0, 0], device="cuda")
    lp = m.muon_token_logprobs(z, y)
    assert lp.tolist() == pytest.approx([-math.log(v), -math.log(v), 0.0], rel=1e-6, abs=1e-6)
    one = torch.ones(3, device="cuda")
    cfg = m.muon_policy_config_default(reduction=m.MUON_REDUCE_SUM)
    grads = [m.muon_policy_loss(z, y, lp, -one, config=cfg)[2],
             m.muon_preference_loss(z, y, torch.tensor([0, 3, 3], device="cuda"), one[:2] * 0,
                                    config=m.muon_preference_config_default(beta=1e-6))[3] * -2e6]
    for g, tol in zip(grads, (2.0 ** -8, 2.0 ** -7)):
        want = torch.full((3, v), -1.0 / v, device="cuda")
        want[2] = 0
        want[[0, 1], y[:2]] += 1
        assert ((g.float() - want).abs() <= tol * want.abs() + 1e-6).all()


@pytest.mark.parametrize("where", [0, 3, 699])
@pytest.mark.parametrize("value", [math.nan, math.inf])
def test_nonfinite_logits_show(m, where, value):
    import torch
    z = torch.zeros(2, 700, device="cuda")
    z[0, where] = value
    y = torch.tensor([1, 1], device="cuda")
    lp = m.muon_token_logprobs(z, y).tolist()
    assert math.isnan(lp[0]) and lp[1] == pytest.approx(-math.log(700), rel=1e-6)


def test_masked_positions_are_not_read(m):
    import torch
    b = Batch(40, 600, drop=0.5)
    dead = _dev(~b.mask)
    b.logits[dead] = math.nan
    b.y = torch.where(dead, -100, b.y)            # a target outside the vocabulary
    b.z = np.where(b.mask[:, None], b.z, 0.0)
    _, logp, _ = _policy(m, b, 0.2, "token")
    assert (logp[dead] == 0).all()
    _preference(m, b, 3)
    # old_logp, advantages and ref_logp of masked positions may be anything too
    x = torch.where(dead, math.nan, torch.zeros(40, device="cuda"))
    cfg = m.muon_policy_config_default(kl_beta=0.1)
    stats, _, grad = m.muon_policy_loss(b.logits, b.y, x, x, mask=b.dmask, ref_logp=x, config=cfg)
    assert torch.isfinite(stats).all() and torch.isfinite(grad).all()


@pytest.mark.parametrize("target", [-1, 50, 1 << 40])
def test_targets_outside_the_vocabulary_give_nan(m, target):
    import torch
    z = torch.zeros(3, 50, device="cuda")
    y = torch.tensor([7, target, 7], device="cuda")
    lp = m.muon_token_logprobs(z, y)
    assert math.isnan(lp[1].item()) and lp[0].item() == pytest.approx(-math.log(50), rel=1e-6)
    one = torch.ones(3, device="cuda")
    stats, _, grad = m.muon_policy_loss(z, y, one * lp[0], one)
    assert math.isnan(stats[0].item()) and torch.isnan(grad[1]).all() and torch.isfinite(grad[[0, 2]]).all()


def test_extreme_ratios(m):
    """Ratios that overflow: held where the clip applies, zero where the advantage is."""
    import torch
    z = torch.zeros(4, 16, device="cuda")
    y = torch.zeros(4, dtype=torch.int64, device="cuda")
    old = torch.full((4,), -200.0, device="cuda")
    adv = torch.tensor([1.0, 0.0, -1.0, 1.0], device="cuda")
    cfg = m.muon_policy_config_default(reduction=m.MUON_REDUCE_SUM)
    stats, _, grad = m.muon_policy_loss(z[:2], y[:2], old[:2], adv[:2], config=cfg)
    assert stats[0].item() == pytest.approx(-1.2, rel=1e-6) and (grad == 0).all()
    stats, _, _ = m.muon_policy_loss(z[2:3], y[2:3], old[2:3], adv[2:3], config=cfg)
    assert stats[0].item() == math.inf            # an unbounded loss is reported as one
    stats, _, grad = m.muon_policy_loss(z[3:], y[3:], -old[3:], adv[3:], config=cfg)
    assert stats[0].item() == 0.0 and (grad == 0).all()


def test_small_kl_keeps_its_digits(m):
    """k = d^2 / 2 for tiny d: no cancellation beyond logp's own rounding."""
    import torch
    z = torch.zeros(1, 2, device="cuda")          # logp = -log 2
    y = torch.zeros(1, dtype=torch.int64, device="cuda")
    lp = m.muon_token_logprobs(z, y)
    for d in (1e-2, 0.09, 0.11, 1.0):
        ref = (lp.double() + d).float()
        exact = (ref.double() - lp.double()).item()
        cfg = m.muon_policy_config_default(kl_beta=1.0)
        stats, _, _ = m.muon_policy_loss(z, y, lp, torch.ones(1, device="cuda"), ref_logp=ref, config=cfg)
        assert stats[2].item() == pytest.approx(math.expm1(exact) - exact, rel=3e-6)


@pytest.mark.parametrize("which", ["policy", "preference"])
def test_gradient_against_differences_of_the_kernel(m, which):
    """The kernel's own loss, differenced in fp32 logits.  The loss carries an error of about
    2e-6; with a step of 2^-5 the quotient is within 2e-6 / 2^-5 = 6e-5, plus the third
    derivative's h^2 / 6 = 1.6e-4 of the slope: 4e-4."""
    import torch
    b = Batch(6, 13, drop=0.2, seed=5)
    old, adv, ref = b.policy_inputs(0.2)
    off = np.array([0, 1, 3, 4, 6], np.int64)

    def loss(z):
        if which == "policy":
            cfg = m.muon_policy_config_default(kl_beta=0.2, **CLIP)
            stats, _, g = m.muon_policy_loss(z, b.y, _dev(old), _dev(adv), mask=b.dmask, ref_logp=_dev(ref), config=cfg)
            return stats[0].item(), g
        cfg = m.muon_preference_config_default(beta=0.5)
        out = m.muon_preference_loss(z, b.y, _dev(off), torch.zeros(4, device="cuda"), mask=b.dmask, config=cfg)
        return out[0].item(), out[3]

    _, g = loss(b.logits)
    if which == "policy":     # rows whose ratio crosses a limit within the step have no derivative there
        r = np.exp(b.logp - old)
        rows = [t for t in range(6) if min(abs(math.log(r[t] / 0.8)), abs(math.log(r[t] / 1.28))) > 0.05]
    else:
        rows = range(6)
    h = 2.0 ** -5
    for t in rows:
        for j in range(13):
            up, down = b.logits.clone(), b.logits.clone()
            up[t, j] += h
            down[t, j] -= h
            d = (loss(up)[0] - loss(down)[0]) / (up[t, j] - down[t, j]).item()
            assert g[t, j].item() == pytest.approx(d, abs=4e-4), (t, j)


def test_offsets_past_32_bits(m):
    """2^31 elements and more: the first and last rows, the others masked."""
    import torch
    n, v = 16400, 131072
    z = torch.empty(n, v, device="cuda", dtype=torch.bfloat16)
    rows = [0, 1, 16383, 16384, n - 2, n - 1]
    rng = np.random.default_rng(0)
    vals = _dev(rng.normal(0, 2, (len(rows), v)).astype(np.float32)).bfloat16()
    z[rows] = vals
    y = np.zeros(n, np.int64)
    y[rows] = rng.integers(0, v, len(rows))
    mask = np.zeros(n, bool)
    mask[rows] = True
    want = losses.token_logprobs(_f64(vals), y[rows])
    dm, dy = _dev(mask), _dev(y)
    lp = m.muon_token_logprobs(z, dy, mask=dm)
    assert np.abs(_f64(lp)[rows] - want).max() <= 2e-5 and (lp[~dm] == 0).all()
    old = lp + 0.05
    adv = torch.ones(n, device="cuda")
    _, _, grad = m.muon_policy_loss(z, dy, old, adv, mask=dm)
    slope = np.full(len(rows), -math.exp(-0.05) / len(rows))
    ref = losses.logits_gradient(_f64(vals), y[rows], slope)
    got = _f64(grad[rows])
    assert (np.abs(got - ref) <= 2.0 ** -8 * np.abs(ref) + 1e-4 * abs(slope[0]) * (np.abs(ref) / abs(slope[0])) + 1e-37).all()
    assert all((grad[a:a + 1024][~dm[a:a + 1024]] == 0).all() for a in range(0, n, 1024))
    off = torch.tensor([0, 16384, n], device="cuda")
    out = m.muon_preference_loss(z, dy, off, torch.zeros(2, device="cuda"), mask=dm, grad=grad)
    assert np.abs(_f64(out[2]) - [want[:3].sum(), want[3:].sum()]).max() <= 1e-4
    d = -0.1 / (1 + math.exp(0.1 * (want[:3].sum() - want[3:].sum())))
    ref = losses.logits_gradient(_f64(vals), y[rows], np.array([d] * 3 + [-d] * 3))
    assert (np.abs(_f64(grad[rows]) - ref) <= (2.0 ** -8 + 1e-4) * np.abs(ref) + 1e-37).all()


def test_same_bits_each_time_and_on_another_stream(m):
    import torch
    b = Batch(50, 30011, "bfloat16", drop=0.2)
    old, adv, ref = (_dev(x) for x in b.policy_inputs(0.1))
    cfg = m.muon_policy_config_default(kl_beta=0.1)
    off = _dev(b.offsets(4))

    def both(**kw):
        return (*m.muon_policy_loss(b.logits, b.y, old, adv, mask=b.dmask, ref_logp=ref, config=cfg, **kw),
                *m.muon_preference_loss(b.logits, b.y, off, ref[:4], mask=b.dmask, **kw))

    first = both()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    seen = [both(stream=side) for _ in range(6)] + [both(stream=side.cuda_stream)]
    torch.cuda.synchronize()
    for s in seen:
        assert all(torch.equal(a, c) for a, c in zip(first, s))


def test_graph_capture(m):
    import torch
    b = Batch(20, 2000, "bfloat16", drop=0.2)
    old, adv, _ = (None if x is None else _dev(x) for x in b.policy_inputs(0.0))
    off = _dev(b.offsets(4))
    refs = torch.zeros(4, device="cuda")
    ws = torch.empty(m.muon_loss_workspace_bytes(20, 4), dtype=torch.uint8, device="cuda")
    z = b.logits.clone()
    outs = m.muon_policy_loss(z, b.y, old, adv, mask=b.dmask, workspace=ws)
    pref = m.muon_preference_loss(z, b.y, off, refs, mask=b.dmask, workspace=ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        m.muon_policy_loss(z, b.y, old, adv, mask=b.dmask, workspace=ws, stats=outs[0], logp=outs[1], grad=outs[2],
                           stream=side)
        m.muon_preference_loss(z, b.y, off, refs, mask=b.dmask, workspace=ws, loss=pref[0], margins=pref[1],
                               seq_logp=pref[2], grad=pref[3], stream=side)
    z.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    got = [t.clone() for t in (*outs, *pref)]
    want = (*m.muon_policy_loss(z, b.y, old, adv, mask=b.dmask), *m.muon_preference_loss(z, b.y, off, refs, mask=b.dmask))
    assert all(torch.equal(a, c) for a, c in zip(got, want))


def test_refusals(m):
    import torch
    z, y = torch.zeros(4, 30, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    f = torch.zeros(4, device="cuda")
    for args, kw in (((z.half(), y), {}), ((z[:, ::2], y), {}), ((z[0], y), {}), ((z, y.int()), {}), ((z, y[:3]), {}),
                     ((z, y), dict(mask=f)), ((z, y), dict(mask=y[:3].bool())), ((z.expand(4, 30).t(), y), {}),
                     ((z[:1].expand(4, 30), y), {}), ((z, y.cpu()), {})):
        with pytest.raises((TypeError, ValueError)):
            m.muon_token_logprobs(*args, **kw)
    for kw in (dict(grad=z[:3]), dict(grad=z.bfloat16()), dict(ref_logp=f[:2]), dict(stats=f[:3]),
               dict(grad=torch.zeros(30, 4, device="cuda").t())):
        with pytest.raises(ValueError):
            m.muon_policy_loss(z, y, f, f, **kw)
    with pytest.raises(ValueError):
        m.muon_policy_loss(z, y, f.double(), f)
    with pytest.raises(ValueError):
        m.muon_preference_loss(z, y, torch.zeros(2, dtype=torch.int64, device="cuda"), f[:1])
    with pytest.raises(m.MuonError) as e:
        m.muon_policy_loss(z, y, f, f, config=m.muon_policy_config_default(kl_beta=0.1))
    assert e.value.status == m.MUON_ERR_INVALID
    with pytest.raises(m.MuonError) as e:
        m.muon_policy_loss(z, y, f, f, workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == m.MUON_ERR_NO_WORKSPACE
    assert m.muon_token_logprobs(z, y)[0].item() == pytest.approx(-math.log(30), rel=1e-6)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("v", [200, 5003, 131072])
@pytest.mark.parametrize("mean", [False, True])
@pytest.mark.parametrize("smooth", [0.0, 0.25, 1.0])
@pytest.mark.parametrize("answer", ["preferred", "other"])
def test_preference_of_impossible_answers(m, dtype, v, mean, smooth, answer):
    """An answer with a token that cannot be taken: margin +-inf, a loss that is infinite only
    where its weight is not 0, and finite gradients."""
    b = Batch(9, v, dtype, pad=1, drop=None)
    offsets = np.array([0, 2, 4, 7, 9], np.int64)     # pair 0: rows 0-1 over 4-6, pair 1: rows 2-3 over 7-8
    row = 3 if answer == "preferred" else 7
    b.logits[row, int(b.targets[row])] = -math.inf
    b.z = _f64(b.logits)
    with np.errstate(divide="ignore"):
        b.logp = losses.token_logprobs(b.z, b.targets)
    ref = b.rng.normal(-5, 1, 4).astype(np.float32)
    want = losses.preference_loss(b.z, b.targets, offsets, ref, beta=0.5, smooth=smooth, mean=mean, logp=b.logp)
    cfg = m.muon_preference_config_default(beta=0.5, label_smoothing=smooth, length_normalize=int(mean))
    loss, margins, sums, grad = m.muon_preference_loss(b.logits, b.y, _dev(offsets), _dev(ref), config=cfg)
    sign = -1 if answer == "preferred" else 1
    assert margins[1].item() == sign * math.inf and sums[1 if answer == "preferred" else 3].item() == -math.inf
    # rows 0-1 and 4-6: at most LP_ABS + LP_REL |logp| each
    off = 0.5 * sum(LP_ABS + LP_REL * abs(b.logp[t]) for t in (0, 1, 4, 5, 6)) + 2 ** -22 * (1 + abs(want["margins"][0]))
    assert abs(margins[0].item() - want["margins"][0]) <= off
    if smooth == (0.0 if answer == "other" else 1.0):
        assert abs(loss.item() - want["loss"]) <= off + 2e-6 * (1 + want["loss"])
    else:
        assert loss.item() == math.inf == want["loss"]
    b.check_grad(grad, want["slope"], np.abs(want["slope"]) * (2 + 1e4 * 0.25 * off) + 1e-12)
