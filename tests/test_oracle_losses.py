"""The fp64 loss oracle against closed forms and differences (no library code runs)."""
import numpy as np
import pytest

from oracle import losses


def _batch(rng, n=7, v=11, scale=2.0):
    logits = rng.normal(0, scale, (n, v))
    targets = rng.integers(0, v, n)
    mask = rng.random(n) > 0.25
    return logits, targets, mask


def _differences(f, logits, h=1e-6):
    g = np.zeros_like(logits)
    for i in np.ndindex(*logits.shape):
        up, down = logits.copy(), logits.copy()
        up[i] += h
        down[i] -= h
        g[i] = (f(up) - f(down)) / (2 * h)
    return g


def test_logprobs_of_a_uniform_row_and_shift_invariance():
    rng = np.random.default_rng(0)
    assert losses.token_logprobs(np.zeros((1, 8)), [3])[0] == pytest.approx(-np.log(8), rel=1e-15)
    logits, targets, _ = _batch(rng)
    a = losses.token_logprobs(logits, targets)
    assert a == pytest.approx(losses.token_logprobs(logits + 100.0, targets), abs=1e-12)
    # the probabilities over all targets sum to one
    p = sum(np.exp(losses.token_logprobs(logits, np.full(7, j))) for j in range(11))
    assert p == pytest.approx(np.ones(7), abs=1e-14)


@pytest.mark.parametrize("reduction", ["token", "sequence", "sum"])
@pytest.mark.parametrize("beta", [0.0, 0.3])
@pytest.mark.parametrize("temperature", [1.0, 0.6])
def test_policy_gradient_against_differences(reduction, beta, temperature):
    rng = np.random.default_rng(1)
    logits, targets, mask = _batch(rng)
    offsets = [0, 2, 2, 7]
    old = losses.token_logprobs(logits, targets, None, temperature) + rng.normal(0, 0.3, 7)
    kw = dict(mask=mask, ref_logp=old + 0.2, offsets=offsets, temperature=temperature, kl_beta=beta,
              reduction=reduction)
    adv = rng.normal(0, 1, 7)
    out = losses.policy_loss(logits, targets, old, adv, **kw)
    got = losses.logits_gradient(logits, targets, out["slope"], mask, temperature)
    want = _differences(lambda z: losses.policy_loss(z, targets, old, adv, **kw)["stats"][0], logits)
    assert got == pytest.approx(want, abs=2e-8)
    assert out["stats"][0] == pytest.approx(out["stats"][1] + beta * out["stats"][2], abs=1e-14)


def test_policy_at_the_rollout_policy():
    # logp = old: every ratio is 1, nothing is clipped, the loss is -mean(A)
    rng = np.random.default_rng(2)
    logits, targets, _ = _batch(rng)
    old = losses.token_logprobs(logits, targets)
    adv = rng.normal(0, 1, 7)
    out = losses.policy_loss(logits, targets, old, adv, ref_logp=old, kl_beta=1.0)
    assert out["stats"] == pytest.approx([-adv.mean(), -adv.mean(), 0.0, 0.0], abs=1e-14)
    assert out["slope"] == pytest.approx(-adv / 7, abs=1e-15)


def test_policy_clipping_has_the_four_corners():
    lp = np.log([1.5, 1.5, 0.5, 0.5])
    out = losses.policy_loss(None, np.zeros(4, int), np.zeros(4), [1, -1, 1, -1.0], reduction="sum", logp=lp)
    # a gain above the upper limit and a loss below the lower one are held, and have no slope
    assert out["slope"] == pytest.approx([0, 1.5, -0.5, 0], abs=1e-14)
    assert out["stats"][3] == 2 and out["stats"][1] == pytest.approx(-(1.2 - 1.5 + 0.5 - 0.8), abs=1e-14)


@pytest.mark.parametrize("smooth", [0.0, 0.2])
@pytest.mark.parametrize("mean", [False, True])
def test_preference_gradient_against_differences(smooth, mean):
    rng = np.random.default_rng(3)
    logits, targets, mask = _batch(rng)
    offsets, ref = [0, 2, 3, 3, 7], rng.normal(-4, 1, 4)      # one answer is empty
    kw = dict(mask=mask, temperature=0.8, beta=0.7, smooth=smooth, mean=mean)
    out = losses.preference_loss(logits, targets, offsets, ref, **kw)
    got = losses.logits_gradient(logits, targets, out["slope"], mask, 0.8)
    want = _differences(lambda z: losses.preference_loss(z, targets, offsets, ref, **kw)["loss"], logits)
    assert got == pytest.approx(want, abs=2e-9)


def test_preference_of_equal_answers_is_log_two():
    rng = np.random.default_rng(4)
    logits, targets, _ = _batch(rng, n=4)
    logits, targets = np.concatenate([logits, logits]), np.concatenate([targets, targets])
    out = losses.preference_loss(logits, targets, [0, 4, 8], np.zeros(2))
    assert out["loss"] == pytest.approx(np.log(2), rel=1e-14) and out["margins"][0] == pytest.approx(0, abs=1e-14)
    # swapping the answers of a pair turns the margin's sign
    ref = np.array([-1.0, -2.5])
    a = losses.preference_loss(logits, targets, [0, 4, 8], ref)["margins"]
    b = losses.preference_loss(logits, targets, [0, 4, 8], ref[::-1])["margins"]
    assert a == pytest.approx(-b, abs=1e-14)


def test_clip_factor():
    g = [np.array([3.0]), np.array([[0.0, 4.0]])]
    assert losses.grad_norm(g) == 5.0
    assert losses.clip_factor(5.0, 1.0, 0.0) == pytest.approx(0.2)
    assert losses.clip_factor(5.0, 5.0, 0.0) == 1.0 and losses.clip_factor(0.0, 0.0, 0.0) == 1.0
    assert losses.clip_factor(np.inf, 1.0, 0.0) == 1.0 and losses.clip_factor(np.nan, 1.0, 0.0, True) == 0.0


@pytest.mark.parametrize("smooth", [0.0, 0.25, 1.0])
def test_preference_of_impossible_answers(smooth):
    """A margin of +-inf: a term of weight 0 is 0, another is its limit."""
    logp, offsets, ref = np.array([-1.0, -np.inf, -2.0, -3.0]), [0, 1, 2, 3, 4], np.zeros(4)
    # pair 0: an ordinary answer over an ordinary one (h = 0.1), pair 1: an impossible one over an ordinary one
    out = losses.preference_loss(None, np.zeros(4, int), offsets, ref, logp=logp, smooth=smooth)
    one = (1 - smooth) * np.log1p(np.exp(-0.1)) + smooth * np.log1p(np.exp(0.1))
    assert out["margins"].tolist() == [pytest.approx(0.1), -np.inf]
    assert out["loss"] == (pytest.approx(one / 2) if smooth == 1.0 else np.inf)
    # pair 1 turned round
    turned = losses.preference_loss(None, np.zeros(4, int), offsets, ref, logp=logp[[0, 3, 2, 1]], smooth=smooth)
    assert turned["margins"].tolist() == [pytest.approx(0.1), np.inf]
    assert turned["loss"] == (pytest.approx(one / 2) if smooth == 0.0 else np.inf)
    # d loss / d margin = smooth sigmoid(h) - (1 - smooth) sigmoid(-h)
    assert out["slope"][[1, 3]] == pytest.approx([-0.05 * (1 - smooth), 0.05 * (1 - smooth)])
    assert turned["slope"][[1, 3]] == pytest.approx([0.05 * smooth, -0.05 * smooth])
