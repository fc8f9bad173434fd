"""examples/finetune_step.py with drafted rollouts and activations kept in 8 bits: it runs, and
its gradients are those of the values it kept.

Tolerance, derived before the first run: a gradient sums products whose factors dh, dgate, dup
and h were rounded to bf16, half a step of 2^-8 each and dgate of a rounded dh besides, and is
rounded to bf16 itself: 3 * 2^-8 of the sum of magnitudes.
"""
import math
import os
import sys

import pytest

from gpu_util import nsm

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module")
def example():
    nsm()
    import finetune_step
    return finetune_step


@pytest.mark.parametrize("drafts,gated", [(3, False), (0, True), (4, True)])
def test_policy_training_runs(example, drafts, gated):
    kind = example.GatedModel if gated else example.TokenModel
    rewarded = example.train_policy(steps=3, drafts=drafts, model_type=kind)
    assert len(rewarded) == 3 and all(0 <= r <= 1 and math.isfinite(r) for r in rewarded)


def test_preference_training_runs(example):
    margins = example.train_preference(steps=3, model_type=example.GatedModel)
    assert len(margins) == 3 and all(math.isfinite(v) for v in margins)


def test_drafted_rollout(example):
    import torch
    gen = torch.Generator("cuda").manual_seed(3)
    logits = torch.randn(120, 500, generator=gen, device="cuda")
    reference = logits + 0.5 * torch.randn(120, 500, generator=gen, device="cuda")
    tokens, logp = example.drafted_rollout(logits, reference, 3, gen)
    t = tokens.view(30, 4)
    drawn = t >= 0
    assert drawn[:, 0].all() and (drawn[:, 1:] <= drawn[:, :-1]).all()   # tokens first, -1 behind them
    want = logits.double().log_softmax(1).gather(1, tokens.clamp(min=0)[:, None])[:, 0]
    live = tokens >= 0
    assert (logp[~live] == 0).all() and (logp.double() - want)[live].abs().max() <= 1e-5 + 4e-7 * want.abs().max()


def test_gated_gradients_are_those_of_the_saved_values(example):
    import torch
    gen = torch.Generator("cuda").manual_seed(4)
    model = example.GatedModel()
    x = torch.randn(300, 128, generator=gen, device="cuda").bfloat16()
    logits, saved = model.logits(x)
    dlogits = (torch.randn(logits.shape, generator=gen, device="cuda") * 0.01).bfloat16()
    model.backward(x, saved, dlogits)
    m = example.nsm
    lx, lg, lu = (m.muon_checkpoint_load(c).double() for c in saved)
    d, w = dlogits.double(), model.weights[2].bfloat16().double()
    g, u = lg.clone().requires_grad_(), lu.clone().requires_grad_()
    h = torch.nn.functional.silu(g) * u
    h.backward(d @ w)
    dh_terms = d.abs() @ w.abs()                       # dh is a rounded sum of these
    sig = torch.sigmoid(lg)
    dg_terms = dh_terms * lu.abs() * sig * (1 + lg.abs() * (1 - sig))
    du_terms = dh_terms * (lg * sig).abs()
    for got, left, right, lt, rt in ((model.grads[0], g.grad, lx, dg_terms, lx.abs()), (model.grads[1], u.grad, lx, du_terms, lx.abs()),
                                     (model.grads[2], d, h.detach(), d.abs(), h.detach().abs())):
        want, terms = left.t() @ right, lt.t() @ rt
        assert ((got.double() - want).abs() <= 3 * 2.0 ** -8 * terms).all()
        assert got.double().abs().max() > 0
