"""examples/finetune_step.py: loss, gradient, clipping and Muon step together learn what they are given."""
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


def test_policy_training_raises_the_reward(example):
    # 1024 sampled tokens: the untrained share is 1/2 with a standard deviation of 0.016
    rewarded = example.train_policy(steps=25)
    assert 0.4 < rewarded[0] < 0.6
    assert sum(rewarded[-5:]) / 5 > 0.8


def test_preference_training_opens_the_margins(example):
    margins = example.train_preference(steps=25)
    assert abs(margins[0]) < 1e-4              # the reference is the model itself
    assert margins[-1] > 1.0 and margins[-1] > margins[5]


def test_gradients_are_clipped_on_the_way(example):
    import torch
    model = example.TokenModel()
    x = torch.randn(64, 128, device="cuda").bfloat16()
    logits, h = model.logits(x)
    norm = model.step(x, h, torch.ones_like(logits), max_norm=0.5)
    got = torch.sqrt(sum(g.double().square().sum() for g in model.clipped))
    want = torch.sqrt(sum(g.double().square().sum() for g in model.grads))
    assert norm[0].item() == pytest.approx(want.item(), rel=1e-5)
    assert norm[1].item() < 1 and got.item() == pytest.approx(0.5, rel=1e-4)
