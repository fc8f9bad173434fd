"""Fine-tuning with the whole chain on one GPU: loss, gradient, clipping, Muon step.

A two-layer token model (logits = relu(x W1^T) W2^T, fp32 master weights, bf16 products)
is trained
  policy      on tokens sampled from itself and rewarded where they are even, with the
              clipped policy loss and a KL term to the initial model;
  preference  on pairs of fixed answers, with the preference loss.
Each step: logits by torch, the loss and its gradient by muon_policy_loss or
muon_preference_loss (in place of the logits), the weights' gradients by torch, their
clipping by muon_clip_grad_norm, and muon_step.

  python examples/finetune_step.py [policy|preference] [--steps N]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_muon_gb300 as nsm  # noqa: E402


class TokenModel:
    """x [tokens, inputs] bf16 -> logits [tokens, vocab] bf16."""

    def __init__(self, inputs=128, hidden=512, vocab=2048, seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.weights = [torch.randn(hidden, inputs, generator=gen, device="cuda") * inputs ** -0.5,
                        torch.randn(vocab, hidden, generator=gen, device="cuda") * hidden ** -0.5]
        self.momentum = [torch.zeros_like(w) for w in self.weights]
        config = nsm.muon_config_default(grad_dtype=nsm.MUON_DTYPE_F32)
        self.plan = nsm.muon_plan([tuple(w.shape) for w in self.weights], config=config)
        nsm.allocate_workspace(self.plan)
        # the gradients' place: bf16 as the products leave them, clipped into fp32
        self.grads = [torch.empty_like(w, dtype=torch.bfloat16) for w in self.weights]
        self.clipped = [torch.empty_like(w) for w in self.weights]
        self.grad_set = nsm.GradSet(self.grads, self.clipped)

    def logits(self, x):
        w1, w2 = (w.bfloat16() for w in self.weights)
        h = torch.relu(x @ w1.t())
        return h @ w2.t(), h

    def step(self, x, h, dlogits, max_norm=1.0, lr=0.05, momentum=0.9):
        """Backward from the logits' gradient, clip, update; returns the (norm, factor) tensor."""
        torch.matmul(dlogits.t(), h, out=self.grads[1])
        dh = (dlogits @ self.weights[1].bfloat16()) * (h > 0)
        torch.matmul(dh.t(), x, out=self.grads[0])
        norm = nsm.muon_clip_grad_norm(self.grad_set, max_norm)
        nsm.muon_step(self.plan, self.weights, self.clipped, self.momentum, lr, momentum, True, 0.0)
        return norm


def train_policy(steps=30, tokens=1024, sequences=32, updates=2, seed=0):
    """Returns the share of rewarded tokens at each step (1/2 for an untrained model)."""
    gen = torch.Generator("cuda").manual_seed(seed + 1)
    model = TokenModel(seed=seed)
    reference = [w.clone() for w in model.weights]
    offsets = torch.linspace(0, tokens, sequences + 1, device="cuda").long()
    config = nsm.muon_policy_config_default(kl_beta=0.02, clip_high=0.28, reduction=nsm.MUON_REDUCE_SEQUENCE_MEAN)
    rewarded = []
    for _ in range(steps):
        x = torch.randn(tokens, 128, generator=gen, device="cuda").bfloat16()
        # rollout: the sampled tokens' log-probabilities under this policy and the initial one
        logits, _ = model.logits(x)
        sampled = torch.multinomial(logits.float().softmax(1), 1, generator=gen)[:, 0]
        old = nsm.muon_token_logprobs(logits, sampled)
        now, model.weights = model.weights, reference
        ref = nsm.muon_token_logprobs(model.logits(x)[0], sampled)
        model.weights = now
        reward = (sampled % 2 == 0).float()
        rewarded.append(reward.mean().item())
        advantage = (reward - reward.mean()) / reward.std().clamp(min=1e-3)
        prompt = torch.rand(tokens, generator=gen, device="cuda") < 0.1   # positions that take no part
        for _ in range(updates):
            logits, h = model.logits(x)
            _, _, dlogits = nsm.muon_policy_loss(logits, sampled, old, advantage, mask=~prompt, ref_logp=ref,
                                                 seq_offsets=offsets, config=config, grad=logits)
            model.step(x, h, dlogits)
        status, nonfinite = nsm.muon_sync(model.plan)
        assert status == nsm.MUON_OK and nonfinite == 0
    return rewarded


def train_preference(steps=30, pairs=16, length=24, seed=0):
    """Returns the mean margin at each step (0 for an untrained model)."""
    gen = torch.Generator("cuda").manual_seed(seed + 2)
    model = TokenModel(seed=seed)
    tokens = 2 * pairs * length
    x = torch.randn(tokens, 128, generator=gen, device="cuda").bfloat16()
    answers = torch.randint(0, 2048, (tokens,), generator=gen, device="cuda")
    offsets = torch.arange(0, tokens + 1, length, device="cuda")
    mask = torch.rand(tokens, generator=gen, device="cuda") > 0.2
    config = nsm.muon_preference_config_default(beta=0.1, label_smoothing=0.05)
    # the reference policy's sums: those of the initial model
    ref = nsm.muon_preference_loss(model.logits(x)[0], answers, offsets, torch.zeros(2 * pairs, device="cuda"),
                                   mask=mask, with_grad=False)[2].clone()
    margins = []
    for _ in range(steps):
        logits, h = model.logits(x)
        _, margin, _, dlogits = nsm.muon_preference_loss(logits, answers, offsets, ref, mask=mask, config=config,
                                                         grad=logits)
        margins.append(margin.mean().item())
        model.step(x, h, dlogits, lr=0.005)
    status, nonfinite = nsm.muon_sync(model.plan)
    assert status == nsm.MUON_OK and nonfinite == 0
    return margins


def main():
    parser = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    parser.add_argument("loss", nargs="?", default="policy", choices=["policy", "preference"])
    parser.add_argument("--steps", type=int, default=30)
    args = parser.parse_args()
    train, what = {"policy": (train_policy, "share of rewarded tokens"),
                   "preference": (train_preference, "mean margin")}[args.loss]
    for step, value in enumerate(train(args.steps)):
        print(f"step {step:3d}  {what} {value:.4f}")


if __name__ == "__main__":
    main()
