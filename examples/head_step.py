"""Policy-gradient steps on one MI355X whose head's logits are never kept.

As examples/policy_step.py, a linear head over WORLD vocabulary shards in rank
order, trained by REPLICAS data-parallel replicas; but the head's products are
the library's.  Samples come from logits of the head in 8-bit integers
(rog_quantize_i8 of the states per call, of the weights once per step, then
rog_linear_i8 and rog_logprob).  Updates score the tokens straight from the states
and weights (rog_linear_logprob), take the clipped policy loss (rog_policy_loss)
and carry its gradient to states and weights (rog_linear_logprob_grad); the
replicas' weight gradients are summed in rank order (rog_reduce).  Prompts are
ragged: rows that are padding carry token -1 and cost nothing.

    python examples/head_step.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from deterministic_collective_movement_amd import rog  # noqa: E402

WORLD, REPLICAS, EPOCHS = 4, 2, 3
VOCAB, HIDDEN, PROMPTS = 10000, 256, 256


def sample(states, head8, generator):
    """One token per row from the softmax of the 8-bit head's logits."""
    q = rog.rog_quantize_i8(states)
    logits = rog.rog_linear_i8(q.q, q.scale, [w.q for w in head8], [w.scale for w in head8], dtype=torch.float32)
    lse = rog.rog_logprob(logits).lse
    p = torch.exp(torch.cat(logits, 1) - lse[:, None])
    u = torch.rand(p.shape[0], 1, generator=generator, device=p.device)
    return torch.searchsorted(p.cumsum(1), u * p.sum(1, keepdim=True)).clamp_max(VOCAB - 1)[:, 0]


def update(states, weights, tokens, old, advantage, weight, entropy_coef=0.001):
    """(loss, gradients) of one replica's tokens under the weights as they are."""
    now = rog.rog_linear_logprob(states, weights, tokens)
    loss = rog.rog_policy_loss(now.logp, old, advantage, weight=weight, entropy=now.entropy, entropy_coef=entropy_coef)
    return loss, rog.rog_linear_logprob_grad(states, weights, tokens, now.lse, now.entropy, loss.g_logp, loss.g_entropy)


def run(steps: int = 20, seed: int = 0, lr: float = 4.0):
    """Trains and returns (mean reward per step, the weight shards in binary32)."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    width = VOCAB // WORLD
    master = [0.1 * torch.randn(width, HIDDEN, generator=gen, device=dev) for _ in range(WORLD)]
    # prompts have most in common, so that what one of them learns of a token tells the others
    prompts = [(1.0 + 0.3 * torch.randn(PROMPTS, HIDDEN, generator=gen, device=dev)).bfloat16() for _ in range(REPLICAS)]
    padding = [torch.rand(PROMPTS, generator=gen, device=dev) < 0.2 for _ in range(REPLICAS)]
    liked = torch.rand(VOCAB, generator=gen, device=dev) < 0.25          # the tokens that are rewarded
    rewards = []
    for _ in range(steps):
        weights = [w.bfloat16() for w in master]
        head8 = [rog.rog_quantize_i8(w) for w in weights]
        batches, total = [], 0.0
        for x, pad in zip(prompts, padding):
            tokens = torch.where(pad, -1, sample(x, head8, gen))
            old = rog.rog_linear_logprob(x, weights, tokens).logp
            kept = (~pad).float()
            reward = liked[tokens.clamp_min(0)].float()
            mean = (reward * kept).sum() / kept.sum()
            total += float(mean)
            batches.append((x, tokens, old, (reward - mean) * kept, kept / kept.sum()))
        for _ in range(EPOCHS):
            weights = [w.bfloat16() for w in master]
            grads = [update(x, weights, tokens, old, advantage, weight)[1] for x, tokens, old, advantage, weight in batches]
            for r, w in enumerate(master):
                g = rog.rog_reduce([d.d_weights[r] for d in grads])
                w.sub_(lr / REPLICAS * g.view_as(w).float())
        rewards.append(total / REPLICAS)
    return rewards, master


def main():
    rewards, _ = run(int(sys.argv[1]) if len(sys.argv) > 1 else 20)
    for i, r in enumerate(rewards):
        if i % 5 == 0 or i + 1 == len(rewards):
            print("step %3d  mean reward %.3f" % (i, r))


if __name__ == "__main__":
    main()
