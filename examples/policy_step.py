"""Policy-gradient steps on one MI355X with a sharded policy head.

A linear policy head over WORLD vocabulary shards in rank order is trained by
REPLICAS data-parallel replicas.  Each step samples one token per prompt
(rog_logprob's log-sum-exp and alternatives score the samples, one row as well
as many) and then takes EPOCHS updates on those tokens: it scores them under the
weights as they are by then, takes the clipped policy loss against the scores
they were sampled with, with a KL term to the first policy (rog_policy_loss),
carries its gradient back to every shard's logits (rog_logprob_grad), and sums
the replicas' weight gradients in rank order (rog_reduce).  Every sum has a
fixed order, so a run repeats bit for bit, and in a step's first update, before
the weights move, every ratio is exactly 1.

    python examples/policy_step.py [steps]
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from deterministic_collective_movement_amd import rog  # noqa: E402

WORLD, REPLICAS, EPOCHS = 4, 2, 3
VOCAB, HIDDEN, PROMPTS = 10000, 64, 256


def sample(shards, lse, generator):
    """One token per row from softmax(logits), by the inverse of the cumulative sum."""
    p = torch.exp(torch.cat([s.float() for s in shards], 1) - lse[:, None])
    u = torch.rand(p.shape[0], 1, generator=generator, device=p.device)
    return torch.searchsorted(p.cumsum(1), u * p.sum(1, keepdim=True)).clamp_max(VOCAB - 1)[:, 0]


def run(steps: int = 30, seed: int = 0, lr: float = 0.15, clipped=None):
    """Trains and returns (mean reward per step, the weight shards).  ``clipped``:
    a list that gets, per step, the share of clipped tokens in each update."""
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    width = VOCAB // WORLD
    weights = [0.35 * torch.randn(HIDDEN, width, generator=gen, device=dev) for _ in range(WORLD)]
    first = [w.clone() for w in weights]
    # prompts have most in common, so that what one of them learns of a token tells the others
    prompts = [1.0 + 0.3 * torch.randn(PROMPTS, HIDDEN, generator=gen, device=dev) for _ in range(REPLICAS)]
    liked = torch.rand(VOCAB, generator=gen, device=dev) < 0.25          # the tokens that are rewarded
    rewards = []
    for _ in range(steps):
        batches, total = [], 0.0
        for x in prompts:
            logits = [(x @ w).bfloat16() for w in weights]
            before = rog.rog_logprob(logits, top_k=4)
            tokens = sample(logits, before.lse, gen)
            old = rog.rog_logprob(logits, tokens).logp
            ref = rog.rog_logprob([(x @ w).bfloat16() for w in first], tokens).logp
            reward = liked[tokens].float()
            total += float(reward.mean())
            batches.append((x, tokens, old, ref, reward - reward.mean()))
        shares = []
        for _ in range(EPOCHS):
            replica_grads, share = [], 0.0
            for x, tokens, old, ref, advantage in batches:
                logits = [(x @ w).bfloat16() for w in weights]
                now = rog.rog_logprob(logits, tokens)
                loss = rog.rog_policy_loss(now.logp, old, advantage, ref_logp=ref, entropy=now.entropy, kl_coef=0.01,
                                           entropy_coef=0.001)
                share += float(loss.stats[3]) / REPLICAS
                d = rog.rog_logprob_grad(logits, tokens, now.lse, now.entropy, loss.g_logp, loss.g_entropy, out=logits)
                replica_grads.append([x.t() @ g.float() for g in d])
            for r, w in enumerate(weights):
                grad = rog.rog_reduce([g[r].contiguous() for g in replica_grads])
                w.sub_(lr / REPLICAS * grad.view_as(w))
            shares.append(share)
        rewards.append(total / REPLICAS)
        if clipped is not None:
            clipped.append(shares)
    return rewards, weights


def main():
    clipped = []
    rewards, weights = run(int(sys.argv[1]) if len(sys.argv) > 1 else 30, clipped=clipped)
    for i in range(0, len(rewards), 5):
        print("step %3d  mean reward %.3f  clipped in its updates %s" % (i, rewards[i], ["%.2f" % c for c in clipped[i]]))
    print("last      mean reward %.3f" % rewards[-1])
    # one request's next token, with its best alternatives
    x = torch.ones(1, HIDDEN, device="cuda")
    r = rog.rog_logprob([(x @ w).bfloat16() for w in weights], top_k=5)
    print("alternatives", list(zip(r.top_ids[0].tolist(), [round(v, 3) for v in r.top_logp[0].tolist()])))


if __name__ == "__main__":
    main()
