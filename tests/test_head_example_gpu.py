"""examples/head_step.py runs, repeats bit for bit, and its gradients are the
formula's (64 bits, automatic differentiation)."""
from __future__ import annotations

import math

import pytest
import torch

from examples import head_step

pytestmark = pytest.mark.gpu


def test_runs_and_repeats(gpu):
    a, wa = head_step.run(steps=3, seed=1)
    b, wb = head_step.run(steps=3, seed=1)
    assert len(a) == 3 and all(math.isfinite(r) for r in a) and a == b
    assert all(torch.equal(x, y) and bool(torch.isfinite(x).all()) for x, y in zip(wa, wb))


def test_gradients(gpu):
    gen = torch.Generator(device=gpu)
    gen.manual_seed(3)
    n, dim = 70, head_step.HIDDEN
    x = torch.randn(n, dim, generator=gen, device=gpu).bfloat16()
    weights = [(0.1 * torch.randn(250, dim, generator=gen, device=gpu)).bfloat16() for _ in range(2)]
    tokens = torch.randint(0, 500, (n,), generator=gen, device=gpu)
    tokens[::6] = -1
    kept = tokens >= 0
    weight = kept.float() / kept.sum()
    advantage = torch.randn(n, generator=gen, device=gpu)
    h, w = x.double().requires_grad_(), torch.cat(weights).double().requires_grad_()
    lp = torch.log_softmax(h @ w.t(), 1)
    logp = lp[torch.arange(n, device=gpu), tokens.clamp_min(0)]
    old = (logp.detach() + 0.05).float()
    entropy = -(lp.exp() * lp).sum(1)
    loss = (weight * (-advantage * torch.exp(logp - old) - 0.001 * entropy)).sum()
    loss.backward()
    got, grads = head_step.update(x, weights, tokens, old, advantage, weight)
    assert abs(float(got.stats[0]) - float(loss.detach())) < 1e-5
    # coefficients and outputs are each rounded to bfloat16, by at most 2^-8
    for a, b in ((grads.d_hidden, h.grad), (torch.cat(grads.d_weights), w.grad)):
        assert float((a.double() - b).norm() / b.norm()) < 2 * 2.0 ** -8
    assert bool((grads.d_hidden[::6] == 0).all())
