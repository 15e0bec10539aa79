"""The README's example of the vocabulary-side operators runs as written and agrees with the formulas in 64 bits."""
from __future__ import annotations

import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_readme_head_example(gpu):
    blocks = [b for b in re.findall(r"```python\n(.*?)```", open(README).read(), re.S) if "rog_logprob" in b]
    assert len(blocks) == 1
    ns = {}
    exec(compile(blocks[0], "README.md", "exec"), ns)
    torch.cuda.synchronize()
    x = torch.cat(ns["shards"], 1).cpu()
    tokens, adv, r, loss = ns["tokens"].cpu(), ns["advantage"].cpu().double(), ns["r"], ns["loss"]
    z = (x.double() / 0.8).requires_grad_()
    lp = torch.log_softmax(z, 1)
    logp, entropy = lp.gather(1, tokens[:, None])[:, 0], -(lp.exp() * lp).sum(1)
    # numbers below 32 in binary32, from a few roundings: 1e-5 is more than five of the largest
    for got, want in ((r.logp, logp), (r.entropy, entropy), (r.lse, torch.logsumexp(z, 1))):
        assert torch.allclose(got.cpu().double(), want.detach(), rtol=0, atol=1e-5)
    ids = r.top_ids.cpu()
    assert torch.equal(x.gather(1, ids), torch.topk(x, 5, 1).values)
    assert torch.allclose(r.top_logp.cpu().double(), lp.detach().gather(1, ids), rtol=0, atol=1e-5)
    # the ratio is 1 everywhere (logp is old_logp)
    total = (-adv - 0.01 * entropy.detach()).mean()
    assert abs(float(loss.stats[0]) - float(total)) < 1e-5
    (torch.exp(logp - logp.detach()) * -adv - 0.01 * entropy).mean().backward()
    want = z.grad / 0.8
    # bf16: half a unit in the last place, at most 2^-8 of the value, and what binary32 statistics leave (1e-5 of a term that is at most |g|)
    got = torch.cat(ns["grads"], 1).cpu().double()
    assert ((got - want).abs() <= want.abs() * 2.0**-8 + 1e-5 * adv.abs().max() / 256).all()
