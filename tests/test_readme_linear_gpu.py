"""The README's example of the policy head's products runs as written and its results agree with each other."""
from __future__ import annotations

import os
import re

import pytest
import torch

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_readme_head_products(gpu):
    block = next(b for b in re.findall(r"```python\n(.*?)```", open(README).read(), re.S) if "rog_linear_logprob" in b)
    ns = {}
    exec(compile(block, "README.md", "exec"), ns)
    torch.cuda.synchronize()
    h, w = ns["hidden"].double(), torch.cat(ns["weights"]).double()
    z = h @ w.t()
    logp = torch.log_softmax(z, 1).gather(1, ns["tokens"][:, None])[:, 0]
    # binary32 sums of 512 exact products: their terms' magnitudes times 512 / 2 roundings of 2^-24, twice (token and lse)
    most = (h.abs() @ w.abs().t()).max()
    assert bool((ns["r"].logp.double() - logp).abs().max() < 512 * 2.0 ** -24 * most + 1e-5)
    # 8-bit rows are off by half a step of their own: 1/254 of the largest element, 512 random signs of it and of the weights'
    x = torch.cat(ns["logits"], 1).double()
    step = h.abs().amax(1, keepdim=True) * w.abs().sum(1) / 254 + h.abs().sum(1, keepdim=True) * (w.abs().amax(1) / 254)
    step += 512 * h.abs().amax(1, keepdim=True) * w.abs().amax(1) / 254 ** 2
    assert bool(((x - z).abs() <= step * (1 + 1e-5)).all())
    assert ns["grad"].d_hidden.dtype is torch.bfloat16 and ns["grad"].d_hidden.shape == ns["hidden"].shape
    p = torch.softmax(z, 1)
    g = -p
    g[torch.arange(100, device=gpu), ns["tokens"]] += 1
    dh = g @ w
    # G and the output are rounded to bf16: half a step of 2^-8 of the terms, and of the result
    tol = 2.0 ** -8 * (g.abs() @ w.abs() + dh.abs()) + 1e-4
    assert bool(((ns["grad"].d_hidden.double() - dh).abs() <= tol).all())
