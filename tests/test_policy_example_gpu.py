"""The policy-step example learns, and repeats bit for bit; the operators under
several host threads."""
from __future__ import annotations

import importlib.util
import os
import threading

import pytest
import torch

from deterministic_collective_movement_amd import rog

pytestmark = pytest.mark.gpu

EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "policy_step.py")


def _example():
    spec = importlib.util.spec_from_file_location("policy_step", EXAMPLE)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_learns_and_repeats(gpu):
    ex = _example()
    rewards, weights = ex.run(steps=20)
    assert sum(rewards[-3:]) / 3 > sum(rewards[:3]) / 3 + 0.1, rewards
    again, same = ex.run(steps=20)
    assert rewards == again and all(torch.equal(a, b) for a, b in zip(weights, same))


def test_host_threads_on_their_own_streams(gpu):
    gen = torch.Generator(device=gpu)
    gen.manual_seed(1)
    x = torch.randn(5, 30011, generator=gen, device=gpu).bfloat16()
    tokens = torch.randint(0, 30011, (5,), generator=gen, device=gpu)
    n = 20001
    logp, old, adv = (torch.randn(n, generator=gen, device=gpu) for _ in range(3))
    want, loss = rog.rog_logprob([x], tokens, 7), rog.rog_policy_loss(logp, old, adv)
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(40):
                    got, l2 = rog.rog_logprob([x], tokens, 7), rog.rog_policy_loss(logp, old, adv)
                    s.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)) or not torch.equal(l2.stats, loss.stats):
                        bad.append("bits")
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:3]
