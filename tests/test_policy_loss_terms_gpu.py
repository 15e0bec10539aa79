"""The policy loss where binary32 alone would lose what the formula says:
infinite ratios that it multiplies by zero, and tokens that cancel."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from deterministic_collective_movement_amd import rog
from tests import head_ref as ref

pytestmark = pytest.mark.gpu


def vec(values, gpu):
    return torch.tensor(values, dtype=torch.float32, device=gpu)


RATIOS = [0.0, 5.0, 88.0, 88.8, 95.0, 200.0, 1e30, -88.8, -200.0, -1e30]


def test_no_advantage_no_term(gpu):
    """An advantage of 0 adds 0, however large the ratio."""
    d = vec(RATIOS, gpu)
    zero = torch.zeros(len(RATIOS), device=gpu)
    for adv in (zero, -zero):
        for high in (0.2, math.inf):
            got = rog.rog_policy_loss(d, zero, adv, weight=torch.ones(len(RATIOS), device=gpu), clip_low=1.0, clip_high=high)
            assert got.stats.tolist() == [0.0] * 4 and bool((got.g_logp == 0).all())
    # beside tokens that count
    both, adv = torch.cat([d, vec([0.1], gpu)]), torch.cat([zero, vec([-2.0], gpu)])
    got = rog.rog_policy_loss(both, torch.zeros_like(both), adv, weight=torch.ones_like(both))
    want = 2.0 * math.exp(float(np.float32(0.1)))
    assert abs(float(got.stats[0]) - want) <= 8 * ref.U * want and float(got.g_logp[-1]) == pytest.approx(want, rel=8 * ref.U)


def test_an_advantage_of_nothing_hides_no_nan(gpu):
    zero = torch.zeros(3, device=gpu)
    got = rog.rog_policy_loss(vec([0.0, math.nan, 0.0], gpu), zero, zero, weight=torch.ones(3, device=gpu))
    assert math.isnan(got.stats[0].item()) and [math.isnan(v) for v in got.g_logp.tolist()] == [False, True, False]


def test_kl_that_is_only_watched(gpu):
    """kl_coef 0 with a reference: stats hold the KL, the loss and the gradient nothing of it."""
    q = vec(RATIOS, gpu)
    n = len(RATIOS)
    zero, one = torch.zeros(n, device=gpu), torch.ones(n, device=gpu)
    got = rog.rog_policy_loss(zero, zero, -one, weight=one, ref_logp=q, kl_coef=0.0)
    plain = rog.rog_policy_loss(zero, zero, -one, weight=one)
    assert got.stats[0].item() == plain.stats[0].item() == n and torch.equal(got.g_logp, plain.g_logp)
    assert got.stats[1].item() == math.inf
    some = rog.rog_policy_loss(zero[:3], zero[:3], -one[:3], weight=one[:3], ref_logp=q[:3], kl_coef=0.0)
    want = sum(math.expm1(v) - v for v in RATIOS[:3])
    # e^88 as a product with a rounded exponent: 88 u put back, a few roundings left
    assert abs(float(some.stats[1]) - want) <= 2 * 90 * ref.U * want


def test_tokens_that_cancel(gpu):
    """Terms that are exact in binary32 and whose sum is: the sums lose nothing of them, wherever the tokens stand."""
    for n in (4, 5, 1027, 4099, 300001):
        for at in {0, min(1, n - 4), max(0, n // 2 - 2), n - 4}:
            adv = torch.zeros(n, device=gpu)
            adv[at:at + 4] = vec([1e8, 1.0, -1e8, 0.0], gpu)
            same = torch.zeros(n, device=gpu)
            got = rog.rog_policy_loss(same, same, adv, weight=torch.ones(n, device=gpu))
            assert got.stats.tolist() == [-1.0, 0.0, 0.0, 0.0], (n, at)
            assert torch.equal(got.g_logp, -adv)


def test_entropy_and_clip_sums_cancel_too(gpu):
    """Weights of both signs: sum w entropy and sum w [clipped] of exact terms, exactly."""
    w = vec([1e8, 1.0, -1e8, 0.5], gpu)
    one, old = torch.ones(4, device=gpu), torch.zeros(4, device=gpu)
    got = rog.rog_policy_loss(one, old, one, weight=w, entropy=one, clip_high=0.5)
    assert got.stats[2:].tolist() == [1.5, 1.5]


def test_large_weighted_terms_do_not_overflow_on_the_way(gpu):
    adv = vec([3e38, 3e38, -3e38, -3e38, 2.0], gpu)
    same = torch.zeros(5, device=gpu)
    got = rog.rog_policy_loss(same, same, adv, weight=torch.ones(5, device=gpu))
    assert got.stats[0].item() == -2.0
