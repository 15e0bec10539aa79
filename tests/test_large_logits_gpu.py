"""Log-sum-exp, entropy and gradient of rows whose logits are all large, against
the formulas in 64 bits.  lse is one binary32 number, so at |lse| = 2^e it
leaves 2^(e - 24) of every log p open; what a kernel adds to that is bounded by
a constant that does not grow with |lse|, and rows that are uniform over their
largest logits (fully masked ones, ones that are sure of a token) hold to that
constant alone."""
from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from deterministic_collective_movement_amd import rog
from tests import head_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
IDS = {BF16: "bf16", F16: "f16", F32: "f32"}


def left_open(lse):
    """What binary32 sums, exponentials and logarithms may leave in log p and in
    the entropy: 256 roundings of 1 (an exponent below 64, its product with
    log2 e, a logarithm below 64, at most 60 additions above a term); and as the
    sums are held against a reference that is itself rounded, by up to half a unit
    of |lse| log2 e and 32 at the most, 64 roundings of twice that."""
    return ref.U * (256 + 64 * (lse.abs() * (1.45 * 2.0 ** -23)).clamp(max=64.0))


def half_ulp(x):
    """Half a binary32 unit in the last place of x, as float64."""
    return torch.from_numpy(np.spacing(np.abs(x.double().cpu().numpy()).astype(np.float32)).astype(np.float64) / 2).to(x.device)


def temperature(T):
    return float(np.float32(T))      # the interface takes it in binary32


def exact(x, T):
    """(lse, log p, entropy) of rows x in 64 bits; the largest logit is taken off before the division."""
    x = x.double()
    m = x.amax(1, keepdim=True)
    y = (x - m) / T
    S = torch.exp(y).sum(1)
    lp = y - torch.log(S)[:, None]
    p = torch.exp(lp)
    return m[:, 0] / T + torch.log(S), lp, -torch.where(p > 0, p * lp, 0.0).sum(1)


def check(x, T, tokens, uniform):
    T = temperature(T)
    rows, V = x.shape
    r = rog.rog_logprob([x], tokens, temperature=T)
    lse, lp, H = exact(x, T)
    open_ = left_open(lse)
    # 1 / T is held to 2^-48 of itself: a 2^-22 of half a unit
    assert bool(((r.lse.double() - lse).abs() <= half_ulp(lse) * (1 + 2.0 ** -20) + open_).all()), (r.lse.tolist(), lse.tolist())
    assert bool(((r.entropy.double() - H).abs() <= open_ * (1 + H)).all()), (r.entropy.tolist(), H.tolist())
    # logp comes from the sums: nothing of lse's rounding, four roundings of its own size
    logp = lp.gather(1, tokens[:, None])[:, 0]
    ok = (r.logp.double() == logp) | ((r.logp.double() - logp).abs() <= open_ + 4 * ref.U * logp.abs())
    assert bool(ok.all()), (r.logp[~ok].tolist(), logp[~ok].tolist())
    gen = torch.Generator(device=x.device)
    gen.manual_seed(V)
    g, h = (torch.randn(rows, generator=gen, device=x.device) for _ in range(2))
    # one binary32 lse: a rounding of log p, and as much again where log p is taken to be -H within it
    left = open_ + (torch.zeros_like(H) if uniform else 2.1 * half_ulp(lse))
    rel, least = ref.ROUND[x.dtype]
    p = torch.exp(lp)
    hit = torch.zeros_like(p)
    hit[torch.arange(rows, device=x.device), tokens] = 1.0
    for gh in (None, h):
        got = rog.rog_logprob_grad([x], tokens, r.lse, r.entropy, g, gh, temperature=T)[0].double()
        hd = torch.zeros(rows, 1, device=x.device, dtype=torch.float64) if gh is None else h.double()[:, None]
        gd = g.double()[:, None]
        surprise = torch.where(p > 0, lp + H[:, None], 0.0)
        want = (gd * (hit - p) - hd * p * surprise) / T
        # p off by a factor e^left, log p by left, H as above; eight roundings of the largest terms
        grow = torch.expm1(left)[:, None]
        tol = (p * grow * (gd.abs() + hd.abs() * surprise.abs()) + p * (1 + grow) * hd.abs() * (left + open_ * (1 + H))[:, None]
               + 8 * ref.U * (gd.abs() * (hit + p) + hd.abs() * p * (1 + H[:, None]))) / T + 1e-37
        err = (got - want).abs()
        ok = err <= tol + rel * (want.abs() + tol) + least
        bad = [(int(i), int(j), float(got[i, j]), float(want[i, j]), float(r.lse[i])) for i, j in torch.nonzero(~ok)[:4].tolist()]
        assert bool(ok.all()), (T, gh is not None, bad)
    if uniform:
        # with g = 1 the probabilities stand in the gradient: they sum to 1, to the outputs' own rounding
        one = rog.rog_logprob_grad([x], tokens, r.lse, r.entropy, torch.ones(rows, device=x.device), temperature=T)[0].double()
        total = (hit - T * one).sum(1)
        assert bool(((total - 1).abs() <= 2 * open_ + 2 * rel + 8 * ref.U + V * T * least).all()), total.tolist()


LEVELS = [-1e2, -1e3, -1e4, -65504.0, -1e6, -1e8, -5e8, 3e4, 1e6, 3.7e7, 5.37e8, -1e9, 2e9]
TEMPERATURES = [1.0, 0.7, 0.3, 1.9, 8.0, 0.01, 700.0]


@pytest.mark.parametrize("T", TEMPERATURES)
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=IDS.get)
@pytest.mark.parametrize("V", [5, 3001, 50257])
def test_uniform_rows(gpu, V, dtype, T):
    """Fully masked rows, rows that are sure of one token, rows that are uniform over some columns."""
    levels = [c for c in LEVELS if abs(c) <= torch.finfo(dtype).max]
    x = torch.empty(4 * len(levels), V, dtype=dtype, device=gpu)
    tokens = torch.arange(len(x), device=gpu) * 7 % V
    for i, c in enumerate(levels):
        far = -math.inf if c < 0 else 0.0
        x[4 * i] = c                                             # masked with one value, all of it
        x[4 * i + 1] = far                                       # sure of its token
        x[4 * i + 1, tokens[4 * i + 1]] = c
        x[4 * i + 2] = c                                         # sure of another
        x[4 * i + 2] -= 4096 * max(1.0, T) if abs(c) < 1e4 else abs(c) / 4 * max(1.0, T / 20)
        x[4 * i + 2].clamp_(min=torch.finfo(dtype).min)
        x[4 * i + 2, V - 1] = c
        x[4 * i + 3] = far                                       # a third of the columns left
        x[4 * i + 3, ::3] = c
    # rows whose columns lie too near for a temperature to be uniform over the largest are another test's
    _, lp, _ = exact(x, temperature(T))
    best = lp.amax(1, keepdim=True)
    keep = ((lp == best) | (lp < best - 60)).all(1)
    assert int(keep.sum()) >= 2 * len(levels)
    check(x[keep], T, tokens[keep], True)


@pytest.mark.parametrize("T", TEMPERATURES[:5])
@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=IDS.get)
def test_rows_of_near_values(gpu, dtype, T):
    """A few neighbouring values far from zero: what one binary32 lse leaves open, and no more."""
    V = 4003
    steps = {BF16: [-256.0, -1000.0, 500.0], F16: [-2048.0, -65504.0, 8000.0], F32: [-1e4, -1e5, -1e6, 3e6, -1e7]}[dtype]
    x = torch.empty(len(steps), V, dtype=dtype, device=gpu)
    for i, c in enumerate(steps):
        step = float(torch.tensor(abs(c)).to(dtype)) * {BF16: 2.0 ** -7, F16: 2.0 ** -10, F32: 2.0 ** -22}[dtype]
        x[i] = (c + max(step, 0.25) * torch.arange(V, device=gpu).remainder(5).double()).to(dtype)
    check(x, T, torch.arange(len(steps), device=gpu) * 11 % V, False)


@pytest.mark.parametrize("T", [1.0, 0.7, 3.0])
def test_around_the_extreme_rows(gpu, T):
    """|lse| on both sides of 2^30 ln 2, where a row counts as uniform without its logits' differences."""
    edge = 2.0 ** 30 * math.log(2.0) * temperature(T)
    V = 700
    at = [edge + k * 64 * temperature(T) for k in (-40, -6, -5, -4, -3, -2, -1, 0, 1, 2, 3, 4, 5, 6, 40)]
    x = torch.full((2 * len(at), V), -math.inf, device=gpu)
    for i, c in enumerate(at):
        x[2 * i, ::2] = c
        x[2 * i + 1] = -c
    check(x, T, torch.arange(len(x), device=gpu) * 4 % V, True)
