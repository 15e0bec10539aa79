"""Logits that are masks: blocks of columns, and whole rows, of large values of
either sign, against the formulas without those columns or over them alone; and
logits so large that log2(e) / T times them leaves the binary32 range, which count
as infinite of their sign, in every number of the row alike."""
from __future__ import annotations

import math

import pytest
import torch

from deterministic_collective_movement_amd import rog
from tests import linear_ref as ref

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def huge(gpu, n, x, T):
    """A head whose column 7 has the logit x in every row, the others about 1."""
    h, ws, tokens = ref.head(n, [300], 64, BF16, gpu, sigma=1.0, sure=False)
    h[:, 0] = 1.0
    ws[0][:, 0] = 0
    ws[0][7] = 0
    ws[0][7, 0] = x
    tokens[0], tokens[1:] = 7, 5
    return h, ws, tokens, T


@pytest.mark.parametrize("n", [2, 40, 100, 300])
@pytest.mark.parametrize("x,T", [(3e38, 1.0), (2e38, 0.5), (1e36, 2.0 ** -10)])
def test_large_positive(gpu, n, x, T):
    h, ws, tokens, T = huge(gpu, n, x, T)
    r = rog.rog_linear_logprob(h, ws, tokens, temperature=T)
    assert all(bool(torch.isnan(v).all()) for v in r[:3])
    d = rog.rog_linear_logprob_grad(h, ws, tokens, r.lse, r.entropy, torch.ones(n, device=gpu), temperature=T)
    assert bool(torch.isnan(d.d_hidden).all()) and bool(torch.isnan(d.d_weights[0]).all())


@pytest.mark.parametrize("n", [2, 40, 100, 300])
@pytest.mark.parametrize("x,T", [(-3e38, 1.0), (-2e38, 0.5), (-1e36, 2.0 ** -10)])
def test_large_negative(gpu, n, x, T):
    # a mask by the lowest values: probability 0, and the others are what they are without the column
    h, ws, tokens, T = huge(gpu, n, x, T)
    r = rog.rog_linear_logprob(h, ws, tokens, temperature=T)
    assert float(r.logp[0]) == -math.inf
    keep = torch.arange(300, device=gpu) != 7
    (logp, entropy, lse), (a, b, c) = ref.score64(h[1:], [ws[0][keep]], tokens[1:], T)
    for got, want, tol in zip((r.logp, r.entropy, r.lse), (logp, entropy, lse), (a, b, c)):
        assert bool(((got[1:].double() - want).abs() <= tol).all())
    d = rog.rog_linear_logprob_grad(h, ws, tokens, r.lse, r.entropy, torch.ones(n, device=gpu), temperature=T)
    assert bool(torch.isfinite(d.d_weights[0]).all()) and bool(torch.isfinite(d.d_hidden[1:, 1:]).all())


@pytest.mark.parametrize("n", [2, 100])
@pytest.mark.parametrize("x,T", [(2e38, 1.0), (1e38, 0.5)])
def test_the_largest_that_are_finite(gpu, n, x, T):
    h, ws, tokens, T = huge(gpu, n, x, T)
    r = rog.rog_linear_logprob(h, ws, tokens, temperature=T)
    want = float(ws[0][7, 0]) / T
    assert float(r.logp[0]) == 0 and bool((r.entropy == 0).all())
    assert bool(((r.lse.double() - want).abs() <= 2.0 ** -21 * want).all())
    assert bool((r.logp[1:].double() <= -want * (1 - 2.0 ** -21)).all())


LEVELS = [-1e4, -1e6, -1e9, -1.5e9, -1e10, -1e12, -1e20, -1e30, -1e38]


@pytest.mark.parametrize("n", [3, 40, 100, 300])
@pytest.mark.parametrize("dtype", [BF16, torch.float16])
def test_blocks_of_masked_columns(gpu, n, dtype):
    """Whole leaves and blocks, an end of a shard and single columns: probability 0, whatever masks them."""
    T = 0.9
    h, ws, tokens = ref.head(n, [512, 77], 64, dtype, gpu, sigma=2.0, sure=False)
    h[:, 0] = 1.0
    masked = torch.zeros(589, dtype=torch.bool, device=gpu)
    masked[128:256] = masked[300:400] = masked[410] = masked[480:512] = masked[560:] = True
    part = [masked[:512], masked[512:]]
    tokens = torch.nonzero(~masked)[:, 0][tokens % int((~masked).sum())]
    g = torch.randn(n, device=gpu) * (16 if dtype is torch.float16 else 1)
    place = (~masked).cumsum(0) - 1
    kept = [w[~m] for w, m in zip(ws, part)]
    for c in LEVELS:
        if abs(c) > torch.finfo(dtype).max:
            continue
        for w, m in zip(ws, part):
            w[m, 0] = c
        r = rog.rog_linear_logprob(h, ws, tokens, temperature=T)
        want, tol = ref.score64(h, kept, place[tokens], T)
        for got, w, t in zip(r[:3], want, tol):
            assert bool(((got.double() - w).abs() <= t).all()), c
        d = rog.rog_linear_logprob_grad(h, ws, tokens, r.lse, r.entropy, g, 0.1 * g, temperature=T)
        (dh, dw), (dh_tol, dw_tol) = ref.grad_head64(h, kept, place[tokens], T, r.lse, r.entropy, g, 0.1 * g)
        assert bool(((d.d_hidden.double() - dh).abs() <= dh_tol).all()), c
        for got, m, w, t in zip(d.d_weights, part, dw, dw_tol):
            assert bool(((got[~m].double() - w).abs() <= t).all()) and bool((got[m] == 0).all()), c


LARGE = LEVELS + [2e4, 1e6, 1e9, 1.5e9, 1e10, 1e20, 1e38]


def uniform(gpu, n, T, c):
    """A head whose columns are all at c (c < 0), or 96 of them over others near 0: (states, weights, tokens, those columns, c / T)."""
    h, ws, _ = ref.head(n, [512], 64, BF16, gpu, sigma=1.0, sure=False)
    h[:, 0] = 1.0
    ws[0][:, 0] = 0
    top = torch.arange(512, device=gpu) if c < 0 else torch.arange(384, 480, device=gpu)
    ws[0][top] = 0
    ws[0][top, 0] = c
    return h, ws, top[torch.arange(n, device=gpu) * 7 % len(top)], top, float(ws[0][top[0], 0]) / T


@pytest.mark.parametrize("n", [3, 40, 100, 300])
@pytest.mark.parametrize("T", [1.0, 0.7, 3.0])
@pytest.mark.parametrize("c", LARGE)
def test_rows_that_are_uniform_over_large_logits(gpu, n, T, c):
    h, ws, tokens, top, x = uniform(gpu, n, T, c)
    k = len(top)
    r = rog.rog_linear_logprob(h, ws, tokens, temperature=T)
    # three roundings of a number of x log2(e) and as many of lse, and those of a logarithm and its sums
    assert bool(((r.lse.double() - x - math.log(k)).abs() <= 2.0 ** -21 * abs(x) + 1e-5).all())
    assert bool(((r.logp.double() + math.log(k)).abs() <= 2e-6).all())
    assert bool(((r.entropy.double() - math.log(k)).abs() <= 2e-5).all())


@pytest.mark.parametrize("n", [3, 40, 100, 300])
@pytest.mark.parametrize("T", [1.0, 0.7, 3.0])
@pytest.mark.parametrize("c", LARGE)
def test_gradient_of_rows_that_are_uniform_over_large_logits(gpu, n, T, c):
    """p is 1 / k at each of the k, whatever lse's rounding leaves open."""
    h, ws, tokens, top, _ = uniform(gpu, n, T, c)
    r = rog.rog_linear_logprob(h, ws, tokens, temperature=T)
    g = torch.randn(n, device=gpu)
    d = rog.rog_linear_logprob_grad(h, ws, tokens, r.lse, r.entropy, g, 0.3 * g, temperature=T)
    G = torch.zeros(n, 512, dtype=torch.float64, device=gpu)
    G[:, top] = -1.0 / len(top)
    G[torch.arange(n, device=gpu), tokens] += 1.0
    G *= g.double()[:, None] / T
    want, size = G.t() @ h.double(), G.abs().t() @ h.double().abs()
    # G rounded once, the sum once; p to lse's rounding below 2^14 / log2(e) and to that of e^{-H} above, log p + H likewise
    tol = 2.0 ** -8 * (want.abs() + size) + 0.004 * size + 1e-6
    assert bool(((d.d_weights[0].double() - want).abs() <= tol).all())
    # the top columns' other weights are 0, and G is 0 outside; element 0 is a sum of terms of up to |g| |c| / T, which
    # pass the binary32 range (3.4e38) where c is 1e38 and |g| / T above 3.4
    assert bool((d.d_hidden[:, 1:] == 0).all()) and (abs(c) > 1e37 or bool(torch.isfinite(d.d_hidden).all()))


@pytest.mark.parametrize("n", [3, 40, 100, 300])
@pytest.mark.parametrize("c", [64.0, 1024.0, 8192.0, 2.0 ** 14, 2.0 ** 15, -2.0 ** 15, 2.0 ** 17, -2.0 ** 18, 2.0 ** 20])
def test_gradient_of_rows_of_near_values(gpu, n, c):
    """Values half an integer apart, far from zero: what one binary32 lse leaves open, twice at most."""
    V = 515
    h = torch.zeros(n, 64, dtype=BF16, device=gpu)
    w = torch.zeros(V, 64, dtype=BF16, device=gpu)
    h[:, 0] = 1.0
    w[:, 0] = c
    h[:, 1] = torch.arange(n, device=gpu) % 4 + 1.0
    w[:, 1] = torch.arange(V, device=gpu) * 5 % 7 * 0.5             # every logit is exact in binary32
    h[:, 2:] = torch.randn(n, 62, device=gpu)                       # over weights of 0: for the weights' gradients alone
    tokens = torch.arange(n, device=gpu) * 11 % V
    x = h[:, :2].double() @ w[:, :2].double().t()
    r = rog.rog_linear_logprob(h, [w], tokens)
    lse = torch.logsumexp(x, 1)
    p, g, gh = torch.softmax(x, 1), torch.randn(n, device=gpu), 0.3 * torch.randn(n, device=gpu)
    lp = torch.log_softmax(x, 1)
    H = -(p * lp).sum(1)
    assert bool(((r.logp.double() - lp[torch.arange(n, device=gpu), tokens]).abs() <= 1e-5).all())
    assert bool(((r.entropy.double() - H).abs() <= 3e-5).all()) and bool(((r.lse.double() - lse).abs() <= 2.0 ** -22 * lse.abs() + 1e-5).all())
    d = rog.rog_linear_logprob_grad(h, [w], tokens, r.lse, r.entropy, g, gh)
    G = -g.double()[:, None] * p - gh.double()[:, None] * p * (lp + H[:, None])
    G[torch.arange(n, device=gpu), tokens] += g.double()
    left = 2.0 ** -20 * lse.abs()[:, None] + 1e-4                   # of log p
    a = g.double().abs()[:, None] + gh.double().abs()[:, None] * (lp.abs() + H[:, None] + 1)
    tol = p * torch.expm1(left) * a * (2 + left)
    tol = tol + ref.HALF[BF16] * (G.abs() + tol)
    want, size = G.t() @ h.double(), h.double().abs()
    tol = tol.t() @ size + (n + 64) * 2 * 2.0 ** -24 * (G.abs().t() @ size)
    assert bool(((d.d_weights[0].double() - want).abs() <= tol + ref.HALF[BF16] * (want.abs() + tol)).all())
