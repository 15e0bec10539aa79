"""Plain 64-bit forms of the vocabulary-side operators, and the error that a
binary32 evaluation of them may have.  Written from the definitions in
include/rog.h; shares no code with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

U = 2.0 ** -24          # unit roundoff of binary32


def rows64(shards):
    return torch.cat([s.double() for s in shards], 1)


def logprob64(x, tokens, T, k):
    """(logp, entropy, lse, top_logp, top_ids) of rows x (float64, any device)."""
    n, V = x.shape
    dev = x.device
    z = x / T
    neg = torch.full((n,), -math.inf, dtype=torch.float64, device=dev)
    if V == 0:
        z = torch.full((n, 1), -math.inf, dtype=torch.float64, device=dev)
    m = z.amax(1)
    bad = torch.isnan(z).any(1) | torch.isposinf(m)
    empty = torch.isneginf(m)
    mm = torch.where(torch.isfinite(m), m, 0.0)
    y = z - mm[:, None]
    e = torch.exp(y)
    S = e.sum(1)
    L = torch.log(S)
    p = e / S[:, None]
    lp = y - L[:, None]
    lse = torch.where(empty, neg, mm + L)
    entropy = torch.where(empty, 0.0, -torch.where(p > 0, p * lp, 0.0).sum(1))
    lp = torch.where(empty[:, None], neg[:, None], lp)
    nan = torch.full_like(neg, math.nan)
    if tokens is None:
        logp = None
        off = torch.zeros(n, dtype=torch.bool, device=dev)
    else:
        off = tokens < 0
        over = tokens >= V
        logp = lp.gather(1, tokens.clamp(0, max(0, V - 1))[:, None])[:, 0]
        logp = torch.where(bad | over, nan, logp)
        logp = torch.where(off, 0.0, logp)
    lse = torch.where(off, 0.0, torch.where(bad, nan, lse))
    entropy = torch.where(off, 0.0, torch.where(bad, nan, entropy))
    top_logp = torch.full((n, k), -math.inf, dtype=torch.float64, device=dev)
    top_ids = torch.full((n, k), -1, dtype=torch.int64, device=dev)
    if k and V:
        order = torch.sort(torch.where(torch.isnan(x), -math.inf, x) + 0.0, dim=1, descending=True, stable=True)
        kk = min(k, V)
        ids = order.indices[:, :kk]
        none = torch.isneginf(order.values[:, :kk])
        top_ids[:, :kk] = torch.where(none, -1, ids)
        top_logp[:, :kk] = torch.where(none, -math.inf, lp.gather(1, ids))
    top_ids = torch.where((bad | off)[:, None], -1, top_ids)
    top_logp = torch.where(off[:, None], 0.0, torch.where(bad[:, None], nan[:, None], top_logp))
    return logp, entropy, lse, top_logp, top_ids


def scale_of(x, T):
    """Per row, the largest finite |z| a rounding error scales with; masks of the
    lowest finite values have probability 0 and do not count."""
    z = (x / T).abs()
    z = torch.where(torch.isfinite(z) & (z < 1e20), z, 0.0)
    return z.amax(1) if z.shape[1] else z.new_zeros(z.shape[0])


def logprob_tol(x, T, entropy):
    """(tolerance of log probabilities and lse, of the entropy), absolute, per row.

    z is a product with a rounded scale and one rounding (2 u |z|), its reference
    is rounded alike (another 2 u |z|); every term of the sums has one exponential
    (2 u) and at most 60 additions and rescalings of binary32 above it (each u,
    all terms of one sign); lse and the difference round once more (2 u |z|).
    The entropy's terms weigh these errors by |log p| on top."""
    zmax = scale_of(x, T)
    a = U * (6 * zmax + 64)
    return a, a * (2 + 2 * entropy.abs())


def grad64(x, tokens, T, lse, entropy, g, gh):
    """d (sum g logp + gh entropy) / d x, from its own p (not from lse)."""
    n, V = x.shape
    z = x / T
    empty = torch.isneginf(z).all(1)
    z = torch.where(empty[:, None], 0.0, z)
    lp = torch.log_softmax(z, 1)
    p = torch.exp(lp)
    hit = torch.zeros_like(p)
    inside = (tokens >= 0) & (tokens < V)
    hit[torch.arange(n, device=x.device)[inside], tokens[inside]] = 1.0
    H = -torch.where(p > 0, p * lp, 0.0).sum(1)
    d = g[:, None] * (hit - p) - gh[:, None] * torch.where(p > 0, p * (lp + H[:, None]), 0.0)
    d = d / T
    d[tokens >= V] = math.nan
    d[(tokens < 0) | empty] = 0.0
    # what a binary32 p may be off by, carried through; lse and entropy come rounded to binary32
    zmax = scale_of(x, T)
    rel = U * (8 * zmax + 64)[:, None]
    lp0 = torch.where(p > 0, lp, 0.0)
    a = (g[:, None].abs() + gh[:, None].abs() * (lp0.abs() + H[:, None].abs() + 1)) / T
    tol = rel * p * a * (2 + lp0.abs()) + 4 * U * hit * g[:, None].abs() / T + 1e-37
    return d, torch.where(torch.isfinite(tol), tol, 0.0)


ROUND = {torch.float32: (2.0 ** -24, 2.0 ** -149), torch.bfloat16: (2.0 ** -8, 2.0 ** -134),
         torch.float16: (2.0 ** -11, 2.0 ** -25)}


def policy64(logp, old, adv, w, ref, ent, lo, hi, kl_coef, ent_coef, scale):
    """numpy float32 inputs -> (stats, g_logp, g_entropy) and their tolerances."""
    n = len(logp)
    d = (logp - old).astype(np.float64)               # binary32 differences by definition
    q = (ref - logp).astype(np.float64) if ref is not None else np.zeros(n)
    a = adv.astype(np.float64)
    W = w.astype(np.float64) if w is not None else np.full(n, float(np.float32(1.0 / n)) if n else 0.0)
    H = ent.astype(np.float64) if ent is not None else np.zeros(n)
    b = kl_coef if ref is not None else 0.0
    over, under = (a > 0) & (d > hi), (a < 0) & (d < lo)
    with np.errstate(all="ignore"):
        r = np.exp(np.where(over, hi, np.where(under, lo, d)))
        kl = np.expm1(q) - q
        l = -a * r + b * kl - ent_coef * H
        slope = np.where(over | under, 0.0, -a * np.exp(d)) - b * np.expm1(q)
        kept = W != 0
        zero = lambda v: np.where(kept, W * v, 0.0)  # noqa: E731
        c = (over | under).astype(np.float64)
        stats = np.array([math.fsum(zero(v)) for v in (l, kl, H, c)])
        g = scale * zero(slope)
        gh = -scale * zero(np.full(n, ent_coef))
        # an exponential to 2 u, its argument exact, a handful of roundings; the sums are binary64
        kl_err = U * (8 * kl + 4 * np.minimum(1.0, np.abs(q)) * (np.abs(q) > 0.5))
        size = 8 * U * (np.abs(a) * r + np.abs(ent_coef * H) + b * kl) + abs(b) * kl_err
        stat_tol = np.array([math.fsum(zero(size)), math.fsum(zero(kl_err)), U * abs(stats[2]), U * abs(stats[3])])
        stat_tol = np.abs(stat_tol) + 2 * U * np.abs(stats) + 1e-38
        g_tol = 8 * U * abs(scale) * np.abs(zero(np.abs(a) * r + abs(b) * np.abs(np.expm1(q)) * 2)) + 1e-38
        gh_tol = 4 * U * np.abs(gh) + 1e-38
    return (stats, g, gh), (stat_tol, g_tol, gh_tol)
