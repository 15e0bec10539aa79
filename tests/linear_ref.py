"""Plain 64-bit forms of the policy head's products, and the error that an
evaluation with binary32 sums may have.  Written from the definitions in
include/rog.h; shares no code with the library."""
from __future__ import annotations

import math

import torch

from tests.head_ref import U, grad64, logprob64

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step, relative
LEAST = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}        # half a subnormal step


def head(n, widths, dim, dtype, dev, seed=0, sigma=2.5, extra=0, sure=True, pad=0.0):
    """States, weight shards and tokens: logits of about sigma, a third of the rows sure of their token."""
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed * 7919 + n * 31 + sum(widths) + dim)
    ws = []
    for w in widths:
        full = torch.randn(w, dim + extra, generator=gen, device=dev) * (sigma / math.sqrt(dim))
        ws.append(full.to(dtype)[:, :dim])
    V = sum(widths)
    tokens = torch.randint(0, max(V, 1), (n,), generator=gen, device=dev)
    h = torch.randn(n, dim + extra, generator=gen, device=dev)
    if sure and V:
        at = torch.arange(0, n, 3, device=dev)
        h[at, :dim] += 2.5 * torch.cat([w.float() for w in ws])[tokens[at]]
    h = h.to(dtype)[:, :dim]
    if pad:
        tokens[torch.rand(n, generator=gen, device=dev) < pad] = -1
    return h, ws, tokens


def logits64(h, ws):
    """(logits in float64, the error of each with binary32 sums): products of two
    elements are exact, each of at most dim + 1 additions errs by at most a step
    (2 U: a matrix unit may cut instead of rounding) of what the partial sum can be."""
    W = torch.cat([w.double() for w in ws])
    x = h.double() @ W.t()
    err = (h.shape[1] + 1) * 2 * U * (h.double().abs() @ W.abs().t())
    return x, err


def score64(h, ws, tokens, T):
    """((logp, entropy, lse), their tolerances)."""
    x, err = logits64(h, ws)
    logp, entropy, lse, _, _ = logprob64(x, tokens, T, 0)
    z = (x / T).abs()
    zmax = z.amax(1) if x.shape[1] else z.new_zeros(z.shape[0])
    ex = err.amax(1) / T if x.shape[1] else zmax
    # logits off by ex move lse by at most ex and a log probability by twice that; the
    # statistics as in head_ref.logprob_tol (at most 60 additions and joins a term)
    a = 2 * ex + U * (8 * zmax + 96)
    return (logp, entropy, lse), (a, a * (2 + 2 * entropy.abs()), a)


def grad_head64(h, ws, tokens, T, lse, entropy, g, gh):
    """((d_hidden, [d_weights]), tolerances), in 64 bits."""
    dtype = h.dtype
    x, err = logits64(h, ws)
    V = x.shape[1]
    G, tol = grad64(x, tokens, T, lse.double(), entropy.double(), g.double(), gh.double())
    read = (tokens >= 0)[:, None]
    p = torch.softmax(x / T, 1)
    lp = torch.log_softmax(x / T, 1)
    # p moves by a factor of e^(2 err / T) and log p by as much
    move = 2 * err.amax(1, keepdim=True) / T
    a = (g.double().abs()[:, None] + gh.double().abs()[:, None] * (lp.abs() + entropy.double()[:, None].abs() + 2)) / T
    tol = torch.where(read, tol + 2 * move * p * a, 0.0)
    # rounded to the states' type; binary16 after a power of two of at least 2^13 / the largest that |G| can be
    tol = tol + HALF[dtype] * (G.abs() + tol)
    if dtype is torch.float16:
        most = ((g.double().abs() + 22 * gh.double().abs())[tokens >= 0].amax() if (tokens >= 0).any() else torch.zeros((), device=h.device)) / T
        tol = tol + 2.0 ** -25 * most / 2.0 ** 13
    tol = torch.where(read, tol, 0.0)
    W, H = torch.cat([w.double() for w in ws]), torch.where(read, h.double(), 0.0)
    n = h.shape[0]
    dh, dw = G @ W, G.t() @ H
    # sums of V (and of n) products in binary32
    dh_tol = tol @ W.abs() + (V + 64) * 2 * U * (G.abs() @ W.abs())
    dw_tol = tol.t() @ H.abs() + (n + 64) * 2 * U * (G.abs().t() @ H.abs())
    dh_tol = dh_tol + HALF[dtype] * (dh.abs() + dh_tol) + LEAST[dtype]
    dw_tol = dw_tol + HALF[dtype] * (dw.abs() + dw_tol) + LEAST[dtype]
    sizes = [w.shape[0] for w in ws]
    return (dh, list(dw.split(sizes))), (dh_tol, list(dw_tol.split(sizes)))


def quantize_cpu(x):
    """(q, scale) by the definition, with the processor's binary32 division."""
    x = x.float().cpu()
    most = x.abs().amax(1)
    s = torch.clamp_min(most / torch.full_like(most, 127.0), 2.0 ** -126)
    q = torch.round(x / s[:, None])
    bad = ~torch.isfinite(x).all(1)
    s[bad] = math.nan
    q[bad] = 0
    return q.to(torch.int8), s


def linear_i8_cpu(q, s, w, r, dtype):
    """The definition, step by step: an exact sum, its binary32, two products, one rounding."""
    total = q.cpu().double() @ w.cpu().double().t()      # below 2^53: exact
    return ((total.float() * s.cpu()[:, None]) * r.cpu()).to(dtype)
