"""The vocabulary-side operators as a user's program calls them: cases, inputs and plain forms.

Three operators of a policy head that is held as W vocabulary shards in rank
order: ``logprob`` (log probability of a given token per row, entropy,
log-sum-exp, the K best alternatives), ``grad`` (its gradient in every shard)
and ``loss`` (clipped policy loss over ragged token weights, with its
gradient).  ``run`` computes them in plain torch operations in 32 bits, or,
where ``own`` is true, through the library's entry points.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f16": 2, "f32": 4}


def _head(op, name, rows, vocab, dtype, W=1, top_k=0, T=1.0, pad=0.0, masked=0.0, extra=0):
    """A case over logits: rows x vocab in W shards; pad: share of rows that are
    not scored; masked: share of the vocabulary at -inf; extra: unused columns
    behind each shard's row (a row stride larger than the width)."""
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "W": W, "top_k": top_k,
            "T": T, "pad": pad, "masked": masked, "extra": extra}


def _loss(name, n, ref, entropy, kept):
    """A case over n tokens, of which the share `kept` carries weight."""
    return {"name": name, "op": "loss", "n": n, "ref": ref, "entropy": entropy, "kept": kept}


def listed():
    return [
        # one new token of one request, with a few alternatives: latency
        _head("logprob", "logprob 1x131072 k5", 1, 131072, "bf16", top_k=5),
        # a decode batch over eight ranks' shards, twenty alternatives, grammar masks that leave some rows nothing
        _head("logprob", "logprob 64x131072 w8 k20 masked", 64, 131072, "bf16", W=8, top_k=20, T=0.8, masked=0.5),
        # a prompt batch scored with alternatives in f32 over two uneven shards
        _head("logprob", "logprob 509x32003 f32 w2 k8", 509, 32003, "f32", W=2, top_k=8),
        # many rows of a short vocabulary (the library's own 8627 x 8192 shape)
        _head("logprob", "logprob 8627x8192", 8627, 8192, "bf16"),
        # odd vocabulary, every row of another alignment, some rows padding
        _head("logprob", "logprob 1021x50257 f16", 1021, 50257, "f16", T=0.7, pad=0.125),
        # a training step's rows over eight ranks' shards
        _head("logprob", "logprob 4096x131072 w8", 4096, 131072, "bf16", W=8),
        # gradients: a small batch in f32, an odd vocabulary with padding rows, a training step
        _head("grad", "grad 33x32003 f32", 33, 32003, "f32", W=2),
        _head("grad", "grad 1021x50257 f16", 1021, 50257, "f16", T=0.7, pad=0.125, extra=47),
        _head("grad", "grad 4096x131072 w8", 4096, 131072, "bf16", W=8),
        # the loss of a small batch, an ordinary one, a large one; the small one without reference or entropy
        _loss("loss 1021", 1021, False, False, 0.7),
        _loss("loss 131072", 131072, True, True, 0.6),
        _loss("loss 4194307", 4194307, True, True, 0.8),
    ]


MOST_BYTES = 4096 * 131072 * 2


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["logprob", "logprob", "grad", "loss"])
    if op == "loss":
        case = _loss("", _log_uniform(rng, 300, 4194307), rng.random() < 0.7, rng.random() < 0.7,
                     round(rng.uniform(0.3, 1.0), 3))
    else:
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        vocab = _log_uniform(rng, 1000, 131072)
        rows = _log_uniform(rng, 1, min(16384, MOST_BYTES // (ESIZE[dtype] * vocab)))
        case = _head(op, "", rows, vocab, dtype, W=rng.choice([1, 1, 2, 4, 8]),
                     top_k=rng.choice([0, 0, 1, rng.randint(2, 32)]) if op == "logprob" else 0,
                     T=rng.choice([1.0, 1.0, round(rng.uniform(0.3, 1.6), 2)]),
                     pad=rng.choice([0.0, 0.0, 0.125]), masked=rng.choice([0.0, 0.0, 0.5]) if op == "logprob" else 0.0,
                     extra=rng.choice([0, 0, rng.randint(1, 64)]))
    del case["name"]
    return case


def _widths(vocab, W):
    """W shard widths in rank order: equal where W divides the vocabulary, the last ones a column shorter where not."""
    return [vocab // W + (1 if r < vocab % W else 0) for r in range(W)]


def _padded_rows(case):
    return int(case["rows"] * case["pad"])


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _make_head(case, gen, dev):
    rows, vocab, dtype = case["rows"], case["vocab"], DTYPES[case["dtype"]]
    tokens = torch.randint(0, vocab, (rows,), generator=gen, device=dev)
    shards = []
    for width in _widths(vocab, case["W"]):
        x = torch.randn(rows, width + case["extra"], generator=gen, device=dev, dtype=dtype)
        x.mul_(2.5)
        shards.append(x[:, :width])
    # a third of the rows are sure of their token, as a trained policy is of most
    lo = 0
    for x in shards:
        at = torch.nonzero((tokens >= lo) & (tokens < lo + x.shape[1]) & (torch.arange(rows, device=dev) % 3 == 0))[:, 0]
        x[at, tokens[at] - lo] = 16.0
        lo += x.shape[1]
    if case["masked"]:
        for x in shards:
            x.masked_fill_(torch.rand(x.shape, generator=gen, device=dev) < case["masked"], -math.inf)
            x[rows // 2::37] = -math.inf  # rows that the mask leaves nothing
    pad = torch.randperm(rows, generator=gen, device=dev)[:_padded_rows(case)]
    tokens[pad] = -1
    return shards, tokens


def _make_loss(case, gen, dev):
    n = case["n"]
    logp = -torch.empty(n, device=dev).exponential_(1.0, generator=gen)
    old = logp + 0.15 * torch.randn(n, generator=gen, device=dev)
    ref = logp + 0.2 * torch.randn(n, generator=gen, device=dev) if case["ref"] else None
    entropy = torch.empty(n, device=dev).exponential_(1.5, generator=gen) if case["entropy"] else None
    adv = torch.randn(n, generator=gen, device=dev)
    weight = (torch.rand(n, generator=gen, device=dev) < case["kept"]).float()
    weight /= weight.sum().clamp_min(1.0)
    return logp, old, adv, weight, ref, entropy


CLIP_LOW, CLIP_HIGH, KL_COEF, ENTROPY_COEF = 0.2, 0.28, 0.05, 0.01


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    st = {"op": case["op"], "case": case}
    if case["op"] == "loss":
        st["in"] = _make_loss(case, gen, dev)
        n = case["n"]
        st["out"] = (torch.empty(4, device=dev), torch.empty(n, device=dev),
                     torch.empty(n, device=dev) if case["entropy"] else None)
        return st
    shards, tokens = _make_head(case, gen, dev)
    rows = case["rows"]
    st["shards"], st["tokens"] = shards, tokens
    if case["op"] == "logprob":
        k = case["top_k"]
        st["out"] = (torch.empty(rows, device=dev), torch.empty(rows, device=dev), torch.empty(rows, device=dev),
                     torch.empty(rows, k, device=dev) if k else None,
                     torch.empty(rows, k, device=dev, dtype=torch.int64) if k else None)
        return st
    # what the forward pass has left, and the loss's gradients
    st["lse"], st["entropy"] = _lse_entropy(case, shards, tokens)
    st["g_logp"] = torch.randn(rows, generator=gen, device=dev) / rows
    st["g_entropy"] = 0.02 * torch.randn(rows, generator=gen, device=dev) / rows
    st["out"] = [torch.empty(rows, x.shape[1], dtype=x.dtype, device=dev) for x in shards]
    return st


def _row_chunks(rows, vocab, most=1 << 27):
    step = max(1, most // vocab)
    return [(a, min(rows, a + step)) for a in range(0, rows, step)]


def _lse_entropy(case, shards, tokens):
    """log-sum-exp and entropy per row, in 64 bits, rounded to 32: zero where the row is not scored."""
    lse, ent = [], []
    for a, b in _row_chunks(case["rows"], case["vocab"]):
        z = torch.cat([x[a:b] for x in shards], 1).double() / case["T"]
        l = torch.logsumexp(z, 1)
        ent.append(l - (torch.exp(z - l[:, None]) * z).sum(1))
        lse.append(l)
    scored = tokens >= 0
    return (torch.where(scored, torch.cat(lse), 0.0).float(), torch.where(scored, torch.cat(ent), 0.0).float())


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(st):
    if own:
        return _run_own(st)
    return {"logprob": _plain_logprob, "grad": _plain_grad, "loss": _plain_loss}[st["op"]](st)


def _run_own(st):
    from deterministic_collective_movement_amd import rog
    case = st["case"]
    if st["op"] == "logprob":
        r = rog.rog_logprob(st["shards"], st["tokens"], top_k=case["top_k"], temperature=case["T"], out=st["out"])
        return {"logp": r.logp, "entropy": r.entropy, "lse": r.lse, "top_logp": r.top_logp, "top_ids": r.top_ids}
    if st["op"] == "grad":
        return rog.rog_logprob_grad(st["shards"], st["tokens"], st["lse"], st["entropy"], st["g_logp"],
                                    st["g_entropy"], temperature=case["T"], out=st["out"])
    logp, old, adv, weight, ref, entropy = st["in"]
    r = rog.rog_policy_loss(logp, old, adv, weight=weight, ref_logp=ref, entropy=entropy, clip_low=CLIP_LOW,
                            clip_high=CLIP_HIGH, kl_coef=KL_COEF if case["ref"] else 0.0,
                            entropy_coef=ENTROPY_COEF if case["entropy"] else 0.0, out=st["out"])
    return {"stats": r.stats, "g_logp": r.g_logp, "g_entropy": r.g_entropy}


def _plain_logprob(st):
    case, tokens = st["case"], st["tokens"]
    x = torch.cat([s.float() for s in st["shards"]], 1)
    z = x / case["T"]
    m = z.amax(1, keepdim=True)
    empty = torch.isneginf(m)[:, 0]
    m = torch.where(torch.isneginf(m), 0.0, m)
    y = z - m
    e = torch.exp(y)
    total = e.sum(1)
    log_total = torch.log(total)
    lse = m[:, 0] + log_total
    entropy = torch.where(empty, 0.0, log_total - torch.where(e > 0, e * y, 0.0).sum(1) / total)
    logp = torch.where(empty, -math.inf, y.gather(1, tokens.clamp_min(0)[:, None])[:, 0] - log_total)
    off = tokens < 0
    out = {"logp": torch.where(off, 0.0, logp), "entropy": torch.where(off, 0.0, entropy),
           "lse": torch.where(off, 0.0, lse), "top_logp": None, "top_ids": None}
    if case["top_k"]:
        # unique whole-number keys: the logit's order above, the column's (lowest first) below
        bits = (x + 0.0).view(torch.int32)
        order = (bits ^ ((bits >> 31) & 0x7FFFFFFF)).to(torch.int64)
        column = torch.arange(x.shape[1], device=x.device)
        ids = torch.topk(order * (1 << 32) + ((1 << 32) - 1 - column), case["top_k"], dim=1).indices
        none = torch.isneginf(x.gather(1, ids))
        top = torch.where(none, -math.inf, y.gather(1, ids) - log_total[:, None])
        out["top_ids"] = torch.where(none | off[:, None], -1, ids)
        out["top_logp"] = torch.where(off[:, None], 0.0, top)
    return out


def _plain_grad(st):
    case, tokens = st["case"], st["tokens"]
    z = torch.cat([s.float() for s in st["shards"]], 1) / case["T"]
    logp = z - st["lse"][:, None]
    p = torch.exp(logp)
    g, gh, ent = st["g_logp"][:, None], st["g_entropy"][:, None], st["entropy"][:, None]
    d = -g * p - gh * p * (logp + ent)
    d.scatter_add_(1, tokens.clamp_min(0)[:, None], g)
    d = torch.where(tokens[:, None] < 0, 0.0, d / case["T"])
    return [x.to(s.dtype) for x, s in zip(torch.split(d, [s.shape[1] for s in st["shards"]], 1), st["shards"])]


def _plain_loss(st):
    case = st["case"]
    logp, old, adv, w, ref, entropy = st["in"]
    lo, hi = np.float32(math.log1p(-CLIP_LOW)).item(), np.float32(math.log1p(CLIP_HIGH)).item()
    kept = w != 0
    d = logp - old
    clipped = ((adv > 0) & (d > hi)) | ((adv < 0) & (d < lo))
    r = torch.exp(d)
    loss = -adv * torch.where(clipped, torch.exp(torch.clamp(d, lo, hi)), r)
    g = torch.where(clipped, 0.0, -adv * r)
    kl = torch.zeros_like(logp)
    if ref is not None:
        q = ref - logp
        kl = torch.expm1(q) - q
        loss = loss + KL_COEF * kl
        g = g - KL_COEF * torch.expm1(q)
    ent = torch.zeros_like(logp)
    g_entropy = None
    if entropy is not None:
        ent = entropy
        loss = loss - ENTROPY_COEF * ent
        g_entropy = -ENTROPY_COEF * w
    total = [torch.where(kept, w * v, 0.0).sum() for v in (loss, kl, ent, clipped.float())]
    return {"stats": torch.stack(total), "g_logp": torch.where(kept, w * g, 0.0), "g_entropy": g_entropy}


# ---------------------------------------------------------------------------
# The work of a pass, and its outputs in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    if case["op"] == "loss":
        n = case["n"]
        arrays = 4 + case["ref"] + case["entropy"] + 1 + case["entropy"]  # read, written
        return {"bytes": 4.0 * n * arrays + 16, "flops": 20.0 * n}
    rows = case["rows"]
    cells = float(rows * case["vocab"])
    scored = cells * (rows - _padded_rows(case)) / rows
    if case["op"] == "logprob":
        return {"bytes": scored * ESIZE[case["dtype"]] + rows * (8 + 12 + 12 * case["top_k"]), "flops": 6.0 * scored}
    return {"bytes": (scored + cells) * ESIZE[case["dtype"]] + rows * 24, "flops": 7.0 * scored}


def exact(case, seed):
    """The definition in 64 bits, a block of rows at a time."""
    st = prepare(case, seed)
    if case["op"] == "loss":
        return _exact_loss(case, st)
    shards, tokens, T = st["shards"], st["tokens"], case["T"]
    parts = []
    for a, b in _row_chunks(case["rows"], case["vocab"]):
        x = torch.cat([s[a:b].double() for s in shards], 1)
        t = tokens[a:b]
        if case["op"] == "logprob":
            parts.append(_exact_logprob_rows(x, t, T, case["top_k"]))
        else:
            parts.append(_exact_grad_rows(x, t, T, *(st[k][a:b].double() for k in ("lse", "entropy", "g_logp", "g_entropy"))))
    if case["op"] == "grad":
        return list(torch.split(torch.cat(parts), [s.shape[1] for s in shards], 1))
    names = ["logp", "entropy", "lse", "top_logp", "top_ids"]
    return {n: torch.cat([p[i] for p in parts]) if parts[0][i] is not None else None for i, n in enumerate(names)}


def _exact_logprob_rows(x, t, T, k):
    some = (x > -math.inf).any(1)
    score = torch.log_softmax(torch.where(some[:, None], x, 0.0) / T, 1)
    score[~some] = -math.inf
    lse = torch.logsumexp(x / T, 1)
    p = torch.exp(score)
    entropy = -torch.special.xlogy(p, p).sum(1)
    logp = score[torch.arange(len(t), device=t.device), t.clamp_min(0)]
    read = t >= 0
    zero = torch.zeros_like(lse)
    top_logp = ids = None
    if k:
        best = torch.sort(x, dim=1, descending=True, stable=True)
        ids = torch.where(torch.isneginf(best.values[:, :k]) | ~read[:, None], -1, best.indices[:, :k])
        top_logp = torch.where(read[:, None], score.gather(1, best.indices[:, :k]), 0.0)
    return (torch.where(read, logp, zero), torch.where(read, entropy, zero), torch.where(read, lse, zero), top_logp, ids)


def _exact_grad_rows(x, t, T, lse, entropy, g, gh):
    # through the definition's own terms: logp_t = z_t - lse, H = lse - sum p z
    s = x / T - lse[:, None]
    p = torch.exp(s)
    hit = torch.zeros_like(p)
    hit[torch.arange(len(t), device=t.device), t.clamp_min(0)] = 1.0
    d = (g[:, None] * (hit - p) - gh[:, None] * (torch.special.xlogy(p, p) + p * entropy[:, None])) / T
    d[t < 0] = 0.0
    return d


def _exact_loss(case, st):
    logp, old, adv, w, ref, entropy = st["in"]
    n = case["n"]
    f = lambda v: np.zeros(n) if v is None else v.cpu().numpy().astype(np.float64)  # noqa: E731
    # the two log ratios are binary32 differences by definition, so that every reader clips the same tokens
    d = (logp - old).cpu().numpy().astype(np.float64)
    q = np.zeros(n) if ref is None else (ref - logp).cpu().numpy().astype(np.float64)
    lo, hi = (float(np.float32(math.log1p(v))) for v in (-CLIP_LOW, CLIP_HIGH))
    a, weight, ent = f(adv), f(w), f(entropy)
    over, under = (a > 0) & (d > hi), (a < 0) & (d < lo)
    ratio = np.exp(np.where(over, hi, np.where(under, lo, d)))
    kl = np.expm1(q) - q
    beta, ce = (KL_COEF if ref is not None else 0.0), (ENTROPY_COEF if entropy is not None else 0.0)
    stats = np.array([math.fsum(weight * v) for v in (beta * kl - a * ratio - ce * ent, kl, ent, (over | under).astype(float))])
    g = weight * (np.where(over | under, 0.0, -a * np.exp(d)) - beta * np.expm1(q))
    return {"stats": stats, "g_logp": g, "g_entropy": -ce * weight if entropy is not None else None}
