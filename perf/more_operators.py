"""The policy head's products as a user's program calls them: cases, inputs and plain forms.

Three paths of a head whose weights are W vocabulary shards in rank order:
``score`` (log probability of given tokens from hidden states, with entropy and
log-sum-exp, without keeping the logits), ``grad`` (its gradient in the hidden
states and in every shard's weights) and ``i8`` (logits of the head held in 8-bit
integers: the states are quantized per token, the weights were per channel).
``run`` computes them in plain torch operations in 32 bits, or, where ``own`` is
true, through the library's entry points.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
ESIZE = {"bf16": 2, "f16": 2, "f32": 4}


def _case(op, name, rows, vocab, hidden, dtype, W=1, T=1.0, pad=0.0, extra=0):
    """rows states of `hidden` elements against `vocab` columns in W shards; pad: share
    of rows that are not scored; extra: unused elements behind each state (a row
    stride larger than the width); i8: dtype of the states and the logits."""
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "hidden": hidden, "dtype": dtype, "W": W, "T": T,
            "pad": pad, "extra": extra}


def listed():
    return [
        # one new token of one request: latency
        _case("score", "score 1x32003 d512", 1, 32003, 512, "bf16"),
        # a decode batch over eight ranks' shards: the weights are read once
        _case("score", "score 64x131072 d4096 w8", 64, 131072, 4096, "bf16", W=8, T=0.8),
        # odd vocabulary, odd row count, some rows padding, states inside wider rows
        _case("score", "score 1021x50257 d1600 f16", 1021, 50257, 1600, "f16", T=0.7, pad=0.125, extra=32),
        # a training step's rows over eight ranks' shards
        _case("score", "score 8192x131072 d4096 w8", 8192, 131072, 4096, "bf16", W=8, pad=0.125),
        # gradients: a small batch, an odd vocabulary with padding rows, a training step
        _case("grad", "grad 33x32003 d1024 w2", 33, 32003, 1024, "bf16", W=2),
        _case("grad", "grad 1021x50257 d1600 f16", 1021, 50257, 1600, "f16", T=0.7, pad=0.125, extra=32),
        _case("grad", "grad 4096x131072 d4096 w8", 4096, 131072, 4096, "bf16", W=8, pad=0.125),
        # sampling with 8-bit weights: one request, a decode batch over eight shards, prompts' logits
        _case("i8", "i8 1x32000 d2048", 1, 32000, 2048, "bf16"),
        _case("i8", "i8 48x131072 d4096 w8", 48, 131072, 4096, "bf16", W=8),
        _case("i8", "i8 509x32003 d1000 f32 w2", 509, 32003, 1000, "f32", W=2),
        _case("i8", "i8 4093x50257 d5120 f16", 4093, 50257, 5120, "f16"),
    ]


MOST = {"score": 8192 * 131072 * 4096, "grad": 4096 * 131072 * 4096, "i8": 4093 * 50257 * 5120}


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(["score", "score", "grad", "grad", "i8", "i8"])
    vocab = _log_uniform(rng, 1000, 131072)
    hidden = _log_uniform(rng, 64, 5120)
    unit = rng.choice([64, 64, 64, 64, 64, 64, 64, 16, 8, 1])  # widths of models; now and then any
    hidden = max(unit, hidden // unit * unit)
    rows = _log_uniform(rng, 1, min(8192, MOST[op] // (vocab * hidden)))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"] if op == "i8" else ["bf16", "bf16", "f16"])
    case = _case(op, "", rows, vocab, hidden, dtype, W=rng.choice([1, 1, 2, 4, 8]),
                 T=1.0 if op == "i8" else rng.choice([1.0, 1.0, round(rng.uniform(0.5, 1.6), 2)]),
                 pad=0.0 if op == "i8" else rng.choice([0.0, 0.0, 0.125, 0.4]), extra=rng.choice([0, 0, 64]))
    del case["name"]
    return case


def _widths(vocab, W):
    """W shard widths in rank order: equal where W divides the vocabulary, the last ones a column shorter where not."""
    return [vocab // W + (1 if r < vocab % W else 0) for r in range(W)]


def _padded_rows(case):
    return int(case["rows"] * case["pad"])


def _row_chunks(rows, vocab, most=1 << 28):
    step = max(1, most // vocab)
    return [(a, min(rows, a + step)) for a in range(0, rows, step)]


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

LOSS_SCALE = 4096.0  # of a training program in binary16


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rows, vocab, hidden, dtype = case["rows"], case["vocab"], case["hidden"], DTYPES[case["dtype"]]
    weights = []
    for width in _widths(vocab, case["W"]):
        w = torch.randn(width, hidden, generator=gen, device=dev, dtype=dtype)
        weights.append(w.mul_(2.5 / math.sqrt(hidden)))  # logits of about 2.5
    tokens = torch.randint(0, vocab, (rows,), generator=gen, device=dev)
    states = torch.randn(rows, hidden + case["extra"], generator=gen, device=dev)
    # a third of the rows are sure of their token, as a trained policy is of most
    lo = 0
    for w in weights:
        at = torch.nonzero((tokens >= lo) & (tokens < lo + w.shape[0]) & (torch.arange(rows, device=dev) % 3 == 0))[:, 0]
        states[at, :hidden] += 2.5 * w[tokens[at] - lo].float()
        lo += w.shape[0]
    states = states.to(dtype)[:, :hidden]
    st = {"op": case["op"], "case": case, "states": states}
    if case["op"] == "i8":
        q = [_quantize(w.float()) for w in weights]  # once, when the weights are loaded
        st["weights"], st["scales"] = [a for a, _ in q], [s for _, s in q]
        st["out"] = [torch.empty(rows, w.shape[0], dtype=dtype, device=dev) for w in weights]
        return st
    st["weights"] = weights
    tokens[torch.randperm(rows, generator=gen, device=dev)[:_padded_rows(case)]] = -1
    st["tokens"] = tokens
    if case["op"] == "score":
        st["out"] = (torch.empty(rows, device=dev), torch.empty(rows, device=dev), torch.empty(rows, device=dev), None, None)
        return st
    # what the forward pass has left, and the loss's gradients
    st["lse"], st["entropy"] = _lse_entropy(case, st)
    scale = (LOSS_SCALE if case["dtype"] == "f16" else 1.0) / rows
    st["g_logp"] = torch.randn(rows, generator=gen, device=dev) * scale
    st["g_entropy"] = 0.02 * torch.randn(rows, generator=gen, device=dev) * scale
    st["out"] = (torch.empty(rows, hidden, dtype=dtype, device=dev), [torch.empty_like(w) for w in weights])
    return st


def _quantize(x):
    """Rows of x in 8-bit integers and their scales: s = max |x| / 127, q = x / s to the nearest, ties to even."""
    most = x.abs().amax(1)
    s = (most / torch.full_like(most, 127.0)).clamp_min(2.0 ** -126)  # a division: by a number it is a product with 1 / 127
    return torch.round(x / s[:, None]).to(torch.int8), s


def _lse_entropy(case, st):
    """log-sum-exp and entropy per row, in 64 bits, rounded to 32: zero where the row is not scored."""
    lse, ent = [], []
    W = torch.cat(st["weights"]).double()
    for a, b in _row_chunks(case["rows"], case["vocab"]):
        z = st["states"][a:b].double() @ W.t() / case["T"]
        l = torch.logsumexp(z, 1)
        ent.append(l - (torch.exp(z - l[:, None]) * z).sum(1))
        lse.append(l)
    scored = st["tokens"] >= 0
    return (torch.where(scored, torch.cat(lse), 0.0).float(), torch.where(scored, torch.cat(ent), 0.0).float())


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(st):
    if own:
        return _run_own(st)
    return {"score": _plain_score, "grad": _plain_grad, "i8": _plain_i8}[st["op"]](st)


def _run_own(st):
    from deterministic_collective_movement_amd import rog
    case = st["case"]
    if st["op"] == "score":
        r = rog.rog_linear_logprob(st["states"], st["weights"], st["tokens"], temperature=case["T"], out=st["out"])
        return {"logp": r.logp, "entropy": r.entropy, "lse": r.lse}
    if st["op"] == "grad":
        r = rog.rog_linear_logprob_grad(st["states"], st["weights"], st["tokens"], st["lse"], st["entropy"], st["g_logp"],
                                        st["g_entropy"], temperature=case["T"], out=st["out"])
        return [r.d_hidden] + list(r.d_weights)
    q, s = rog.rog_quantize_i8(st["states"])
    return rog.rog_linear_i8(q, s, st["weights"], st["scales"], out=st["out"])


def _plain_score(st):
    case, tokens = st["case"], st["tokens"]
    z = torch.cat([st["states"].float() @ w.float().t() for w in st["weights"]], 1) / case["T"]
    m = z.amax(1, keepdim=True)
    y = z - m
    e = torch.exp(y)
    total = e.sum(1)
    log_total = torch.log(total)
    logp = y.gather(1, tokens.clamp_min(0)[:, None])[:, 0] - log_total
    entropy = log_total - (e * y).sum(1) / total
    off = tokens < 0
    return {"logp": torch.where(off, 0.0, logp), "entropy": torch.where(off, 0.0, entropy),
            "lse": torch.where(off, 0.0, m[:, 0] + log_total)}


def _plain_grad(st):
    case, tokens = st["case"], st["tokens"]
    h = st["states"].float()
    z = torch.cat([h @ w.float().t() for w in st["weights"]], 1) / case["T"]
    logp = z - st["lse"][:, None]
    p = torch.exp(logp)
    g, gh, ent = st["g_logp"][:, None], st["g_entropy"][:, None], st["entropy"][:, None]
    d = -g * p - gh * p * (logp + ent)
    d.scatter_add_(1, tokens.clamp_min(0)[:, None], g)
    d = torch.where(tokens[:, None] < 0, 0.0, d / case["T"])
    d_hidden, d_weights = torch.zeros_like(h), []
    for part, w in zip(torch.split(d, [w.shape[0] for w in st["weights"]], 1), st["weights"]):
        d_hidden += part @ w.float()
        d_weights.append((part.t() @ h).to(w.dtype))
    return [d_hidden.to(st["states"].dtype)] + d_weights


def _plain_i8(st):
    q, s = _quantize(st["states"].float())
    out = []
    for w, r in zip(st["weights"], st["scales"]):
        y = _sums(q, w) * s[:, None] * r
        out.append(y.to(st["states"].dtype))
    return out


def _sums(q, w):
    """sum_k q_ik w_jk, exactly: products of 1000 columns and fewer stay below 2^24, where binary32 is exact."""
    total = None
    for a in range(0, q.shape[1], 1000):
        part = q[:, a:a + 1000].float() @ w[:, a:a + 1000].float().t()
        total = part if total is None else total.to(torch.int32) + part.to(torch.int32)
    return total.float()


# ---------------------------------------------------------------------------
# The work of a pass, and its outputs in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    n, v, d = case["rows"], case["vocab"], case["hidden"]
    kept = n - _padded_rows(case)
    b = ESIZE[case["dtype"]]
    if case["op"] == "score":
        return {"bytes": float(v * d * b + kept * d * b + n * 20), "flops": 2.0 * kept * v * d}
    if case["op"] == "grad":
        return {"bytes": float(2 * v * d * b + (kept + n) * d * b + n * 24), "flops": 6.0 * kept * v * d}
    return {"bytes": float(v * d + 4 * v + n * d * b + n * v * b), "flops": 2.0 * n * v * d}


def exact(case, seed):
    """The definition in 64 bits, a block of rows at a time."""
    st = prepare(case, seed)
    x = st["states"]
    if case["op"] == "i8":
        return _exact_i8(case, st)
    W = torch.cat(st["weights"]).double()
    tokens, parts, d_w = st["tokens"], [], torch.zeros_like(W) if case["op"] == "grad" else None
    for a, b in _row_chunks(case["rows"], case["vocab"]):
        h, t = x[a:b].double(), tokens[a:b]
        score = torch.log_softmax(h @ W.t() / case["T"], 1)
        hit = torch.arange(b - a, device=x.device), t.clamp_min(0)
        read = t >= 0
        if case["op"] == "score":
            lse = torch.logsumexp(h @ W.t() / case["T"], 1)
            entropy = -(torch.exp(score) * score).sum(1)
            parts.append([torch.where(read, v, 0.0) for v in (score[hit], entropy, lse)])
            continue
        # through the definition's own terms: logp_t = z_t - lse, H = lse - sum p z, with lse and H as they are given
        lse, ent, g, gh = (st[k][a:b].double()[:, None] for k in ("lse", "entropy", "g_logp", "g_entropy"))
        s = h @ W.t() / case["T"] - lse
        p = torch.exp(s)
        d = -(g * p + gh * (p * s + p * ent))
        d[hit] += g[:, 0]
        d = d * read[:, None] / case["T"]
        parts.append(d @ W)
        d_w += d.t() @ h
    if case["op"] == "grad":
        return [torch.cat(parts)] + list(torch.split(d_w, _widths(case["vocab"], case["W"])))
    return {n: torch.cat([p[i] for p in parts]) for i, n in enumerate(("logp", "entropy", "lse"))}


def _exact_i8(case, st):
    x = st["states"].double()
    # the scale and the quotient are binary32 by definition (a quotient of 64 bits rounds to it as the exact one does)
    s = (x.abs().amax(1) / 127.0).float().clamp_min(2.0 ** -126).double()
    q = torch.round((x / s[:, None]).float()).double()
    out = []
    for w, r in zip(st["weights"], st["scales"]):
        parts = [(q[a:b] @ w.double().t()) * (s[a:b, None] * r.double()) for a, b in _row_chunks(case["rows"], w.shape[0])]
        out.append(torch.cat(parts))
    return out
