"""The policy head's products as they are called: broadcast inputs, captured and
replayed, on two streams at once, far into memory, through the plain binding,
and one after the other as a policy's step takes them."""
from __future__ import annotations

import math

import pytest
import torch

from deterministic_collective_movement_amd import rog
from tests import linear_ref as ref
from tests.test_linear_gpu import check_grad, check_score, near

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.mark.parametrize("n", [9, 90, 200])
def test_broadcast_inputs(gpu, n):
    # one state for all rows, one vector for all columns of a shard: rows 0 bytes apart
    h, ws, tokens = ref.head(n, [300, 200], 136, BF16, gpu)
    check_score(h[:1].expand(n, 136), ws, tokens)
    ws = [ws[0], ws[1][:1].expand(200, 136)]
    check_score(h, ws, tokens)
    check_grad(h, ws, tokens)
    check_grad(h[3:4].expand(n, 136), ws, tokens)
    q = rog.rog_quantize_i8(h[:1].expand(n, 136))
    one = ref.quantize_cpu(h[:1])
    assert torch.equal(q.q.cpu(), one[0].expand(n, 136)) and torch.equal(q.scale.cpu(), one[1].expand(n))
    w = torch.randint(-127, 128, (1, 136), device=gpu, dtype=torch.int8).expand(130, 136)
    out = rog.rog_linear_i8(q.q[:1].expand(n, 136), q.scale, [w], [torch.ones(130, device=gpu)], dtype=F32)[0]
    assert torch.equal(out.cpu(), ref.linear_i8_cpu(one[0].expand(n, 136), one[1].expand(n), w, torch.ones(130), F32))


def test_one_row_of_any_stride(gpu):
    # a single row's stride is not read, however large it is called
    h, ws, tokens = ref.head(1, [300], 64, BF16, gpu)
    wide = torch.as_strided(h.contiguous(), (1, 64), (1 << 40, 1))
    a, b = rog.rog_linear_logprob(wide, ws, tokens), rog.rog_linear_logprob(h, ws, tokens)
    assert all(torch.equal(x, y) for x, y in zip(a[:3], b[:3]))


def test_rows_that_are_none_or_not_scored(gpu):
    h, ws, tokens = ref.head(150, [300], 64, BF16, gpu)
    for n in (0, 10, 64, 150):
        t = torch.full((n,), -1, dtype=torch.int64, device=gpu)
        r = rog.rog_linear_logprob(h[:n], ws, t)
        assert all(v.shape == (n,) and bool((v == 0).all()) for v in r[:3])
        z = torch.ones(n, device=gpu)
        g = rog.rog_linear_logprob_grad(h[:n], ws, t, z, z, z)
        assert bool((g.d_hidden == 0).all())
        if n:          # no rows: nothing is enqueued
            assert bool((g.d_weights[0] == 0).all())
    assert rog.rog_linear_i8(torch.empty(0, 64, dtype=torch.int8, device=gpu), torch.empty(0, device=gpu),
                             [torch.ones(5, 64, dtype=torch.int8, device=gpu)], [torch.ones(5, device=gpu)])[0].shape == (0, 5)
    r = rog.rog_linear_logprob(h, [ws[0][:0]], tokens)          # a head without columns
    assert bool((r.lse == -math.inf).all()) and bool(torch.isnan(r.logp).all()) and bool((r.entropy == 0).all())


def step(h, ws, tokens, T):
    s = rog.rog_linear_logprob(h, ws, tokens, temperature=T)
    loss = rog.rog_policy_loss(s.logp, s.logp - 0.1, torch.ones_like(s.logp), entropy=s.entropy, entropy_coef=0.01, grad_scale=64.0)
    g = rog.rog_linear_logprob_grad(h, ws, tokens, s.lse, s.entropy, loss.g_logp, loss.g_entropy, temperature=T)
    q = rog.rog_quantize_i8(h)
    w8 = [rog.rog_quantize_i8(w) for w in ws]
    logits = rog.rog_linear_i8(q.q, q.scale, [w.q for w in w8], [w.scale for w in w8])
    best = rog.rog_logprob(logits, tokens, top_k=3, temperature=T)
    return [s.logp, s.entropy, s.lse, loss.stats, g.d_hidden, *g.d_weights, *logits, best.logp, best.top_ids]


@pytest.mark.parametrize("n,dtype", [(20, BF16), (90, F16), (300, BF16)])
def test_a_policy_step(gpu, n, dtype):
    """The whole run, against the same formulas in 64 bits."""
    T = 0.9
    h, ws, tokens = ref.head(n, [400, 401], 192, dtype, gpu, sigma=1.5)
    got = step(h, ws, tokens, T)
    x = h.double().requires_grad_()
    w = [v.double().requires_grad_() for v in ws]
    lp = torch.log_softmax(x @ torch.cat(w).t() / T, 1)
    entropy = -(lp.exp() * lp).sum(1)
    logp = lp[torch.arange(n, device=gpu), tokens]
    old = (got[0] - 0.1).double()
    loss = -torch.exp(logp - old).mean() - 0.01 * entropy.mean()          # e^0.1 is inside the clip range
    (loss * 64.0).backward()
    assert abs(float(got[3][0]) - float(loss.detach())) < 1e-5
    # two roundings to the states' type of what the sums hold (2^-8 each), and a term's share of cancelling ones
    for a, b in zip([got[4]] + got[5:7], [x.grad] + [v.grad for v in w]):
        assert float((a.double() - b).norm() / b.norm()) < 2 * ref.HALF[dtype]
    # 8-bit logits: |error| <= dim * (half a step of either side times the other, and both)
    sq, sw = h.abs().amax(1).double() / 127, torch.cat(ws).abs().amax(1).double() / 127
    bound = 0.5 * (sq[:, None] * torch.cat(ws).double().abs().sum(1) + sw * h.double().abs().sum(1)[:, None]) + 0.25 * 192 * sq[:, None] * sw
    z = h.double() @ torch.cat(ws).double().t()
    got8 = torch.cat(got[7:9], 1).double()
    assert bool(((got8 - z).abs() <= bound * 1.01 + 2.0 ** -8 * (z.abs() + bound)).all())
    assert torch.equal(got[-1], torch.sort(torch.cat(got[7:9], 1).float(), dim=1, descending=True, stable=True).indices[:, :3])


@pytest.mark.parametrize("n", [3, 40, 100, 300])
def test_captured_and_replayed(gpu, n):
    h, ws, tokens = ref.head(n, [900, 333], 136, BF16, gpu, pad=0.2)
    want = [t.clone() for t in step(h, ws, tokens, 1.0)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(h, ws, tokens, 1.0)
    side.synchronize()
    with torch.cuda.graph(graph):
        got = step(h, ws, tokens, 1.0)
    for i in range(4):
        other = step(h * 0.5, ws, tokens, 1.0)          # eager work between the replays
        graph.replay()
        torch.cuda.synchronize()
        assert len(other) == len(got)
        for a, b in zip(got, want):
            assert torch.equal(a, b), i
    # new inputs in place
    h2, ws2, tokens2 = ref.head(n, [900, 333], 136, BF16, gpu, seed=5, pad=0.5)
    h.copy_(h2), tokens.copy_(tokens2)
    for a, b in zip(ws, ws2):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, step(h2, ws2, tokens2, 1.0)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("n", [30, 200])
def test_two_streams_at_once(gpu, n):
    cases = [ref.head(n, [5000, 3000], 512, BF16, gpu, seed=i) for i in range(2)]
    want = [[t.clone() for t in step(*c, 1.0)] for c in cases]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(step(*c, 1.0))
        torch.cuda.synchronize()
        for g, w in zip(got, want):
            assert all(torch.equal(a, b) for a, b in zip(g, w))


def test_a_stream_by_name_and_a_workspace_of_the_callers(gpu):
    h, ws, tokens = ref.head(100, [500], 64, BF16, gpu)
    want = rog.rog_linear_logprob(h, ws, tokens)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    need = rog.rog_linear_logprob_plan([500], 100, 64)["workspace_bytes"]
    own = rog.rog_workspace(need, stream=s)
    own[(1 << 17):] = 255                     # left-overs of another call; the counters at the front stay zero
    s.wait_stream(torch.cuda.current_stream())
    got = rog.rog_linear_logprob(h, ws, tokens, stream=s, workspace=own)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got[:3], want[:3]))
    assert bool((own[:1 << 17] == 0).all())
    with pytest.raises(rog.RogArgumentError):
        rog.rog_linear_logprob(h, ws, tokens, workspace=own[:need - 1])


def test_the_shared_workspace_still_serves_split_rows(gpu):
    # the same stream's workspace, used by both: a split launch counts arrivals in its front
    x = [torch.randn(4, 60000, device=gpu).to(BF16)]
    t = torch.randint(0, 60000, (4,), device=gpu)
    want = rog.rog_logprob(x, t, top_k=4)
    h, ws, tokens = ref.head(300, [3000], 256, BF16, gpu)
    s = rog.rog_linear_logprob(h, ws, tokens)
    rog.rog_linear_logprob_grad(h, ws, tokens, s.lse, s.entropy, torch.ones(300, device=gpu))
    got = rog.rog_logprob(x, t, top_k=4)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_without_the_compiled_module(gpu, monkeypatch):
    h, ws, tokens = ref.head(70, [300, 100], 64, BF16, gpu)
    want = [t.clone() for t in step(h, ws, tokens, 1.0)]
    monkeypatch.setattr(rog, "_binding", None)
    assert all(torch.equal(a, b) for a, b in zip(step(h, ws, tokens, 1.0), want))


@pytest.mark.parametrize("n", [40, 200])
def test_weights_past_four_gibibytes(gpu, n):
    # the last columns of a shard of more than 2^32 bytes, and their gradient's
    dim, width = 4096, (1 << 32) // (4096 * 2) + 300
    w = torch.zeros(width, dim, dtype=BF16, device=gpu)
    gen = torch.Generator(device=gpu)
    gen.manual_seed(n)
    w[-200:] = (torch.randn(200, dim, generator=gen, device=gpu) * 0.04).to(BF16)
    h = torch.randn(n, dim, generator=gen, device=gpu).to(BF16)
    tokens = torch.randint(width - 200, width, (n,), generator=gen, device=gpu)
    r = rog.rog_linear_logprob(h, [w], tokens)
    z = torch.zeros(n, width, dtype=torch.float64, device=gpu)
    z[:, -200:] = h.double() @ w[-200:].double().t()
    lse = torch.logsumexp(z, 1)
    tol = torch.full_like(lse, 1e-3)          # 4097 additions of at most 2^-23 of sums below 200, twice
    near(r.lse, lse, tol, "lse")
    near(r.logp, z[torch.arange(n, device=gpu), tokens] - lse, tol, "logp")
    g = torch.randn(n, generator=gen, device=gpu)
    d = rog.rog_linear_logprob_grad(h, [w], tokens, r.lse, r.entropy, g)
    p = torch.exp(z - lse[:, None])
    G = -g.double()[:, None] * p
    G[torch.arange(n, device=gpu), tokens] += g.double()
    want = G[:, -200:].t() @ h.double()
    assert float((d.d_weights[0][-200:].double() - want).norm() / want.norm()) < 2 * ref.HALF[BF16]
    want = G[:, -200:] @ w[-200:].double()
    assert float((d.d_hidden.double() - want).norm() / want.norm()) < 2 * ref.HALF[BF16]
    first = G[:, :100].t() @ h.double()
    assert float((d.d_weights[0][:100].double() - first).norm() / first.norm()) < 2 * ref.HALF[BF16]


@pytest.mark.parametrize("n", [1, 50, 120, 300])
def test_logits_far_apart(gpu, n):
    # logits of +-3000: a row is sure of one token, the others' terms are 0 (and 0 times their distance is 0)
    h, ws, tokens = ref.head(n, [500], 64, BF16, gpu, sigma=1000.0, sure=False)
    (logp, entropy, lse), (a, b, c) = ref.score64(h, ws, tokens, 1.0)
    r = rog.rog_linear_logprob(h, ws, tokens)
    near(r.lse, lse, c, "lse")
    near(r.logp, logp, a, "logp")
    assert bool(torch.isfinite(r.entropy).all()) and bool((r.entropy >= 0).all())
