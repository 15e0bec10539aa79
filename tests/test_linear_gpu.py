"""The policy head's products on the GPU against 64 bits: token log
probabilities from hidden states, their gradient, quantized rows and the product
of 8-bit integers."""
from __future__ import annotations

import math

import pytest
import torch

from deterministic_collective_movement_amd import rog
from tests import linear_ref as ref

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


def near(got, want, tol, what):
    got = got.double()
    assert got.shape == want.shape, what
    same = (got == want) | (torch.isnan(got) & torch.isnan(want))
    bad = ~(same | ((got - want).abs() <= tol))
    if bad.any():
        at = tuple(int(v) for v in bad.nonzero()[0])
        raise AssertionError("%s: %d of %d off, first at %s: %r, want %r within %g"
                             % (what, int(bad.sum()), bad.numel(), at, float(got[at]), float(want[at]), float(tol[at])))


def check_score(h, ws, tokens, T=1.0, **kw):
    r = rog.rog_linear_logprob(h, ws, tokens, temperature=T, **kw)
    want, tol = ref.score64(h, ws, tokens, T)
    for name, got, w, t in zip(("logp", "entropy", "lse"), r[:3], want, tol):
        near(got, w, t, name)
    return r


SCORE = [
    # rows, widths, dim, dtype, T
    (1, [1], 1, BF16, 1.0),
    (1, [7], 8, F16, 1.0),
    (3, [33], 64, BF16, 0.7),
    (1, [4001], 512, BF16, 1.0),
    (16, [129, 0, 127], 72, F16, 1.3),
    (17, [1000, 1001], 136, BF16, 1.0),
    (33, [300, 5, 2000, 0], 96, F16, 0.5),
    (64, [1024] * 4, 256, BF16, 1.0),
    (65, [1024] * 4, 256, BF16, 1.0),
    (100, [777, 778], 200, F16, 1.0),
    (128, [2000], 65, BF16, 1.0),
    (129, [511, 513], 128, BF16, 1.0),
    (257, [3001], 67, F16, 0.8),
    (300, [513, 2050], 1000, BF16, 1.0),
    (1021, [2003], 160, F16, 0.7),
    (40, [515], 33, BF16, 1.0),
]


@pytest.mark.parametrize("n,widths,dim,dtype,T", SCORE)
def test_score(gpu, n, widths, dim, dtype, T):
    h, ws, tokens = ref.head(n, widths, dim, dtype, gpu, pad=0.2 if n > 3 else 0.0)
    check_score(h, ws, tokens, T)


@pytest.mark.parametrize("n", [1, 30, 64, 100, 129, 260])
@pytest.mark.parametrize("extra", [8, 3])
def test_score_strides(gpu, n, extra):
    h, ws, tokens = ref.head(n, [300, 401], 120, BF16, gpu, extra=extra)
    check_score(h, ws, tokens)


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("widths,dim", [([1500, 1501], 320), ([2048], 1024), ([700], 33)])
def test_a_row_has_the_same_bits_in_any_batch(gpu, dtype, widths, dim):
    h, ws, tokens = ref.head(300, widths, dim, dtype, gpu)
    whole = rog.rog_linear_logprob(h, ws, tokens)
    for a, b in ((0, 1), (5, 6), (7, 23), (0, 17), (100, 164), (30, 95), (200, 300), (3, 260)):
        part = rog.rog_linear_logprob(h[a:b], ws, tokens[a:b])
        for x, y in zip(part[:3], whole[:3]):
            assert torch.equal(x, y[a:b]), (a, b)
    # rows that are not scored between them change nothing
    some = tokens.clone()
    some[torch.arange(300, device=gpu) % 4 == 1] = -1
    r = rog.rog_linear_logprob(h, ws, some)
    for x, y in zip(r[:3], whole[:3]):
        assert torch.equal(x, torch.where(some >= 0, y, 0.0))


def test_score_without_tokens_and_outputs_left_out(gpu):
    h, ws, tokens = ref.head(70, [400], 64, BF16, gpu)
    full = rog.rog_linear_logprob(h, ws, tokens)
    r = rog.rog_linear_logprob(h, ws)
    assert r.logp is None and torch.equal(r.lse, full.lse) and torch.equal(r.entropy, full.entropy)
    out = rog.RogLogprob(torch.empty(70, device=gpu), None, None, None, None)
    assert torch.equal(rog.rog_linear_logprob(h, ws, tokens, out=out).logp, full.logp)


@pytest.mark.parametrize("n", [5, 100, 300])
def test_unscored_rows_are_not_read_and_bad_ones_stay_alone(gpu, n):
    h, ws, tokens = ref.head(n, [500, 300], 128, BF16, gpu)
    good = rog.rog_linear_logprob(h, ws, tokens)
    h = h.clone()
    h[1] = math.nan
    tokens[1] = -1
    h[2, 5] = math.nan
    tokens[3] = 800
    r = rog.rog_linear_logprob(h, ws, tokens)
    assert [float(v[1]) for v in r[:3]] == [0, 0, 0]
    assert all(math.isnan(float(v[2])) for v in r[:3])
    assert math.isnan(float(r.logp[3])) and float(r.lse[3]) == float(good.lse[3])
    keep = [i for i in range(n) if i not in (1, 2, 3)]
    for x, y in zip(r[:3], good[:3]):
        assert torch.equal(x[keep], y[keep])


@pytest.mark.parametrize("n", [2, 80, 200])
def test_infinite_logits(gpu, n):
    # two huge weights whose product with a state passes the binary32 range: +inf makes NaN, -inf has probability 0
    h, ws, tokens = ref.head(n, [300], 64, BF16, gpu, sure=False)
    h[:, 0] = 3e38
    ws[0][:, 0] = 0
    ws[0][7, 0] = -3e38
    tokens[0] = 7
    r = rog.rog_linear_logprob(h, ws, tokens)
    x, _ = ref.logits64(h, ws)
    x[:, 7] = -math.inf
    lse = torch.logsumexp(x, 1)
    assert float(r.logp[0]) == -math.inf
    assert torch.allclose(r.lse.double(), lse, atol=1e-3) and bool(torch.isfinite(r.entropy).all())
    ws[0][9, 0] = 3e38
    r = rog.rog_linear_logprob(h, ws, tokens)
    assert all(bool(torch.isnan(v).all()) for v in r[:3])


def check_grad(h, ws, tokens, T=1.0, seed=0, entropy_grad=True, **kw):
    gen = torch.Generator(device=h.device)
    gen.manual_seed(seed)
    n = h.shape[0]
    size = 8.0 if h.dtype is F16 else 1.0
    g = torch.randn(n, generator=gen, device=h.device) * size
    gh = 0.1 * torch.randn(n, generator=gen, device=h.device) * size
    s = rog.rog_linear_logprob(h, ws, tokens, temperature=T)
    r = rog.rog_linear_logprob_grad(h, ws, tokens, s.lse, s.entropy, g, gh if entropy_grad else None, temperature=T, **kw)
    (dh, dw), (dh_tol, dw_tol) = ref.grad_head64(h, ws, tokens, T, s.lse, s.entropy, g, gh if entropy_grad else torch.zeros_like(g))
    near(r.d_hidden, dh, dh_tol, "d_hidden")
    for i, (a, b, t) in enumerate(zip(r.d_weights, dw, dw_tol)):
        near(a, b, t, "d_weights[%d]" % i)
    return r


GRAD = [
    (1, [1], 1, BF16, 1.0),
    (1, [300], 64, F16, 1.0),
    (5, [129, 0, 200], 72, BF16, 0.7),
    (33, [1000, 1001], 136, F16, 1.3),
    (64, [2100], 256, BF16, 1.0),
    (65, [511, 513], 264, BF16, 1.0),
    (100, [777], 33, F16, 1.0),
    (130, [1024, 700], 515, BF16, 0.8),
    (300, [2500], 320, F16, 1.0),
    (700, [300, 301], 64, BF16, 1.0),
    (20, [9000], 64, BF16, 1.0),
    (300, [5000, 4500], 600, BF16, 1.0),
]


@pytest.mark.parametrize("n,widths,dim,dtype,T", GRAD)
def test_grad(gpu, n, widths, dim, dtype, T):
    h, ws, tokens = ref.head(n, widths, dim, dtype, gpu, pad=0.25 if n > 3 else 0.0)
    check_grad(h, ws, tokens, T, entropy_grad=n != 64)


def test_grad_large_batch_in_one_running_sum(gpu):
    h, ws, tokens = ref.head(2500, [9000, 1000], 3328, BF16, gpu, pad=0.1)
    check_grad(h, ws, tokens)


WIDE = [
    (1500, [4000, 3001], 515, F16, 0.8),      # large tiles, rows that have to be laid out anew
    (600, [9000, 9001], 264, F16, 1.0),
    (2500, [6000], 300, F16, 1.2),            # more rows than a segment has columns
    (2500, [60000], 64, BF16, 1.0),           # two pieces whose segments are joined
    (20, [1060000], 16, BF16, 1.0),           # the same of few rows
    (100, [1060000], 16, F16, 1.0),
    (9000, [130, 255], 33, F16, 1.0),         # many rows, few weights: sums over parts of the rows
    (9000, [1000, 700], 520, BF16, 0.9),
    (70000, [200], 520, F16, 1.0),            # the same in large tiles
]


@pytest.mark.parametrize("n,widths,dim,dtype,T", WIDE)
def test_grad_large(gpu, n, widths, dim, dtype, T):
    h, ws, tokens = ref.head(n, widths, dim, dtype, gpu, pad=0.25)
    check_grad(h, ws, tokens, T)


def test_grad_of_a_state_has_the_same_bits_in_a_large_batch(gpu):
    h, ws, tokens = ref.head(1500, [5000, 3001], 600, BF16, gpu)
    g, gh = torch.randn(1500, device=gpu), 0.1 * torch.randn(1500, device=gpu)
    s = rog.rog_linear_logprob(h, ws, tokens)
    whole = rog.rog_linear_logprob_grad(h, ws, tokens, s.lse, s.entropy, g, gh).d_hidden
    for rows in ([3], list(range(40)), list(range(0, 1500, 8)), list(range(0, 1500, 3))):
        i = torch.tensor(rows, device=gpu)
        part = rog.rog_linear_logprob_grad(h[i], ws, tokens[i], s.lse[i], s.entropy[i], g[i], gh[i]).d_hidden
        assert torch.equal(part, whole[i]), len(rows)


def test_grad_large_of_rows_that_are_not_scored(gpu):
    h, ws, tokens = ref.head(2100, [6000], 520, F16, gpu)
    one = torch.ones(2100, device=gpu)
    for scored in (0, 1, 70):
        tokens[scored:] = -1
        s = rog.rog_linear_logprob(h, ws, tokens)
        r = rog.rog_linear_logprob_grad(h, ws, tokens, s.lse, s.entropy, one)
        assert bool((r.d_hidden[scored:] == 0).all()) and bool((r.d_weights[0] == 0).all()) == (scored == 0)
        tokens[:] = torch.arange(2100, device=gpu)


@pytest.mark.parametrize("n", [30, 200])
def test_grad_strides_leave_what_is_between_rows(gpu, n):
    h, ws, tokens = ref.head(n, [300, 401], 120, BF16, gpu, extra=5)
    dh = torch.full((n, 140), 7.0, dtype=BF16, device=gpu)
    dw = [torch.full((w.shape[0] + 2, 129), 7.0, dtype=BF16, device=gpu) for w in ws]
    check_grad(h, ws, tokens, out=(dh[:, :120], [d[1:-1, 4:124] for d in dw]))
    assert bool((dh[:, 120:] == 7).all())
    for d in dw:
        assert bool((d[0] == 7).all()) and bool((d[-1] == 7).all()) and bool((d[:, :4] == 7).all()) and bool((d[:, 124:] == 7).all())


@pytest.mark.parametrize("dtype", [BF16, F16])
def test_grad_of_a_state_has_the_same_bits_in_any_batch(gpu, dtype):
    h, ws, tokens = ref.head(300, [5000, 3001], 256, dtype, gpu)
    g, gh = torch.randn(300, device=gpu), 0.1 * torch.randn(300, device=gpu)
    g[0] = 4.0            # the largest, so that binary16 takes one scale for all calls
    s = rog.rog_linear_logprob(h, ws, tokens)
    whole = rog.rog_linear_logprob_grad(h, ws, tokens, s.lse, s.entropy, g, gh).d_hidden
    for rows in ([0], [0, 7], list(range(20)), list(range(0, 300, 3))):
        i = torch.tensor(rows, device=gpu)
        part = rog.rog_linear_logprob_grad(h[i], ws, tokens[i], s.lse[i], s.entropy[i], g[i], gh[i]).d_hidden
        assert torch.equal(part, whole[i]), len(rows)


def test_grad_ignores_unscored_states(gpu):
    h, ws, tokens = ref.head(90, [600], 64, BF16, gpu)
    h = h.clone()
    tokens[5::7] = -1
    h[5::7] = math.nan
    g = torch.ones(90, device=gpu)
    s = rog.rog_linear_logprob(h, ws, tokens)
    g[5::7] = math.inf
    r = rog.rog_linear_logprob_grad(h, ws, tokens, s.lse, s.entropy, g)
    assert bool((r.d_hidden[5::7] == 0).all()) and bool(torch.isfinite(r.d_hidden).all()) and bool(torch.isfinite(r.d_weights[0]).all())
    tokens[:] = -1
    r = rog.rog_linear_logprob_grad(h, ws, tokens, s.lse, s.entropy, g)
    assert bool((r.d_hidden == 0).all()) and bool((r.d_weights[0] == 0).all())


def test_grad_against_differences(gpu):
    h, ws, tokens = ref.head(6, [40, 21], 16, BF16, gpu, sigma=1.0)
    g, gh = torch.randn(6, device=gpu), torch.randn(6, device=gpu)
    s = rog.rog_linear_logprob(h, ws, tokens)
    r = rog.rog_linear_logprob_grad(h, ws, tokens, s.lse, s.entropy, g, gh)

    def f(x, w):
        lp = torch.log_softmax(x @ w.t(), 1)
        return (g.double() * lp[torch.arange(6, device=gpu), tokens]).sum() - (gh.double()[:, None] * lp.exp() * lp).sum()

    x, w, e = h.double(), torch.cat([v.double() for v in ws]), 1e-5
    dw = torch.cat(r.d_weights).double()
    for i in range(6):
        for k in range(0, 16, 5):
            d = torch.zeros_like(x)
            d[i, k] = e
            slope = (f(x + d, w) - f(x - d, w)) / (2 * e)
            assert abs(float(slope - r.d_hidden[i, k].double())) < 2.0 ** -6 * (1 + abs(float(slope)))
    for j in range(0, 61, 7):
        d = torch.zeros_like(w)
        d[j, j % 16] = e
        slope = (f(x, w + d) - f(x, w - d)) / (2 * e)
        assert abs(float(slope - dw[j, j % 16])) < 2.0 ** -6 * (1 + abs(float(slope)))


# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("n,dim,extra", [(1, 1, 0), (1, 4096, 0), (7, 33, 3), (300, 1000, 8), (65, 5121, 1), (3, 20000, 0)])
def test_quantize(gpu, dtype, n, dim, extra):
    gen = torch.Generator(device=gpu)
    gen.manual_seed(dim)
    x = (torch.randn(n, dim + extra, generator=gen, device=gpu) * torch.logspace(-3, 3, n, device=gpu)[:, None]).to(dtype)[:, :dim]
    if n > 4:
        x[2] = 0
        x[3, dim // 2] = math.nan
        x[4, dim - 1] = -math.inf
        x[1] = (torch.arange(dim, device=gpu) % 128 + 0.5 * (torch.arange(dim, device=gpu) % 2)).to(dtype)  # ties
        x[1, 0] = 127.0
    got = rog.rog_quantize_i8(x)
    q, s = ref.quantize_cpu(x)
    assert torch.equal(got.q.cpu(), q)
    assert torch.equal(got.scale.cpu().nan_to_num(-1), s.nan_to_num(-1))


def test_quantize_tiny_rows_and_strided_output(gpu):
    x = torch.tensor([[1e-44, 0, -1e-44], [1e-38, 2e-38, -3e-38], [3e38, -3.4e38, 1.0]], device=gpu)
    buf = torch.full((3, 10), 99, dtype=torch.int8, device=gpu)
    got = rog.rog_quantize_i8(x, out=(buf[:, 2:5], torch.empty(3, device=gpu)))
    q, s = ref.quantize_cpu(x)
    assert torch.equal(got.q.cpu(), q) and torch.equal(got.scale.cpu(), s)
    assert bool((buf[:, :2] == 99).all()) and bool((buf[:, 5:] == 99).all())


I8 = [
    (1, [1], 1, BF16), (1, [300], 64, F32), (5, [129, 0, 200], 72, F16), (1, [4001], 2048, BF16), (16, [1000], 128, F32),
    (17, [1001, 1002], 144, BF16), (64, [515], 1000, F16), (65, [2000], 256, BF16), (128, [700, 33], 333, F32),
    (129, [1024], 512, BF16), (257, [1003, 1004], 1040, F16), (300, [2049], 100, F32), (40, [515], 33, BF16), (1021, [777], 65, F16),
]


@pytest.mark.parametrize("n,widths,dim,dtype", I8)
def test_linear_i8(gpu, n, widths, dim, dtype):
    gen = torch.Generator(device=gpu)
    gen.manual_seed(n + dim)
    q = torch.randint(-128, 128, (n, dim), generator=gen, device=gpu, dtype=torch.int8)
    s = torch.rand(n, generator=gen, device=gpu) * 0.01
    ws = [torch.randint(-128, 128, (w, dim), generator=gen, device=gpu, dtype=torch.int8) for w in widths]
    rs = [torch.rand(w, generator=gen, device=gpu) * 0.01 for w in widths]
    out = rog.rog_linear_i8(q, s, ws, rs, dtype=dtype)
    for i, w in enumerate(ws):
        assert out[i].dtype is dtype
        assert torch.equal(out[i].cpu(), ref.linear_i8_cpu(q, s, w, rs[i], dtype)), i


def test_linear_i8_largest_sums(gpu):
    # every product 2^14: the sum of 2^17 - 1 of them is the largest that there can be, and 32 bits hold it
    dim = (1 << 17) - 1
    q = torch.full((3, dim), -128, dtype=torch.int8, device=gpu)
    q[1] = 127
    w = torch.full((40, dim), -128, dtype=torch.int8, device=gpu)
    one = [torch.ones(40, device=gpu)]
    out = rog.rog_linear_i8(q, torch.ones(3, device=gpu), [w], one, dtype=F32)[0]
    assert torch.equal(out.cpu(), ref.linear_i8_cpu(q, torch.ones(3), w, one[0], F32))


@pytest.mark.parametrize("n", [3, 70, 200])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_linear_i8_strides_leave_what_is_between_rows(gpu, n, dtype):
    gen = torch.Generator(device=gpu)
    gen.manual_seed(n)
    q = torch.randint(-127, 128, (n, 100), generator=gen, device=gpu, dtype=torch.int8)[:, 3:90]
    w = torch.randint(-127, 128, (301, 99), generator=gen, device=gpu, dtype=torch.int8)[1:, 5:92]
    s, r = torch.rand(n, device=gpu), torch.rand(300, device=gpu)
    buf = torch.full((n, 311), 7.0, dtype=dtype, device=gpu)
    out = rog.rog_linear_i8(q, s, [w], [r], out=[buf[:, 5:305]])
    assert torch.equal(out[0].cpu(), ref.linear_i8_cpu(q, s, w, r, dtype))
    assert bool((buf[:, :5] == 7).all()) and bool((buf[:, 305:] == 7).all())


@pytest.mark.parametrize("n", [1, 40, 100, 300])
@pytest.mark.parametrize("dim", [10, 42, 100, 1000])
def test_rows_that_end_inside_16_bytes(gpu, n, dim):
    # 4-byte aligned rows whose last 16 bytes are the next row's too: elements past K must count for nothing
    h, ws, tokens = ref.head(n, [300, 77], dim, BF16, gpu)
    check_score(h, ws, tokens)
    if dim % 2 == 0:
        gen = torch.Generator(device=gpu)
        gen.manual_seed(n)
        d = dim // 2 * 4
        q = torch.randint(-128, 128, (n, d), generator=gen, device=gpu, dtype=torch.int8)
        w = torch.randint(-128, 128, (333, d), generator=gen, device=gpu, dtype=torch.int8)
        s, r = torch.rand(n, device=gpu), torch.rand(333, device=gpu)
        out = rog.rog_linear_i8(q, s, [w], [r], dtype=F32)[0]
        assert torch.equal(out.cpu(), ref.linear_i8_cpu(q, s, w, r, F32))
