"""Token log probabilities and their gradient on the GPU against plain 64-bit
forms: sizes where blocks, quads and shards end, masks and infinities, strides
and alignments, launch forms, streams and graphs."""
from __future__ import annotations

import math

import pytest
import torch

from deterministic_collective_movement_amd import rog
from tests import head_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
LOWEST = {t: torch.finfo(t).min for t in (BF16, F16, F32)}


def make(rows, widths, dtype, seed, gpu, spread=3.0):
    gen = torch.Generator(device=gpu)
    gen.manual_seed(seed)
    return [(spread * torch.randn(rows, w, generator=gen, device=gpu)).to(dtype) for w in widths]


def some_tokens(rows, V, seed, gpu, skip=True):
    gen = torch.Generator(device=gpu)
    gen.manual_seed(seed + 1)
    t = torch.randint(0, max(1, V), (rows,), generator=gen, device=gpu)
    if skip and rows > 2:
        t[rows // 2] = -1
    return t


def forms_of(widths, rows, k):
    """Every launch form that takes rows of these widths."""
    found = []
    for form in (rog.ROG_LOGPROB_ROW, rog.ROG_LOGPROB_SPLIT, rog.ROG_LOGPROB_WAVE):
        try:
            rog.rog_logprob_plan_widths(widths, rows, rog.ROG_DTYPE_BF16, k, form)
        except rog.RogArgumentError:
            continue
        found.append(form)
    return found


def same_bits(a, b):
    return all((x is None and y is None) or torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def check(shards, tokens, T=1.0, k=0):
    """Runs every form, holds them to equal bits and the first to the 64-bit form."""
    x = ref.rows64(shards)
    outs = [rog.rog_logprob_ex(shards, tokens, k, T, form=f)
            for f in forms_of([s.shape[1] for s in shards], shards[0].shape[0], k)]
    assert outs
    got = outs[0]
    for other in outs[1:]:
        assert same_bits(got, other)
    assert same_bits(got, rog.rog_logprob(shards, tokens, k, T))
    logp, entropy, lse, top_logp, top_ids = ref.logprob64(x, tokens, T, k)
    tol, tol_h = ref.logprob_tol(x, T, torch.nan_to_num(entropy))
    lse = lse.clamp(-3.4028234e38, 3.4028234e38).where(torch.isfinite(lse), lse)   # held in the finite range

    def near(a, b, tol, what):
        a = a.double()
        tol = tol.expand_as(b) + 2 * ref.U * torch.where(torch.isfinite(b), b.abs(), 0.0)   # its own rounding
        ok = (a == b.float()) | (torch.isnan(a) & torch.isnan(b)) | ((a - b).abs() <= tol)   # past the binary32 range: infinite
        assert bool(ok.all()), (what, a[~ok][:4], b[~ok][:4], tol[~ok][:4])

    if logp is not None:
        near(got.logp, logp, tol, "logp")
    near(got.lse, lse, tol, "lse")
    near(got.entropy, entropy, tol_h, "entropy")
    if k:
        assert torch.equal(got.top_ids, top_ids), (got.top_ids, top_ids)
        near(got.top_logp, top_logp, tol[:, None], "top_logp")
    return got


WIDTHS = [[1], [5], [64], [511], [512], [2047], [2048], [2049], [8192], [8193], [1000, 1], [0, 7, 0], [1] * 64,
          [4096, 2048, 5000], [16001, 16002], [50257], [131072], [16384] * 8, [140001]]


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("widths", WIDTHS, ids=lambda w: "+".join(map(str, w[:3])) + ("x%d" % len(w) if len(w) > 3 else ""))
def test_sizes(gpu, widths, dtype):
    V = sum(widths)
    for rows, k, T in ((1, 5, 1.0), (5, 0, 0.7), (7, 32, 1.3)):
        shards = make(rows, widths, dtype, V + rows, gpu)
        check(shards, some_tokens(rows, V, V, gpu), T, k)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("widths", [[37], [3000], [9001, 9000], [70001]], ids=str)
def test_masks_and_infinities(gpu, widths, dtype):
    V, T, k = sum(widths), 0.9, 20
    x = torch.cat(make(24, widths, dtype, V, gpu), 1)
    low = LOWEST[dtype]
    gen = torch.Generator(device=gpu)
    gen.manual_seed(V)
    half = torch.rand(V, generator=gen, device=gpu) < 0.5
    tokens = some_tokens(24, V, V, gpu, skip=False)
    x[0] = -math.inf                                   # nothing left
    x[1] = low                                         # masked with the lowest finite value: uniform
    x[2, half] = -math.inf
    x[3, half] = low
    x[4] = -math.inf
    x[4, V // 3] = 1.5                                 # one column left
    x[5] = -math.inf
    x[5, V // 2:V // 2 + 7] = torch.linspace(-2, 2, 7, device=gpu).to(dtype)   # fewer left than alternatives
    x[6] = 0.25                                        # all equal: the lowest columns first
    x[7] = low
    x[7, half] = -math.inf                             # uniform over what is not -inf
    x[8, V - 1] = math.inf
    x[9, V // 4] = math.nan
    x[10] = math.nan
    x[11, 0] = -math.inf
    x[11, V - 1] = -math.inf
    tokens[11] = V - 1                                 # a token that the mask forbids
    x[12, ::2] = -0.0
    x[12, 1::2] = 0.0                                  # -0 and +0 are one value
    x[13] = torch.arange(V, device=gpu).remainder(3).to(dtype)     # a third of the columns tie
    x[14] = torch.arange(V, device=gpu).div(V).to(dtype)           # rising: the best columns last
    x[15] = -torch.arange(V, device=gpu).div(V).to(dtype)
    x[16] = -low                                       # the largest finite value everywhere
    x[17] = -low
    x[17, ::3] = 1.0
    x[18] = low
    x[18, V // 2] = low / 2
    tokens[18] = V // 2
    x[19, 5] = -low
    tokens[20] = -1
    x[20] = math.nan                                   # not scored: not read
    tokens[21] = V                                     # past the end
    tokens[22] = 2 ** 40
    x[23, V // 2] = 60.0                               # sure of one token
    tokens[23] = V // 2
    shards = [s.contiguous() for s in torch.split(x, widths, 1)]
    got = check(shards, tokens, T, k)
    assert torch.isneginf(got.logp[0]) and got.entropy[0] == 0 and torch.isneginf(got.lse[0])
    assert bool((got.top_ids[6] == torch.arange(k, device=gpu)).all())


@pytest.mark.parametrize("T", [1.0, 8.0, 1024.0])
@pytest.mark.parametrize("dtype", [F16, BF16], ids=["f16", "bf16"])
@pytest.mark.parametrize("widths", [[3], [37], [3000], [9001, 9000], [70001]], ids=str)
def test_lowest_logits_beside_infinities(gpu, widths, dtype, T):
    """-inf stays nothing where the others are binary16's lowest values, however small a temperature makes the distance."""
    V = sum(widths)
    ramp = (-65504.0 + 32.0 * torch.arange(V, device=gpu).remainder(8)).to(dtype)
    x = torch.full((6, V), -math.inf, dtype=dtype, device=gpu)
    x[0, V // 2] = -65472.0
    x[1, ::2] = ramp[::2]
    x[2, V - 1] = -65504.0
    x[3, 3 * V // 4:] = ramp[3 * V // 4:]
    x[4, :2] = ramp[:2]
    x[5, ::3] = -60000.0
    tokens = torch.tensor([V // 2, 0, V - 1, 0, 1, 0], device=gpu)
    check(list(torch.split(x, widths, 1)), tokens, T, 5)


@pytest.mark.parametrize("k", [1, 3, 20, 31, 32])
def test_alternatives_under_ties(gpu, k):
    """Few distinct values, so that far more columns reach the K-th best value than are wanted."""
    gen = torch.Generator(device=gpu)
    gen.manual_seed(k)
    for V, distinct in ((600, 2), (5000, 1), (40000, 3), (140000, 2), (140000, 40)):
        x = torch.randint(0, distinct, (3, V), generator=gen, device=gpu).to(BF16)
        x[1, : V // 2] = 50                            # a long run at the front of the row
        x[2] = x[2].sort().values
        check([x], some_tokens(3, V, k, gpu, skip=False), 1.0, k)


@pytest.mark.parametrize("dtype", [BF16, F32], ids=["bf16", "f32"])
def test_strides_and_alignments(gpu, dtype):
    """Rows at every 16-byte phase, column slices of a wider matrix, one row repeated: the same bits as packed rows."""
    base = torch.cat(make(6, [5000], dtype, 3, gpu), 1)
    tokens = some_tokens(6, 4100, 3, gpu)
    want = check([base[:, 100:4200].contiguous()], tokens, 1.0, 4)
    assert same_bits(want, rog.rog_logprob([base[:, 100:4200]], tokens, 4))
    for shift in range(1, 9):
        buf = torch.full((6 * 4101 + 64,), math.nan, dtype=dtype, device=gpu)
        view = buf[shift:shift + 6 * 4101].view(6, 4101)[:, :4100]
        view.copy_(base[:, 100:4200])
        assert same_bits(want, rog.rog_logprob([view], tokens, 4)), shift
    halves = [base[:, 100:2100], base[:, 2100:4200]]
    split = check(halves, tokens, 1.0, 4)
    assert torch.equal(split.top_ids, want.top_ids)
    one = base[:1, 100:4200].expand(6, 4100)
    rep = rog.rog_logprob([one], torch.full((6,), 17, device=gpu), 4)
    assert all(bool((t == t[:1]).all()) for t in rep)


@pytest.mark.parametrize("widths", [[8192], [32000], [16384] * 8], ids=str)
def test_rows_do_not_depend_on_their_batch(gpu, widths):
    rows, V = 300, sum(widths)
    shards = make(rows, widths, BF16, 11, gpu)
    tokens = some_tokens(rows, V, 11, gpu)
    all_rows = rog.rog_logprob(shards, tokens, 8)
    for a, b in ((0, 1), (17, 18), (100, 107), (250, 300), (0, 299)):
        part = rog.rog_logprob([s[a:b] for s in shards], tokens[a:b].contiguous(), 8)
        assert same_bits(part, [t[a:b].contiguous() for t in all_rows]), (a, b)


def test_optional_outputs(gpu):
    shards = make(4, [3000], BF16, 5, gpu)
    tokens = some_tokens(4, 3000, 5, gpu)
    want = rog.rog_logprob(shards, tokens, 3)
    no_tokens = rog.rog_logprob(shards, None, 3)
    assert no_tokens.logp is None
    scored = tokens >= 0
    assert torch.equal(no_tokens.lse[scored], want.lse[scored])
    lse = torch.empty(4, device=gpu)
    rog.rog_logprob(shards, tokens, 3, out=(None, None, lse, None, None))
    assert torch.equal(lse, want.lse)
    ids = torch.empty(4, 3, dtype=torch.int64, device=gpu)
    rog.rog_logprob(shards, tokens, 3, out=(None, None, None, None, ids))
    assert torch.equal(ids, want.top_ids)
    empty = rog.rog_logprob([torch.empty(0, 50, device=gpu)], torch.empty(0, dtype=torch.int64, device=gpu), 2)
    assert empty.top_ids.shape == (0, 2)
    none = rog.rog_logprob([torch.empty(3, 0, device=gpu)], torch.tensor([0, -1, 5], device=gpu), 2)
    assert none.lse.tolist() == [-math.inf, 0.0, -math.inf] and none.top_ids.eq(-1).all()


def test_offsets_past_32_bits(gpu):
    """Rows more than 4 GiB apart, element offsets past 2^31."""
    stride = 2 ** 31 + 77
    buf = torch.empty(2 * stride + 3000, dtype=BF16, device=gpu)
    view = torch.as_strided(buf, (3, 3000), (stride, 1))
    rows = torch.cat(make(3, [3000], BF16, 9, gpu), 1)
    view.copy_(rows)
    tokens = some_tokens(3, 3000, 9, gpu, skip=False)
    want = rog.rog_logprob([rows], tokens, 5)
    assert same_bits(want, rog.rog_logprob([view], tokens, 5))
    g = torch.randn(3, device=gpu)
    a = rog.rog_logprob_grad([rows], tokens, want.lse, want.entropy, g)[0]
    rog.rog_logprob_grad([view], tokens, want.lse, want.entropy, g, out=[view])
    assert torch.equal(a, view)


def test_very_long_rows(gpu):
    """A hundred million columns: thousands of units, wide table entries, columns past 2^26."""
    V = 100_000_003
    gen = torch.Generator(device=gpu)
    gen.manual_seed(1)
    x = torch.empty(2, V, dtype=BF16, device=gpu)
    x.normal_(0, 2, generator=gen)
    x[0, V - 1] = 40.0
    tokens = torch.tensor([V - 1, 77_777_777], device=gpu)
    got = rog.rog_logprob([x], tokens, 3)
    split = rog.rog_logprob_ex([x[:, : V // 2], x[:, V // 2:]], tokens, 3, form=rog.ROG_LOGPROB_ROW)
    for i in range(2):
        z = x[i].double()
        lse = torch.logsumexp(z, 0)
        best = torch.topk(z, 3).values
        p = torch.exp(z - lse)
        h = lse - (p * z).sum()
        # as logprob_tol, with some 2000 more additions above each term
        tol = ref.U * (6 * 40 + 2500)
        for r in (got, split):
            assert abs(float(r.lse[i]) - float(lse)) <= tol + 2 * ref.U * abs(float(lse))
            assert abs(float(r.logp[i]) - float(z[tokens[i]] - lse)) <= tol + 2 * ref.U * abs(float(r.logp[i]))
            assert abs(float(r.entropy[i]) - float(h)) <= tol * (2 + 2 * float(h))
            assert torch.equal(z[r.top_ids[i]], best)
        assert torch.equal(got.top_ids[i], split.top_ids[i])
    assert same_bits(got, rog.rog_logprob_ex([x], tokens, 3, form=rog.ROG_LOGPROB_ROW))


def test_outputs_stay_in_their_arrays(gpu):
    shards = make(5, [2500, 1], F16, 21, gpu)
    tokens = some_tokens(5, 2501, 21, gpu)
    buf = torch.full((1000,), 7.5, device=gpu)
    ids = torch.full((64,), 77, dtype=torch.int64, device=gpu)
    out = (buf[10:15], buf[20:25], buf[30:35], buf[40:60].view(5, 4), ids[8:28].view(5, 4))
    rog.rog_logprob(shards, tokens, 4, out=out)
    keep = torch.ones(1000, dtype=torch.bool, device=gpu)
    for a, b in ((10, 15), (20, 25), (30, 35), (40, 60)):
        keep[a:b] = False
    assert bool((buf[keep] == 7.5).all()) and bool((ids[:8] == 77).all()) and bool((ids[28:] == 77).all())
    grad = torch.full((5, 2600), 9.0, dtype=F16, device=gpu)
    r = rog.rog_logprob(shards, tokens)
    rog.rog_logprob_grad(shards, tokens, r.lse, r.entropy, torch.ones(5, device=gpu),
                         out=[grad[:, 3:2503], grad[:, 2510:2511]])
    assert bool((grad[:, :3] == 9).all()) and bool((grad[:, 2503:2510] == 9).all()) and bool((grad[:, 2511:] == 9).all())


def test_streams_and_shared_workspace(gpu):
    """Calls on other streams than the inputs', workspaces kept per stream, many calls in flight."""
    shards = make(3, [40000], BF16, 31, gpu)
    tokens = some_tokens(3, 40000, 31, gpu, skip=False)
    want = rog.rog_logprob(shards, tokens, 6)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for i in range(30):
        s = streams[i % 3]
        if i % 2:
            with torch.cuda.stream(s):
                outs.append(rog.rog_logprob(shards, tokens, 6))
        else:
            out = rog.RogLogprob(*[torch.empty_like(t) for t in want])
            s.wait_stream(torch.cuda.current_stream())
            outs.append(rog.rog_logprob(shards, tokens, 6, out=out, stream=s))
    torch.cuda.synchronize()
    assert all(same_bits(want, o) for o in outs)
    ws = rog.rog_workspace(64 << 20)
    for _ in range(3):
        assert same_bits(want, rog.rog_logprob(shards, tokens, 6, workspace=ws))
        assert same_bits(rog.rog_logprob([shards[0][:2]], tokens[:2].contiguous(), 2, workspace=ws),
                         [t[:2, :2].contiguous() if t.dim() == 2 else t[:2].contiguous() for t in want])


def test_graph_replays(gpu):
    shards = make(2, [40000], BF16, 41, gpu)
    tokens = some_tokens(2, 40000, 41, gpu, skip=False)
    g = torch.randn(2, device=gpu)
    rog.rog_logprob(shards, tokens, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        r = rog.rog_logprob(shards, tokens, 4)
        d = rog.rog_logprob_grad(shards, tokens, r.lse, r.entropy, g)
    for seed in range(4):
        new = make(2, [40000], BF16, 50 + seed, gpu)
        shards[0].copy_(new[0])
        graph.replay()
        torch.cuda.synchronize()
        want = rog.rog_logprob(new, tokens, 4)
        assert same_bits(want, r)
        assert torch.equal(d[0], rog.rog_logprob_grad(new, tokens, want.lse, want.entropy, g)[0])


# ---------------------------------------------------------------------------
# Gradient
# ---------------------------------------------------------------------------

def check_grad(shards, tokens, T, g, gh):
    r = rog.rog_logprob(shards, tokens, 0, T)
    got = rog.rog_logprob_grad(shards, tokens, r.lse, r.entropy, g, gh, temperature=T)
    x = ref.rows64(shards)
    want, tol = ref.grad64(x, tokens, T, r.lse, r.entropy, g.double(), gh.double() if gh is not None else torch.zeros_like(g).double())
    rel, least = ref.ROUND[shards[0].dtype]
    a = torch.cat([t.double() for t in got], 1)
    top = torch.finfo(shards[0].dtype).max
    want = want.clamp(-top, top)
    ok = (torch.isnan(a) & torch.isnan(want)) | ((a - want).abs() <= tol + rel * (want.abs() + tol) + least)
    assert bool(ok.all()), (a[~ok][:4], want[~ok][:4], tol[~ok][:4])
    return r, got


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("widths", [[1], [5], [511], [2048], [2049], [0, 7, 0], [1] * 64, [4096, 2048, 5000], [50257], [16384] * 8],
                         ids=lambda w: "+".join(map(str, w[:3])) + ("x%d" % len(w) if len(w) > 3 else ""))
def test_gradient(gpu, widths, dtype):
    V = sum(widths)
    for rows, T, ent in ((1, 1.0, True), (5, 0.7, False), (9, 1.3, True)):
        shards = make(rows, widths, dtype, V + rows, gpu)
        gen = torch.Generator(device=gpu)
        gen.manual_seed(V)
        g = torch.randn(rows, generator=gen, device=gpu)
        gh = torch.randn(rows, generator=gen, device=gpu) if ent else None
        check_grad(shards, some_tokens(rows, V, V, gpu), T, g, gh)


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
def test_gradient_masks(gpu, dtype):
    V = 4500
    x = torch.cat(make(10, [V], dtype, 77, gpu), 1)
    tokens = some_tokens(10, V, 77, gpu, skip=False)
    low = LOWEST[dtype]
    half = torch.arange(V, device=gpu) % 2 == 0
    x[0] = -math.inf
    x[1] = low                                         # uniform
    x[2, half] = -math.inf
    x[3, half] = low
    x[4] = -math.inf
    x[4, 9] = 2.0
    tokens[4] = 9
    x[5, 0] = -math.inf
    tokens[5] = 0                                      # a token that the mask forbids
    tokens[6] = -1
    x[6] = math.nan
    tokens[7] = V
    x[8, 11] = math.nan
    gen = torch.Generator(device=gpu)
    gen.manual_seed(5)
    g, gh = (torch.randn(10, generator=gen, device=gpu) for _ in range(2))
    r, got = check_grad([x], tokens, 1.0, g, gh)
    assert bool((got[0][0] == 0).all()) and bool((got[0][6] == 0).all())
    # in place, and into column slices of one matrix
    y = x.clone()
    rog.rog_logprob_grad([y], tokens, r.lse, r.entropy, g, gh, out=[y])
    assert torch.equal(y.view(torch.uint8), got[0].view(torch.uint8))
    parts = [x[:, :2000].contiguous(), x[:, 2000:].contiguous()]
    whole = torch.zeros_like(x)
    rog.rog_logprob_grad(parts, tokens, r.lse, r.entropy, g, gh, out=[whole[:, :2000], whole[:, 2000:]])
    assert torch.equal(whole.view(torch.uint8), got[0].view(torch.uint8))


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
def test_gradient_at_every_place_of_a_line(gpu, dtype):
    """Rows that begin anywhere in a 128-byte line, with pieces that end anywhere: the same bits, nothing beside them, in place too."""
    size = 4 if dtype is F32 else 2
    piece, line = 2048 // size, 128 // size
    rows = 3
    gen = torch.Generator(device=gpu)
    gen.manual_seed(9)
    g, gh = (torch.randn(rows, generator=gen, device=gpu) for _ in range(2))
    for width in (1, line - 1, piece - line + 1, piece - 1, piece + 2, 2 * piece + 5):
        x = make(rows, [width], dtype, width, gpu)[0]
        tokens = some_tokens(rows, width, width, gpu)
        r = rog.rog_logprob([x], tokens)
        want = rog.rog_logprob_grad([x], tokens, r.lse, r.entropy, g, gh)[0]
        stride = width + 3 + line // 2
        for offset in range(0, line + 1):
            buf = torch.full((rows * stride + 2 * line,), 7.0, dtype=dtype, device=gpu)
            view = torch.as_strided(buf, (rows, width), (stride, 1), offset)
            rog.rog_logprob_grad([x], tokens, r.lse, r.entropy, g, gh, out=[view])
            assert torch.equal(view.contiguous().view(torch.uint8), want.view(torch.uint8)), (width, offset)
            view.fill_(7.0)
            assert bool((buf == 7.0).all()), (width, offset)
            view.copy_(x)
            rog.rog_logprob_grad([view], tokens, r.lse, r.entropy, g, gh, out=[view])
            assert torch.equal(view.contiguous().view(torch.uint8), want.view(torch.uint8)), (width, offset)
            view.fill_(7.0)
            assert bool((buf == 7.0).all()), (width, offset)


def test_gradient_against_differences(gpu):
    """Central differences of the kernel's own log probability and entropy."""
    V, rows, T, h = 301, 3, 0.8, 2.0 ** -4
    x = torch.cat(make(rows, [V], F32, 13, gpu, spread=1.0), 1)
    tokens = torch.tensor([0, 150, 300], device=gpu)
    g, gh = torch.tensor([1.0, -2.0, 0.5], device=gpu), torch.tensor([0.3, 0.0, -1.0], device=gpu)
    r = rog.rog_logprob([x], tokens, 0, T)
    got = rog.rog_logprob_grad([x], tokens, r.lse, r.entropy, g, gh, temperature=T)[0]
    cols = torch.arange(V, device=gpu)

    def value(step):
        y = x[:, None, :].repeat(1, V, 1)
        y[:, cols, cols] += step
        s = rog.rog_logprob([y.view(-1, V)], tokens.repeat_interleave(V), 0, T)
        return g[:, None].double() * s.logp.view(rows, V).double() + gh[:, None].double() * s.entropy.view(rows, V).double()

    diff = (value(h) - value(-h)) / (2 * h)
    # truncation: h^2 / 6 times a third derivative, below (|g| + |gh| (2 + log V)) p / T^3; noise: two
    # binary32 values of size up to log V + max |z| over 2 h
    p = torch.softmax(x.double() / T, 1)
    size = g.abs()[:, None].double() + gh.abs()[:, None].double() * (2 + math.log(V))
    tol = h * h / 6 * 8 * size * p / T ** 3 + 2 * ref.U * 150 * size / (2 * h)
    assert bool(((got.double() - diff).abs() <= tol).all())


def test_refusals_of_tensors(gpu):
    x = torch.zeros(4, 100, device=gpu)
    t = torch.zeros(4, dtype=torch.int64, device=gpu)
    v = torch.zeros(4, device=gpu)
    bad = [lambda: rog.rog_logprob([], t), lambda: rog.rog_logprob([x.double()], t), lambda: rog.rog_logprob([x.cpu()], t),
           lambda: rog.rog_logprob([x, x[:3]], t), lambda: rog.rog_logprob([x, x.bfloat16()], t),
           lambda: rog.rog_logprob([x.t()], t), lambda: rog.rog_logprob([x[0]], t),
           lambda: rog.rog_logprob([x], t.int()), lambda: rog.rog_logprob([x], t[:3]),
           lambda: rog.rog_logprob([x], t, 33), lambda: rog.rog_logprob([x], t, -1),
           lambda: rog.rog_logprob([x], t, temperature=0.0), lambda: rog.rog_logprob([x], t, temperature=math.nan),
           lambda: rog.rog_logprob([x], t, 2, out=(v, v[:3], None, None, None)),
           lambda: rog.rog_logprob([x], t, out=(v, v, None, None, None)),
           lambda: rog.rog_logprob([x], None, out=(v, None, None, None, None)),
           lambda: rog.rog_logprob([x], t, out=(x.view(-1)[:4], None, None, None, None)),
           lambda: rog.rog_logprob_grad([x], t, v, v, None), lambda: rog.rog_logprob_grad([x], t, v, v, v, out=[x[:, :99]]),
           lambda: rog.rog_logprob_grad([x], t, v, v, v, out=[]),
           lambda: rog.rog_logprob_grad([x], t, v, v, v, out=[x.view(-1)[:100].expand(4, 100)])]
    for i, f in enumerate(bad):
        with pytest.raises((ValueError, TypeError)):
            f()
            pytest.fail("case %d was accepted" % i)
