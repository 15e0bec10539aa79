"""Calls of training size and beyond: logits past 128 MiB, whose loads are
streamed by kernels of their own, and launches of more than 2^22 workgroups,
whose grid has a second dimension.  A row's bits do not depend on its call, so
the same rows in smaller calls are the reference; a few are held to the formula."""
from __future__ import annotations

import pytest
import torch

from deterministic_collective_movement_amd import rog
from tests import head_ref as ref

pytestmark = pytest.mark.gpu

BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
STREAMED_FROM = 128 << 20
GROUPS_OF_A_GRID_ROW = 1 << 22


def same_bits(a, b):
    return all((x is None and y is None) or torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def make(rows, widths, dtype, gpu):
    gen = torch.Generator(device=gpu)
    gen.manual_seed(rows + sum(widths))
    shards = [torch.randn(rows, w, generator=gen, device=gpu, dtype=dtype).mul_(2.5) for w in widths]
    tokens = torch.randint(0, sum(widths), (rows,), generator=gen, device=gpu)
    tokens[rows // 3::101] = -1
    g, h = (torch.randn(rows, generator=gen, device=gpu) for _ in range(2))
    return shards, tokens, g, h


@pytest.mark.parametrize("dtype", [BF16, F16, F32], ids=["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,widths", [(8200, [8192]), (8300, [4095, 4096]), (4100, [16411]), (4200, [8001, 0, 8001])], ids=str)
def test_streamed_logits(gpu, rows, widths, dtype):
    """Streamed and not, with and without alternatives, and the gradient, apart and in place: the same bits."""
    V, T = sum(widths), 0.8
    shards, tokens, g, h = make(rows, widths, dtype, gpu)
    size = V * shards[0].element_size()
    assert rows * size >= STREAMED_FROM
    step = rows // 3 + 1
    assert step * size < STREAMED_FROM
    parts = [(a, min(rows, a + step)) for a in range(0, rows, step)]
    for k in (0, 5):
        whole = rog.rog_logprob(shards, tokens, k, T)
        for a, b in parts:
            part = rog.rog_logprob([s[a:b] for s in shards], tokens[a:b], k, T)
            assert same_bits(part, [t if t is None else t[a:b].contiguous() for t in whole]), (k, a)
    grads = rog.rog_logprob_grad(shards, tokens, whole.lse, whole.entropy, g, h, temperature=T)
    for a, b in parts:
        part = rog.rog_logprob_grad([s[a:b] for s in shards], tokens[a:b], whole.lse[a:b], whole.entropy[a:b], g[a:b], h[a:b],
                                    temperature=T)
        assert same_bits(part, [t[a:b] for t in grads]), a
    # a few rows against the formula
    some = torch.tensor([0, 1, rows // 2, rows - 2, rows - 1], device=gpu)
    x = ref.rows64([s[some] for s in shards])
    logp, entropy, lse, top_logp, top_ids = ref.logprob64(x, tokens[some], T, 5)
    tol, tol_h = ref.logprob_tol(x, T, entropy)
    assert torch.equal(whole.top_ids[some], top_ids)
    for got, want, t in ((whole.logp, logp, tol), (whole.lse, lse, tol), (whole.entropy, entropy, tol_h),
                         (whole.top_logp, top_logp, tol[:, None])):
        assert bool(((got[some].double() - want).abs() <= t + 2 * ref.U * want.abs()).all())
    want, tol = ref.grad64(x, tokens[some], T, whole.lse[some], whole.entropy[some], g[some].double(), h[some].double())
    rel, least = ref.ROUND[dtype]
    got = torch.cat([t[some].double() for t in grads], 1)
    assert bool(((got - want).abs() <= tol + rel * (want.abs() + tol) + least).all())
    rog.rog_logprob_grad(shards, tokens, whole.lse, whole.entropy, g, h, temperature=T, out=shards)
    assert same_bits(shards, grads)


@pytest.mark.parametrize("form,rows,widths", [("row", GROUPS_OF_A_GRID_ROW + 70001, [1] * 5),
                                              ("wave", 4 * GROUPS_OF_A_GRID_ROW + 70003, [2, 1])], ids=["row", "wave"])
def test_more_workgroups_than_a_grid_row(gpu, form, rows, widths):
    shards, tokens, _, _ = make(rows, widths, BF16, gpu)
    plan = rog.rog_logprob_plan(shards)
    assert plan["form"] == form and plan["grid"] > GROUPS_OF_A_GRID_ROW
    parts = [(0, 70003), (rows // 2, rows // 2 + 70001), (rows - 80000, rows)]
    for k in (0, 2):
        whole = rog.rog_logprob(shards, tokens, k)
        for a, b in parts:
            part = rog.rog_logprob([s[a:b] for s in shards], tokens[a:b], k)
            assert same_bits(part, [t if t is None else t[a:b].contiguous() for t in whole]), (k, a)
        # every row was written: log-sum-exp of a few columns, in binary32 (2^-7 is a thousand times its roundings)
        x = torch.cat(shards, 1).float()
        want = torch.where(tokens < 0, 0.0, torch.logsumexp(x, 1))
        assert bool(((whole.lse - want).abs() <= 2.0 ** -7).all())


def test_more_gradient_pieces_than_a_grid_row(gpu):
    rows, V = GROUPS_OF_A_GRID_ROW + 130003, 3
    shards, tokens, g, h = make(rows, [V], F32, gpu)
    r = rog.rog_logprob(shards, tokens)
    out = [torch.full((rows, V), 7.0, device=gpu)]
    rog.rog_logprob_grad(shards, tokens, r.lse, r.entropy, g, h, out=out)
    for a, b in ((0, 60001), (rows // 2, rows // 2 + 60001), (rows - 140000, rows)):
        part = rog.rog_logprob_grad([shards[0][a:b]], tokens[a:b], r.lse[a:b], r.entropy[a:b], g[a:b], h[a:b])
        assert torch.equal(part[0], out[0][a:b])
    # the gradient of a row sums to 0: three binary32 numbers of up to |g| + 3 |h|
    assert bool((out[0].double().sum(1).abs() <= 64 * ref.U * (1 + g.double().abs() + 3 * h.double().abs())).all())


def test_more_split_workgroups_than_a_grid_row(gpu):
    """One row of 33.6 million columns, read as 1024 rows (row stride 0): 4097 units each."""
    V, rows = 16385 * 2048 - 5, rog.rog_logprob_max_split_rows()
    gen = torch.Generator(device=gpu)
    gen.manual_seed(3)
    x = torch.empty(1, V, dtype=BF16, device=gpu).normal_(0, 2, generator=gen)
    many = x.expand(rows, V)
    tokens = torch.full((rows,), V - 1, device=gpu)
    info = rog.rog_logprob_plan_widths([V], rows, rog.ROG_DTYPE_BF16, 0, rog.ROG_LOGPROB_SPLIT)
    assert info["grid"] == rows * 4097 > GROUPS_OF_A_GRID_ROW
    ws = rog.rog_workspace(info["workspace_bytes"])
    one = rog.rog_logprob_ex([x], tokens[:1], 0, form=rog.ROG_LOGPROB_ROW)
    got = rog.rog_logprob_ex([many], tokens, 0, workspace=ws, form=rog.ROG_LOGPROB_SPLIT)
    for a, b in zip(got[:3], one[:3]):
        assert bool((a == b).all())
