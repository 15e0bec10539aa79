"""The head's products' C interface on the CPU: validation, tiles, workspaces
(include/rog.h).  No test here launches a kernel: every call fails validation,
has nothing to do, or only plans."""
from __future__ import annotations

import math
import struct

import pytest
import torch

from deterministic_collective_movement_amd import rog

A, B, BIG, WS = 1 << 32, 1 << 36, 1 << 40, 1 << 44     # fake device addresses, 16-byte aligned
F32, BF16, F16 = rog.ROG_DTYPE_F32, rog.ROG_DTYPE_BF16, rog.ROG_DTYPE_F16
OK, INVALID, OVERLAP, TOO_LARGE = (rog.ROG_OK, rog.ROG_ERR_INVALID_ARGUMENT, rog.ROG_ERR_OVERLAP, rog.ROG_ERR_TOO_LARGE)


def shards(*triples):
    return struct.pack("=" + "Qqq" * len(triples), *(v for t in triples for v in t))


def score(h=A, h_stride=64, rows=4, dim=64, sh=shards((B, 64, 1000)), W=1, dtype=BF16, T=1.0, tokens=BIG,
          out=(BIG + 4096, BIG + 8192, BIG + 12288, 0, 0), ws=WS, ws_bytes=1 << 40):
    st = rog.lib().rog_linear_logprob(h or None, h_stride, rows, dim, sh, W, dtype, T, tokens or None,
                                      struct.pack("=5Q", *out) if out is not None else None, ws or None, ws_bytes, None)
    assert st != OK or rows == 0
    return st


def grad(h=A, h_stride=64, rows=4, dim=64, sh=shards((B, 64, 1000)), W=1, dtype=BF16, T=1.0, tokens=BIG, lse=BIG + 4096, ent=BIG + 8192,
         g=BIG + 12288, gh=0, dh=BIG + (1 << 20), dh_stride=64, dw=(BIG + (1 << 24), 64), ws=WS, ws_bytes=1 << 40):
    st = rog.lib().rog_linear_logprob_grad(h or None, h_stride, rows, dim, sh, W, dtype, T, tokens or None, lse or None, ent or None,
                                           g or None, gh or None, dh or None, dh_stride,
                                           struct.pack("=" + "Qq" * (len(dw) // 2), *dw) if dw is not None else None, ws or None, ws_bytes, None)
    assert st != OK or rows == 0
    return st


def quantize(x=A, stride=64, rows=4, dim=64, dtype=BF16, q=B, q_stride=64, scale=BIG):
    st = rog.lib().rog_quantize_i8(x or None, stride, rows, dim, dtype, q or None, q_stride, scale or None, None)
    assert st != OK or rows == 0
    return st


def i8(q=A, q_stride=64, scale=BIG, rows=4, dim=64, sh=(B, 64, 1000, BIG + 4096), W=1, dtype=BF16, out=(BIG + (1 << 20), 1000)):
    st = rog.lib().rog_linear_i8(q or None, q_stride, scale or None, rows, dim, struct.pack("=" + "QqqQ" * (len(sh) // 4), *sh) if sh else None,
                                 W, dtype, struct.pack("=" + "Qq" * (len(out) // 2), *out) if out else None, None)
    assert st != OK or rows == 0
    return st


def test_score_arguments():
    assert score(rows=0) == OK
    assert score(rows=0, h=0, tokens=0, ws=0) == OK
    for bad in (dict(h=0), dict(h=A + 1), dict(h_stride=-1), dict(sh=None), dict(W=0), dict(W=65), dict(dtype=F32), dict(dtype=3), dict(T=0.0),
                dict(T=math.nan), dict(T=2000.0), dict(dim=0), dict(dim=-1), dict(out=None), dict(tokens=0), dict(tokens=BIG + 4),
                dict(out=(BIG + 4098, 0, 0, 0, 0)), dict(out=(BIG + 4096, 0, 0, BIG + 8192, 0)), dict(out=(0, 0, 0, 0, BIG + 8192)),
                dict(ws=0), dict(ws=WS + 8), dict(ws_bytes=1000), dict(sh=shards((0, 64, 10))), dict(sh=shards((B + 1, 64, 10))),
                dict(sh=shards((B, -1, 10))), dict(sh=shards((B, 64, -1)))):
        assert score(**bad) == INVALID, bad
    for bad in (dict(dim=1 << 17), dict(h_stride=1 << 21), dict(sh=shards((B, 1 << 21, 10))), dict(rows=1 << 31),
                dict(sh=shards((B, 64, 1 << 31))), dict(rows=1 << 26, sh=shards((B, 64, 1 << 20))), dict(h=(1 << 64) - 64)):
        assert score(**bad) == TOO_LARGE, bad
    for bad in (dict(out=(A, 0, 0, 0, 0)), dict(out=(B + 128 * 999, 0, 0, 0, 0)), dict(out=(BIG, 0, 0, 0, 0)), dict(out=(WS, 0, 0, 0, 0)),
                dict(out=(BIG + 4096, BIG + 4104, 0, 0, 0)), dict(ws=A - 4096), dict(ws=BIG - 4096)):
        assert score(**bad) == OVERLAP, bad


def test_grad_arguments():
    assert grad(rows=0) == OK
    for bad in (dict(h=0), dict(sh=None), dict(dtype=F32), dict(T=0.0), dict(tokens=0), dict(lse=0), dict(ent=0), dict(g=0), dict(gh=BIG + 2),
                dict(lse=BIG + 4097), dict(dh=0), dict(dh=BIG + 1), dict(dh_stride=63), dict(dw=None), dict(dw=(0, 64)), dict(dw=(BIG + 1, 64)),
                dict(dw=(BIG + (1 << 24), 63)), dict(ws=0), dict(ws_bytes=4096), dict(sh=shards((B, 64, 0))), dict(dim=0)):
        assert grad(**bad) == INVALID, bad
    for bad in (dict(dim=1 << 17), dict(dh_stride=1 << 21), dict(dw=(BIG + (1 << 24), 1 << 21)), dict(rows=1 << 31)):
        assert grad(**bad) == TOO_LARGE, bad
    for bad in (dict(dh=A), dict(dh=B + 64), dict(dw=(B, 64)), dict(dw=(A, 64)), dict(dh=BIG), dict(dw=(BIG, 64)), dict(dw=(WS, 64)), dict(dh=WS),
                dict(ws=B), dict(dh=BIG + (1 << 24))):
        assert grad(**bad) == OVERLAP, bad
    # two shards' gradients on one another
    two = shards((B, 64, 100), (B + (1 << 20), 64, 100))
    assert grad(sh=two, W=2, dw=(BIG + (1 << 24), 64, BIG + (1 << 24) + 64, 64)) == OVERLAP


def test_quantize_arguments():
    assert quantize(rows=0) == OK
    for bad in (dict(x=0), dict(x=A + 1), dict(stride=-1), dict(dim=0), dict(dtype=5), dict(q=0), dict(q_stride=63), dict(scale=0), dict(scale=BIG + 2)):
        assert quantize(**bad) == INVALID, bad
    for bad in (dict(rows=1 << 23), dict(dim=1 << 17), dict(stride=1 << 22), dict(q_stride=1 << 22)):
        assert quantize(**bad) == TOO_LARGE, bad
    for bad in (dict(q=A + 100), dict(scale=A), dict(scale=B)):
        assert quantize(**bad) == OVERLAP, bad


def test_i8_arguments():
    assert i8(rows=0) == OK
    for bad in (dict(q=0), dict(q_stride=-1), dict(scale=0), dict(scale=BIG + 1), dict(sh=None), dict(W=0), dict(W=65), dict(dim=0), dict(dtype=4),
                dict(out=None), dict(out=(0, 1000)), dict(out=(BIG + (1 << 20) + 1, 1000)), dict(out=(BIG + (1 << 20), 999)),
                dict(sh=(B, 64, 1000, 0)), dict(sh=(0, 64, 1000, BIG + 4096)), dict(sh=(B, 64, 1000, BIG + 4097))):
        assert i8(**bad) == INVALID, bad
    for bad in (dict(dim=1 << 17), dict(q_stride=1 << 22), dict(rows=1 << 31), dict(out=(BIG + (1 << 20), 1 << 48))):
        assert i8(**bad) == TOO_LARGE, bad
    for bad in (dict(out=(A, 1000)), dict(out=(B, 1000)), dict(out=(BIG, 1000)), dict(out=(BIG + 4096, 1000))):
        assert i8(**bad) == OVERLAP, bad


def test_the_largest_sum_fits():
    assert ((1 << 17) - 1) * 128 * 128 < 1 << 31          # dim is below 2^17


def test_plans():
    p = rog.rog_linear_logprob_plan
    assert p([16384] * 8, 0, 4096) == {"tile": (0, 0), "pieces": 0, "launches": 0, "workspace_bytes": 0}
    assert p([16384] * 8, 1, 4096)["tile"] == (128, 32) and p([16384] * 8, 33, 4096)["tile"] == (128, 64)
    assert p([16384] * 8, 100, 4096)["tile"] == (128, 128) and p([16384] * 8, 129, 4096)["tile"] == (256, 256)
    assert p([8000], 300, 4096)["tile"] == (128, 128)     # few tiles
    assert p([100], 10, 64)["launches"] == 2 and p([100], 100, 64)["launches"] == 3 and p([100], 100, 64, tokens=False)["launches"] == 2
    assert p([0], 3, 64)["launches"] == 1
    # states of a block of 128 columns per row, and the packed rows: no logits
    for rows in (1, 64, 500, 8192):
        assert p([131072], rows, 4096)["workspace_bytes"] < (1 << 18) + (rows + 16) * (1024 * 16 + 8192 + 64)
    g = rog.rog_linear_logprob_grad_plan
    assert g([1000], 0, 64)["launches"] == 0
    assert g([32003], 33, 1024)["pieces"] == 1
    big = g([16384] * 8, 8192, 4096)
    assert big["pieces"] >= 8 and big["launches"] == 1 + 2 * big["pieces"]
    assert big["workspace_bytes"] < 8192 * (8192 * 2 + 4096 * 6 + 1024) + (1 << 28)      # one segment's coefficients, not the vocabulary's
    for widths in ([5], [300, 0, 1], [50257], [4000] * 8, [131072]):
        for rows in (1, 64, 65, 1000, 5000):
            for dim in (1, 64, 1600, 5120):
                a, b = g(widths, rows, dim), g(widths, rows, dim, F16)
                assert a["pieces"] == b["pieces"] >= 1 and a["workspace_bytes"] <= b["workspace_bytes"]
    with pytest.raises(rog.RogArgumentError):
        g([0], 3, 64)
    with pytest.raises(rog.RogArgumentError):
        p([100], 3, 64, dtype=F32)


def test_pieces_are_whole_segments_and_cover_the_head():
    # the widths decide the segments, rows only how many of them a piece holds
    one = rog.rog_linear_logprob_grad_plan([131072], 64, 4096)["pieces"]
    many = [rog.rog_linear_logprob_grad_plan([131072], rows, 4096)["pieces"] for rows in (1000, 4096, 8192, 100000)]
    assert one == 1 and many == sorted(many) and many[-1] == 16


def test_binding_refuses_before_the_library():
    cpu = torch.zeros(3, 8, dtype=torch.bfloat16)
    for call in (lambda: rog.rog_linear_logprob(cpu, [cpu]), lambda: rog.rog_linear_logprob(cpu.float(), [cpu.float()]),
                 lambda: rog.rog_quantize_i8(cpu), lambda: rog.rog_linear_i8(cpu.char(), torch.zeros(3), [cpu.char()], [torch.zeros(3)]),
                 lambda: rog.rog_linear_logprob_grad(cpu, [cpu], torch.zeros(3).long(), torch.zeros(3), torch.zeros(3), torch.zeros(3))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(TypeError):
        rog.rog_linear_logprob([1], [cpu])
    with pytest.raises(TypeError):
        rog.rog_quantize_i8(None)
