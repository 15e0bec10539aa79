"""The vocabulary-side operators' C interface on the CPU: validation, launch
forms, workspaces (include/rog.h).  No test here launches a kernel: every call
fails validation, has nothing to do, or only plans."""
from __future__ import annotations

import ctypes
import math
import struct

import pytest
import torch

from deterministic_collective_movement_amd import rog

A = 1 << 30                  # a 16-byte aligned fake device address
BIG = 1 << 40
F32, BF16, F16 = rog.ROG_DTYPE_F32, rog.ROG_DTYPE_BF16, rog.ROG_DTYPE_F16
OK, INVALID, OVERLAP, TOO_LARGE = (rog.ROG_OK, rog.ROG_ERR_INVALID_ARGUMENT, rog.ROG_ERR_OVERLAP, rog.ROG_ERR_TOO_LARGE)
WS = 1 << 44


def shards(*triples):
    return struct.pack("=" + "Qqq" * len(triples), *(v for t in triples for v in t))


def logprob(sh, W=1, rows=4, dtype=BF16, T=1.0, tokens=BIG, k=0, out=(BIG + 4096, BIG + 8192, BIG + 12288, 0, 0), ws=WS,
            ws_bytes=1 << 30, form=0):
    """Status of a call whose validation fails (asserted: these addresses are never launched on)."""
    packed = struct.pack("=5Q", *out) if out is not None else None
    st = rog.lib().rog_logprob_ex(sh, W, rows, dtype, T, tokens or None, k, packed, ws or None, ws_bytes, None, form)
    assert st != OK or rows == 0
    return st


def grad(sh, gr, W=1, rows=4, dtype=BF16, T=1.0, tokens=BIG, lse=BIG + 4096, ent=BIG + 8192, g=BIG + 12288, gh=0):
    packed = struct.pack("=" + "Qq" * (len(gr) // 2), *gr) if gr is not None else None
    st = rog.lib().rog_logprob_grad(sh, packed, W, rows, dtype, T, tokens or None, lse or None, ent or None, g or None, gh or None, None)
    assert st != OK or rows == 0
    return st


def loss(ins, n, params=(0.2, 0.2, 0.0, 0.0, 1.0), outs=(BIG, 0, 0), ws=0, ws_bytes=0):
    st = rog.lib().rog_policy_loss(struct.pack("=6Q", *ins), n, struct.pack("=5f", *params), struct.pack("=3Q", *outs),
                                   ws or None, ws_bytes, None)
    assert st != OK
    return st


def test_constants():
    assert rog.rog_max_top_k() == 32
    assert rog.rog_logprob_max_split_rows() >= 176
    assert rog.rog_policy_loss_workspace_bytes(0) == 0
    assert rog.rog_policy_loss_workspace_bytes(1024) == 0
    assert 0 < rog.rog_policy_loss_workspace_bytes(1025) <= rog.rog_policy_loss_workspace_bytes(1 << 33) < 1 << 21


GOOD = shards((A, 1000, 1000))


def test_logprob_arguments():
    bad = 5 * A
    assert logprob(None) == INVALID
    assert logprob(GOOD, W=0) == INVALID and logprob(GOOD, W=65) == INVALID
    assert logprob(GOOD, dtype=3) == INVALID and logprob(GOOD, dtype=-1) == INVALID
    for T in (0.0, -1.0, math.nan, math.inf, 2.0 ** -11, 2048.0):
        assert logprob(GOOD, T=T) == INVALID
    assert logprob(GOOD, k=-1) == INVALID and logprob(GOOD, k=33) == INVALID
    assert logprob(GOOD, form=4) == INVALID and logprob(GOOD, form=-1) == INVALID
    assert logprob(GOOD, out=None) == INVALID
    assert logprob(GOOD, tokens=0) == INVALID                       # logp wanted, no tokens
    assert logprob(GOOD, tokens=BIG + 4) == INVALID                 # misaligned
    assert logprob(GOOD, out=(BIG + 4098, 0, 0, 0, 0)) == INVALID
    assert logprob(GOOD, k=2, out=(0, 0, 0, 0, bad + 4)) == INVALID
    assert logprob(shards((A + 1, 1000, 1000))) == INVALID          # odd address of 2-byte logits
    assert logprob(shards((A + 2, 1000, 1000)), dtype=F32) == INVALID
    assert logprob(shards((0, 1000, 1000))) == INVALID
    assert logprob(shards((A, -1, 1000))) == INVALID and logprob(shards((A, 1000, -1))) == INVALID
    assert logprob(GOOD, rows=0) == OK


def test_logprob_sizes():
    assert logprob(shards((A, 1 << 31, 1 << 31))) == TOO_LARGE
    assert logprob(shards((A, 1 << 30, 1 << 30), (A, 1 << 30, 1 << 30)), W=2) == TOO_LARGE
    assert logprob(GOOD, rows=1 << 31) == TOO_LARGE
    assert logprob(shards((A, 1 << 50, 1000))) == TOO_LARGE
    assert logprob(shards((A, (1 << 48) - 1, 1000)), rows=1 << 30) == TOO_LARGE


def test_logprob_overlaps():
    assert logprob(GOOD, out=(A + 400, 0, 0, 0, 0)) == OVERLAP                       # into the logits
    assert logprob(GOOD, out=(A - 8, 0, 0, 0, 0)) == OVERLAP
    assert logprob(GOOD, out=(BIG + 16, 0, 0, 0, 0)) == OVERLAP                      # into the tokens
    assert logprob(GOOD, out=(BIG + 4096, BIG + 4108, 0, 0, 0)) == OVERLAP           # into each other
    assert logprob(GOOD, k=4, out=(BIG + 4096, 0, 0, BIG + 4112 - 64, 0)) == OVERLAP
    long_rows = shards((A, 131072, 131072))
    assert logprob(long_rows, out=(WS + 64, 0, 0, 0, 0)) == OVERLAP                  # into the workspace


def test_logprob_workspace():
    long_rows = shards((A, 131072, 131072))
    need = rog.rog_logprob_plan_widths([131072], 4, BF16, 0)
    assert need["form"] == "split" and need["workspace_bytes"] > 0
    assert logprob(long_rows, ws=0, ws_bytes=0) == INVALID
    assert logprob(long_rows, ws_bytes=need["workspace_bytes"] - 1) == INVALID
    assert logprob(long_rows, ws=WS + 8) == INVALID


def test_forms():
    plan = rog.rog_logprob_plan_widths
    for widths, rows, form in (([1], 1, "wave"), ([8192], 100000, "wave"), ([2048] * 4, 5, "wave"), ([2048] * 5, 5, "split"),
                               ([131072], 1, "split"), ([131072], 232, "split"), ([131072], 233, "row"), ([10000], 4096, "row"),
                               ([500] * 64, 3, "split"), ([0, 0], 3, "wave")):
        p = plan(widths, rows, BF16)
        assert p["form"] == form, (widths, rows, p)
        assert (p["workspace_bytes"] > 0) == (form == "split")
    for rows, form in ((1, "split"), (167, "split"), (168, "row")):      # alternatives cost a split row more
        assert plan([131072], rows, BF16, 8)["form"] == form
    assert plan([131072], 0, BF16)["form"] == "none"
    # a row's blocks follow its shards' widths, not the type
    assert plan([2049, 1], 3, BF16)["blocks"] == plan([2049, 1], 3, F32)["blocks"] == 3
    for widths, form in (([8192], rog.ROG_LOGPROB_ROW), ([8192], rog.ROG_LOGPROB_SPLIT), ([8193], rog.ROG_LOGPROB_WAVE)):
        with pytest.raises(rog.RogArgumentError) as e:
            plan(widths, 4, BF16, 0, form)
        assert e.value.status == INVALID
    with pytest.raises(rog.RogArgumentError):
        plan([131072], rog.rog_logprob_max_split_rows() + 1, BF16, 0, rog.ROG_LOGPROB_SPLIT)
    assert rog.lib().rog_logprob_plan(GOOD, 1, 4, BF16, 0, 0, None) == INVALID


@pytest.mark.parametrize("seed", range(40))
def test_split_work_covers_every_block_once(seed):
    """Units of a row: every block belongs to one, and a split launch has one workgroup per unit with blocks."""
    import random
    r = random.Random(seed)
    widths = [r.choice([0, 1, 500, 2048, 2049, 30000, 131072]) for _ in range(r.randint(1, 64))]
    blocks = sum(-(-w // 2048) for w in widths)
    rows = r.randint(1, 100)
    p = rog.rog_logprob_plan_widths(widths, rows, BF16)
    assert p["blocks"] == blocks
    if blocks <= 4:
        assert p["form"] == "wave"
        return
    owned = {}
    for unit in range(4 * -(-blocks // 16)):
        for i in range(4):
            b = unit // 4 * 16 + i * 4 + unit % 4
            if b < blocks:
                owned.setdefault(unit, []).append(b)
    assert sorted(b for v in owned.values() for b in v) == list(range(blocks))
    assert sorted(owned) == list(range(len(owned)))          # units without blocks come last
    forced = rog.rog_logprob_plan_widths(widths, rows, BF16, 0, rog.ROG_LOGPROB_SPLIT)
    assert forced["grid"] == rows * len(owned)


def test_gradient_arguments():
    far = 3 * A
    assert grad(None, (far, 1000)) == INVALID and grad(GOOD, None) == INVALID
    assert grad(GOOD, (0, 1000)) == INVALID and grad(GOOD, (far + 1, 1000)) == INVALID
    assert grad(GOOD, (far, 999)) == INVALID and grad(GOOD, (far, -1)) == INVALID
    for miss in ("tokens", "lse", "ent", "g"):
        assert grad(GOOD, (far, 1000), **{miss: 0}) == INVALID
    assert grad(GOOD, (far, 1000), gh=BIG + 2) == INVALID
    assert grad(GOOD, (far, 1000), T=0.0) == INVALID
    assert grad(GOOD, (far, 1 << 50)) == TOO_LARGE
    assert grad(GOOD, (A + 2, 1000)) == OVERLAP                        # not exactly in place
    assert grad(GOOD, (A, 1001)) == OVERLAP                            # another stride
    assert grad(GOOD, (BIG - 100, 1000)) == OVERLAP                    # over the tokens
    two = shards((A, 2000, 1000), (A + 2000, 2000, 1000))              # column slices of one matrix
    assert grad(two, (far, 1000, far + 100, 1000), W=2) == OVERLAP     # the gradients overlap each other
    assert grad(two, (A + 2000, 2000, A, 2000), W=2) == OVERLAP        # each in the other's place
    assert grad(GOOD, (far, 1000), rows=0) == OK


def test_policy_loss_arguments():
    n = 100
    good = (A, A + 4096, A + 8192, 0, 0, 0)
    assert loss((0, A, A, 0, 0, 0), n) == INVALID and loss((A, 0, A, 0, 0, 0), n) == INVALID
    assert loss((A, A + 4096, 0, 0, 0, 0), n) == INVALID
    assert loss((A + 2, A + 4096, A + 8192, 0, 0, 0), n) == INVALID
    assert loss(good, n, outs=(0, 0, 0)) == INVALID
    assert loss(good, n, outs=(BIG + 1, 0, 0)) == INVALID
    assert loss(good, n, outs=(BIG, 0, BIG + 64)) == INVALID           # a gradient of an entropy that is not there
    for params in ((1.5, 0.2, 0, 0, 1), (-0.1, 0.2, 0, 0, 1), (0.2, -0.2, 0, 0, 1), (0.2, math.nan, 0, 0, 1),
                   (0.2, 0.2, math.inf, 0, 1), (0.2, 0.2, 0, math.nan, 1), (0.2, 0.2, 0, 0, math.inf)):
        assert loss(good, n, params) == INVALID, params
    assert loss(good, n, outs=(A + 8, 0, 0)) == OVERLAP
    assert loss(good, n, outs=(BIG, A + 8, 0)) == OVERLAP              # partly over an input
    assert loss(good, n, outs=(BIG, BIG + 8, 0)) == OVERLAP            # over the stats
    assert loss(good, 1 << 34) == TOO_LARGE
    assert loss(good, 5000) == INVALID                                 # needs a workspace
    need = rog.rog_policy_loss_workspace_bytes(5000)
    assert loss((A, A + (1 << 20), A + (1 << 21), 0, 0, 0), 5000, ws=WS, ws_bytes=need - 1) == INVALID
    assert loss((A, A + (1 << 20), A + (1 << 21), 0, 0, 0), 5000, ws=WS + 4, ws_bytes=1 << 30) == INVALID
    assert rog.lib().rog_policy_loss(None, 1, None, None, None, 0, None) == INVALID


def test_binding_refuses_host_tensors():
    x, t, v = torch.zeros(4, 10), torch.zeros(4, dtype=torch.int64), torch.zeros(4)
    for call in (lambda: rog.rog_logprob([x], t), lambda: rog.rog_logprob_grad([x], t, v, v, v),
                 lambda: rog.rog_policy_loss(v, v, v)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        rog.rog_logprob([], t)
    with pytest.raises(TypeError):
        rog.rog_logprob([None], t)
    with pytest.raises(TypeError):
        rog.rog_policy_loss(None, v, v)


def test_plan_makes_no_hip_call_for_bad_forms():
    assert rog.lib().rog_logprob_plan(GOOD, 1, 4, 9, 0, 0, ctypes.byref(rog.rog_head_plan_info())) == INVALID
    assert rog.rog_last_hip_error() == 0
