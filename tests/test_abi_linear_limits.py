"""What the head's products refuse because a launch could not hold it, on the CPU."""
from __future__ import annotations

import pytest

from deterministic_collective_movement_amd import rog
from tests.test_abi_linear import OK, TOO_LARGE, score, shards, B


@pytest.mark.parametrize("widths", [[100], [0], [1, 0, 130]])
@pytest.mark.parametrize("tokens", [True, False])
def test_rows_that_the_join_can_count(widths, tokens):
    most = (1 << 26) - 16                   # 64 threads per row, in workgroups of 16 rows: below 2^32 work-items
    assert rog.rog_linear_logprob_plan(widths, most, 8, tokens=tokens)["launches"] >= 1
    for rows in (most + 1, 1 << 26, 1 << 28, (1 << 31) - 1):
        with pytest.raises(rog.RogArgumentError):
            rog.rog_linear_logprob_plan(widths, rows, 8, tokens=tokens)


def test_such_calls_are_refused_before_anything_is_enqueued():
    # fake addresses on a machine without a GPU: a call that got past its checks would end in a launch error
    for rows in ((1 << 26) - 15, 1 << 26, 1 << 30):
        assert score(rows=rows, sh=shards((B, 64, 100)), h_stride=0, ws_bytes=1 << 60) == TOO_LARGE
        assert score(rows=rows, sh=shards((B, 64, 0)), h_stride=0, ws_bytes=1 << 60) == TOO_LARGE
    assert score(rows=0, sh=shards((B, 64, 100))) == OK
