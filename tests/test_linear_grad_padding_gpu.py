"""The weights' gradients of the same scored rows have the same bits whatever
rows that are not scored stand between them."""
from __future__ import annotations

import pytest
import torch

from deterministic_collective_movement_amd import rog
from tests import linear_ref as ref
from tests.test_linear_gpu import check_grad

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16

# scored rows and all rows around where sums over rows are cut: none and some parts, some and more, large and small tiles
CASES = [
    ([200], 64, 2000, 2047, BF16),
    ([200], 64, 2047, 2049, BF16),
    ([200], 64, 2100, 4096, BF16),
    ([200], 64, 2100, 4096, F16),
    ([130, 255], 33, 4000, 4200, F16),
    ([1000], 256, 4097, 20000, BF16),
    ([1000, 700], 520, 3000, 9000, BF16),
    ([300], 300, 60, 30000, BF16),
    ([300], 300, 700, 30000, F16),
    ([300], 300, 20000, 70000, BF16),
    ([9000], 64, 5000, 40000, BF16),
    ([20000], 64, 9000, 66000, F16),
]


@pytest.mark.parametrize("widths,dim,scored,rows,dtype", CASES)
def test_rows_that_do_not_count_change_no_weight(gpu, widths, dim, scored, rows, dtype):
    h, ws, tokens = ref.head(scored, widths, dim, dtype, gpu)
    gen = torch.Generator(device=gpu)
    gen.manual_seed(rows)
    g, gh = torch.randn(scored, generator=gen, device=gpu), 0.1 * torch.randn(scored, generator=gen, device=gpu)
    s = rog.rog_linear_logprob(h, ws, tokens)
    alone = rog.rog_linear_logprob_grad(h, ws, tokens, s.lse, s.entropy, g, gh)
    at = torch.randperm(rows, generator=gen, device=gpu)[:scored].sort().values
    wide = lambda v, fill: torch.full((rows,) + v.shape[1:], fill, dtype=v.dtype, device=gpu).index_copy_(0, at, v)  # noqa: E731
    padded = rog.rog_linear_logprob_grad(wide(h, 3.0), ws, wide(tokens, -1), wide(s.lse, 0.0), wide(s.entropy, 0.0), wide(g, 5.0), wide(gh, 5.0))
    for a, b in zip(alone.d_weights, padded.d_weights):
        assert torch.equal(a, b)
    assert torch.equal(padded.d_hidden[at], alone.d_hidden)


@pytest.mark.parametrize("widths,dim,scored,rows,dtype", [CASES[2], CASES[4], CASES[8], CASES[10]])
def test_sums_in_fewer_parts_than_there_is_room_for(gpu, widths, dim, scored, rows, dtype):
    h, ws, tokens = ref.head(rows, widths, dim, dtype, gpu)
    tokens[torch.randperm(rows, device=gpu)[:rows - scored]] = -1
    check_grad(h, ws, tokens)
