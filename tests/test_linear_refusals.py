"""Refusals of the head's products name the argument that they refuse."""
from __future__ import annotations

import pytest
import torch

from deterministic_collective_movement_amd import rog

S, Q = torch.zeros(3), torch.zeros(3, 8, dtype=torch.int8)


@pytest.mark.parametrize("q", [[1], None])
def test_states_in_8_bits_that_are_no_tensor(q):
    with pytest.raises(TypeError, match="^q must be"):
        rog.rog_linear_i8(q, S, [Q], [S])


@pytest.mark.parametrize("q", [Q.float(), Q.to(torch.uint8)])
def test_states_in_8_bits_of_another_type(q):
    with pytest.raises(ValueError, match="^q is int8 "):
        rog.rog_linear_i8(q, S, [Q], [S])


def test_states_in_8_bits_elsewhere():
    with pytest.raises(ValueError, match="^q must be on a GPU"):
        rog.rog_linear_i8(Q, S, [Q], [S])


def test_hidden_states():
    with pytest.raises(TypeError, match="^hidden must be"):
        rog.rog_linear_logprob(None, [Q])
    with pytest.raises(ValueError, match="^hidden is bfloat16 or float16 "):
        rog.rog_linear_logprob(S[:, None], [S[:, None]])
    with pytest.raises(ValueError, match="^hidden must be on a GPU"):
        rog.rog_linear_logprob(S[:, None].half(), [S[:, None].half()])
