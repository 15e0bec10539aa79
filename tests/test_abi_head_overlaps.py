"""Overlaps that the vocabulary-side operators refuse, on the CPU: no call here
gets to a launch (a call that validation lets pass fails there, without a GPU)."""
from __future__ import annotations

import struct

from deterministic_collective_movement_amd import rog

A, BIG = 1 << 30, 1 << 40          # fake device addresses


def test_policy_loss_workspace_is_no_input():
    """The workspace is written: one that shares bytes with an input is refused."""
    n, room = 5000, 1 << 20
    need = rog.rog_policy_loss_workspace_bytes(n)
    places = [A + i * room for i in range(6)]
    ins, params, outs = struct.pack("=6Q", *places), struct.pack("=5f", 0.2, 0.2, 0.0, 0.0, 1.0), struct.pack("=3Q", BIG, 0, 0)
    for place in places:
        for ws in (place, place + 4 * n - 16, place - need + 16):
            assert rog.lib().rog_policy_loss(ins, n, params, outs, ws, need, None) == rog.ROG_ERR_OVERLAP, ws - place
