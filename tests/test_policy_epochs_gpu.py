"""The policy-step example takes several updates on the tokens of one sample, so
that the clipped loss works on ratios other than 1."""
from __future__ import annotations

import pytest

from tests.test_policy_example_gpu import _example

pytestmark = pytest.mark.gpu


def test_updates_move_the_ratio(gpu):
    ex = _example()
    clipped = []
    rewards, _ = ex.run(steps=20, clipped=clipped)
    assert len(clipped) == len(rewards) == 20 and all(len(c) == ex.EPOCHS >= 2 for c in clipped)
    # before the weights move a token's score has the bits that it was sampled with: nothing is clipped
    assert all(c[0] == 0 for c in clipped)
    assert any(c[-1] > 0 for c in clipped), clipped
