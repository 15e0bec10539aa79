"""How many waves a SIMD of gfx950 holds of the vocabulary-side kernels, by their
registers: 512 per lane, given out in eights, so that 96 leave five waves and 97
leave four."""
from __future__ import annotations

import pytest

from tests.test_head_resources import kernels  # noqa: F401  (a fixture)


def waves_per_simd(vgprs: int) -> int:
    return min(8, 512 // (-(-vgprs // 8) * 8))


def test_the_rule():
    assert [waves_per_simd(v) for v in (64, 65, 72, 73, 80, 81, 96, 97, 104, 128, 129)] == [8, 7, 7, 6, 6, 5, 5, 4, 4, 4, 3]


@pytest.mark.parametrize("name,least", [("rog_logprob_row_kernel", 5), ("rog_logprob_wave_kernel", 5), ("rog_logprob_split_kernel", 5),
                                        ("rog_logprob_grad_kernel", 5), ("rog_policy_kernel", 5)])
def test_waves_per_simd(kernels, name, least):  # noqa: F811
    found = {k: waves_per_simd(v["vgpr"]) for k, v in kernels.items() if name in k}
    assert found and min(found.values()) >= least, found
