"""Shared memory of the head's product kernels for few rows, which are bound by
the weights' bytes: two workgroups have to fit a CU's 160 KiB, so that one's
loads are in flight while the other starts or ends.  Only where there are no more
workgroups than CUs a score or its coefficients take a deeper form."""
from __future__ import annotations

import re

from tests.test_linear_resources import listings  # noqa: F401

HALF = 160 * 1024 // 2


def shared(listings):  # noqa: F811
    """{kernel: bytes of shared memory}, of all that the assembly lists."""
    got = {}
    for text in listings.values():
        for block in re.findall(r"\.amdhsa_kernel (\S+)(.*?)\.end_amdhsa_kernel", text, re.S):
            got[block[0]] = int(re.search(r"\.amdhsa_group_segment_fixed_size (\d+)", block[1]).group(1))
    return got


def test_two_workgroups_of_few_rows_fit_a_cu(listings):  # noqa: F811
    few = {n: b for n, b in shared(listings).items() if re.search(r"FormILi128ELi(32|64)E|few_weights", n)}
    deep = {n for n in few if "i8_kernel" not in n and "FormILi128ELi32ELi4ELi1ELi4E" in n}
    assert len(deep) == 8
    for kind in ("score_kernel", "coef_kernel", "i8_kernel", "few_weights"):
        assert sum(kind in n for n in few) >= 4, kind
    for name, size in few.items():
        assert size <= (2 * HALF if name in deep else HALF), (name, size)
