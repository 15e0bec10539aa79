"""What tests/test_linear_resources.py leaves out, by the kernels' names: the
product kernels whose operands come through registers are those whose last
argument says so, and of the others every one is looked at -- the weights'
gradient of few rows or little work, the quantization and the joins among them."""
from __future__ import annotations

import re

from tests.test_linear_resources import kernels, listings  # noqa: F401

THROUGH_REGISTERS = ("score_kernel", "coef_kernel", "i8_kernel", "back_kernel", "few_states_kernel")   # where the last argument is false


def through_registers(name):
    return "Lb0EEEv" in name and any(k in name for k in THROUGH_REGISTERS)


def test_the_joins_and_the_weights_of_little_work_are_there(kernels):  # noqa: F811
    for k, n in (("rog_linear_weights_join_kernel", 2), ("rog_linear_back_join_kernel", 2), ("rog_linear_join_kernel", 2),
                 ("rog_linear_pack_kernel", 2), ("rog_quantize_kernel", 6), ("rog_linear_few_weights_kernel", 4)):
        assert sum(k in name for name in kernels) == n, k


def test_nothing_in_scratch(kernels):  # noqa: F811
    looked = 0
    for name, k in kernels.items():
        if through_registers(name) or "back_kernel" in name:
            continue
        looked += 1
        assert k["scratch"] == 0, (name, k)
    assert looked == 10 + 10 + 12 + 2 + 4 + 6 + 2 + 6      # scores, coefficients, 8-bit, states, weights, joins, packing, quantization


def test_nothing_spilled_in_any_loop(listings):  # noqa: F811
    """Every block that multiplies, in a loop or not, of every kernel with direct loads."""
    loops = {}
    for text in listings.values():
        for name in re.findall(r"^(_Z\S+):", text, re.M):
            if through_registers(name):
                continue
            at = text.index("\n" + name + ":")
            for block in re.split(r"\n(?=\.LBB)", text[at:text.index(".Lfunc_end", at)]):
                if "v_mfma" in block and "s_barrier" in block:
                    loops[name] = loops.get(name, 0) + 1
                    assert "scratch_" not in block, name
    for k, n in (("score_kernel", 10), ("coef_kernel", 10), ("i8_kernel", 12), ("back_kernel", 2), ("few_states_kernel", 2),
                 ("few_weights_kernel", 4)):
        assert sum(k in name for name in loops) == n, (k, n, sorted(loops))
    assert any("few_weights_kernelILi1ELb0E" in name for name in loops)
