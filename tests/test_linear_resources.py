"""Device-code resources of the head's product kernels, from the gfx950 assembly
that hipcc emits on the CPU: no packed binary32 instructions, no calls, one
argument struct at offset 0, registers for two waves per SIMD, and nothing
spilled inside the loops that multiply (a spill's load there waits for every
load that is in flight)."""
from __future__ import annotations

import os
import re
import shutil
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from deterministic_collective_movement_amd import build as b
from tests.test_kernel_resources import _parse

SOURCES = ("rog_linear_score.hip", "rog_linear_grad.hip", "rog_linear_i8.hip")


@pytest.fixture(scope="module")
def listings(tmp_path_factory):
    hipcc = shutil.which("hipcc") or os.path.join(b.ROCM, "bin", "hipcc")
    folder = tmp_path_factory.mktemp("asm")

    def listing(src):
        out = str(folder / (src + ".s"))
        subprocess.check_call([hipcc, "-O3", "-std=c++17", "--offload-arch=gfx950", "--offload-device-only", "-S",
                               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                               "-Wno-unused-command-line-argument", "-I", b.INCLUDE, "-I", b.CSRC,
                               os.path.join(b.CSRC, src), "-o", out], stderr=subprocess.DEVNULL)
        return open(out).read()

    with ThreadPoolExecutor(len(SOURCES)) as pool:
        return dict(zip(SOURCES, pool.map(listing, SOURCES)))


@pytest.fixture(scope="module")
def kernels(listings):
    ks = {}
    for text in listings.values():
        ks.update(_parse(text))
    return ks


def straight(name):
    """Whether the kernel's operands go straight to the shared memory (its last template argument)."""
    return "Lb0EEEv" not in name


def test_no_packed_binary32_and_no_calls(listings):
    for src, text in listings.items():
        for banned in ("v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32", "s_swappc"):
            assert banned not in text, (src, banned)


def test_every_kernel_is_present(kernels):
    names = " ".join(kernels)
    for k in ("rog_linear_score_kernel", "rog_linear_join_kernel", "rog_linear_pack_kernel", "rog_linear_coef_kernel", "rog_linear_back_kernel",
              "rog_linear_few_states_kernel", "rog_linear_few_weights_kernel", "rog_linear_back_join_kernel", "rog_quantize_kernel",
              "rog_linear_i8_kernel"):
        assert k in names, k


def test_registers_and_arguments(kernels):
    for name, k in kernels.items():
        assert not k["dyn_stack"], name
        assert k["vgpr"] <= 256, (name, k)
        if straight(name) and "back_kernel" not in name:
            assert k["scratch"] == 0, (name, k)
        assert len(k["explicit_args"]) == 1 and k["explicit_args"][0][0] == 0, (name, k["explicit_args"])
        assert k["explicit_args"][0][1] <= 4096, name


def test_nothing_spilled_in_the_loops(listings):
    loops = 0
    for text in listings.values():
        for name in re.findall(r"^(_Z\S+):", text, re.M):
            if not straight(name):
                continue
            at = text.index("\n" + name + ":")
            for block in re.split(r"\n(?=\.LBB)", text[at:text.index(".Lfunc_end", at)]):
                if block.count("v_mfma") >= 64 and "s_barrier" in block:
                    loops += 1
                    assert "scratch_" not in block, name
    assert loops >= 12
