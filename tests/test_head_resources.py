"""Device-code resources of the vocabulary-side kernels, from the gfx950
assembly that hipcc emits on the CPU: no scratch, no dynamic stack, registers
within what keeps the long-row kernels at five waves per SIMD or more, one
argument struct at offset 0."""
from __future__ import annotations

import os
import shutil
import subprocess

import pytest

from deterministic_collective_movement_amd import build as b
from tests.test_kernel_resources import _parse

SOURCES = ("rog_logprob.hip", "rog_logprob_grad.hip", "rog_policy.hip")


@pytest.fixture(scope="module")
def kernels(tmp_path_factory):
    hipcc = shutil.which("hipcc") or os.path.join(b.ROCM, "bin", "hipcc")
    ks = {}
    for src in SOURCES:
        out = str(tmp_path_factory.mktemp("asm") / (src + ".s"))
        subprocess.check_call([hipcc, "-O3", "-std=c++17", "--offload-arch=gfx950", "--offload-device-only", "-S",
                               "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
                               "-Wno-unused-command-line-argument", "-I", b.INCLUDE, "-I", b.CSRC,
                               os.path.join(b.CSRC, src), "-o", out], stderr=subprocess.DEVNULL)
        text = open(out).read()
        for banned in ("v_pk_add_f32", "v_pk_mul_f32", "v_pk_fma_f32", "s_swappc"):
            assert banned not in text, (src, banned)
        ks.update(_parse(text))
    return ks


def test_every_kernel_is_present(kernels):
    names = " ".join(kernels)
    for k in ("rog_logprob_row_kernel", "rog_logprob_split_kernel", "rog_logprob_wave_kernel", "rog_logprob_grad_kernel",
              "rog_policy_kernel"):
        assert k in names, k


def test_no_scratch_and_registers(kernels):
    for name, k in kernels.items():
        assert k["scratch"] == 0 and not k["dyn_stack"], (name, k)
        assert k["vgpr"] <= 104, (name, k)          # five waves per SIMD beside 512 registers, rounded to 8


def test_one_argument_struct_at_offset_zero(kernels):
    for name, k in kernels.items():
        assert len(k["explicit_args"]) == 1 and k["explicit_args"][0][0] == 0, (name, k["explicit_args"])
        assert k["explicit_args"][0][1] <= 4096, name
