"""The compiled marshalling (_rog_binding.so) is a quicker way through rog.py, not a part that it needs: a package
with librog.so alone imports and validates as before, and says so where a module that is there cannot be loaded."""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

import pytest
import torch

from deterministic_collective_movement_amd import build, rog

PROGRAM = """
import sys, warnings
sys.path.insert(0, sys.argv[1])
with warnings.catch_warnings(record=True) as seen:
    warnings.simplefilter("always")
    from deterministic_collective_movement_amd import rog
assert rog.LIB_PATH.startswith(sys.argv[1]), rog.LIB_PATH
print(len([w for w in seen if "_rog_binding" in str(w.message)]))
print(rog.rog_status_of_ptrs([1 << 30], 1, 4096, 1 << 31))
print(rog.rog_logprob_plan_widths([131072], 4, rog.ROG_DTYPE_BF16)["form"])
import torch
for call in (lambda: rog.rog_gather([torch.zeros(4)]), lambda: rog.rog_logprob([torch.zeros(2, 3)]),
             lambda: rog.rog_policy_loss(*[torch.zeros(4)] * 3, out=(torch.zeros(4), None, None)),
             lambda: rog.rog_logprob([torch.zeros(2, 3)], out=(None, torch.zeros(2), None, None, None)),
             lambda: rog.rog_logprob_grad([torch.zeros(2, 3)], *[torch.zeros(2)] * 4, out=[torch.zeros(2, 3)])):
    try:
        call()
    except ValueError:
        continue
    raise AssertionError("accepted")
"""


@pytest.mark.parametrize("module", [None, b"\x7fELF no such module"], ids=["absent", "broken"])
def test_import_without_the_module(tmp_path, module):
    pkg = tmp_path / "deterministic_collective_movement_amd"
    pkg.mkdir()
    for name in os.listdir(build.PKG):
        if name.endswith(".py") or name == "librog.so":
            shutil.copy(os.path.join(build.PKG, name), pkg / name)
    if module is not None:
        (pkg / os.path.basename(build.BINDING_PATH)).write_bytes(module)
    done = subprocess.run([sys.executable, "-c", PROGRAM, str(tmp_path)], capture_output=True, text=True, cwd=str(tmp_path))
    assert done.returncode == 0, done.stderr
    assert done.stdout.split() == [str(int(module is not None)), "0", "split"]


@pytest.mark.gpu
def test_calls_without_the_module(gpu, monkeypatch):
    """Calls with their outputs in hand, which the module would take: the same bits without it."""
    gen = torch.Generator(device=gpu)
    gen.manual_seed(2)
    x = torch.randn(6, 40007, generator=gen, device=gpu).bfloat16()
    tokens = torch.randint(0, 40007, (6,), generator=gen, device=gpu)
    logp, old, adv, h = (torch.randn(30001, generator=gen, device=gpu) for _ in range(4))

    def calls():
        out = rog.RogLogprob(*(torch.full(s, 3.0, device=gpu) for s in ((6,), (6,), (6,), (6, 4))),
                             torch.full((6, 4), 3, dtype=torch.int64, device=gpu))
        r = rog.rog_logprob([x], tokens, 4, out=out)
        d = rog.rog_logprob_grad([x], tokens, r.lse, r.entropy, r.logp, out=[torch.full_like(x, 3.0)])
        l_out = (torch.full((4,), 3.0, device=gpu), torch.full((30001,), 3.0, device=gpu), torch.full((30001,), 3.0, device=gpu))
        loss = rog.rog_policy_loss(logp, old, adv, entropy=h, entropy_coef=0.1, out=l_out)
        return [*r, *d, *loss]

    with_module = calls()
    monkeypatch.setattr(rog, "_binding", None)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for without in (calls(), calls()):
        assert all(torch.equal(a, b) for a, b in zip(with_module, without))
    with torch.cuda.stream(side):        # a stream that has no workspace yet
        without = calls()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(with_module, without))
