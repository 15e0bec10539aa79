"""The policy head's products called by several host threads on one stream: their
launches hand data to each other through a workspace, which no other call may
have while they are being enqueued."""
from __future__ import annotations

import threading

import pytest
import torch

from deterministic_collective_movement_amd import rog
from tests import linear_ref as ref

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


class Recorded:
    """The library, but for calls that take a workspace: those enqueue nothing and
    note the workspace; while the first of them is under way, `between` runs."""

    PLACE = {"rog_linear_logprob": 10, "rog_linear_logprob_grad": 16, "rog_logprob_ex": 8}   # of the workspace's address

    def __init__(self, lib, needs, between):
        self.lib, self.needs, self.between, self.taken = lib, needs, between, []

    def __getattr__(self, name):
        if name not in self.PLACE:
            return getattr(self.lib, name)

        def call(*args):
            at, size = args[self.PLACE[name]:self.PLACE[name] + 2]
            if not at or size < self.needs[name]:
                return rog.ROG_ERR_INVALID_ARGUMENT
            self.taken.append((name, at, at + size))
            if len(self.taken) == 1:
                other = threading.Thread(target=self.between)
                other.start()
                other.join()
            return rog.ROG_OK

        return call


def test_a_call_has_its_workspace_to_itself(gpu, monkeypatch):
    """Nothing is launched: another thread's calls come in the middle of one, on its stream."""
    h, ws, tokens = ref.head(100, [500, 300], 64, BF16, gpu)
    x, t = [torch.zeros(4, 60000, dtype=BF16, device=gpu)], torch.zeros(4, dtype=torch.int64, device=gpu)
    z = torch.zeros(100, device=gpu)
    stream = torch.cuda.current_stream()
    needs = {"rog_linear_logprob": rog.rog_linear_logprob_plan([500, 300], 100, 64)["workspace_bytes"],
             "rog_linear_logprob_grad": rog.rog_linear_logprob_grad_plan([500, 300], 100, 64)["workspace_bytes"],
             "rog_logprob_ex": rog.rog_logprob_plan(x)["workspace_bytes"]}

    def score():
        rog.rog_linear_logprob(h, ws, tokens)

    def grad():
        rog.rog_linear_logprob_grad(h, ws, tokens, z, z, z)

    def split():
        rog.rog_logprob(x, t)

    monkeypatch.setattr(rog, "_binding", None)
    lib = rog._lib
    for call in (score, grad):
        failed = []

        def between():
            try:
                with torch.cuda.stream(stream):
                    for other in (score, grad, split):
                        other()
            except Exception as e:  # noqa: BLE001
                failed.append(e)

        recorded = Recorded(lib, needs, between)
        monkeypatch.setattr(rog, "_lib", recorded)
        call()
        monkeypatch.setattr(rog, "_lib", lib)
        assert not failed, failed
        assert [n for n, _, _ in recorded.taken[1:]] == ["rog_linear_logprob", "rog_linear_logprob_grad", "rog_logprob_ex"]
        _, begin, end = recorded.taken[0]
        for name, a, b in recorded.taken[1:]:
            assert b <= begin or a >= end, name


def call(case, g):
    """One thread's call, through the compiled module where it is there: outputs of its own."""
    h, ws, tokens = case
    n, dev = h.shape[0], h.device
    out = rog.RogLogprob(*(torch.empty(n, device=dev) for _ in range(3)), None, None)
    s = rog.rog_linear_logprob(h, ws, tokens, out=out)
    d = rog.rog_linear_logprob_grad(h, ws, tokens, s.lse, s.entropy, g,
                                    out=rog.RogLinearGrad(torch.empty_like(h), [torch.empty_like(w) for w in ws]))
    return [s.logp, s.entropy, s.lse, d.d_hidden, *d.d_weights]


@pytest.mark.parametrize("compiled", [True, False])
def test_two_threads_on_one_stream(gpu, monkeypatch, compiled):
    if not compiled:
        monkeypatch.setattr(rog, "_binding", None)
    # sizes that need different workspaces, packed rows and not, a split call of another operator's beside them
    cases = [ref.head(300, [1000, 500], 192, BF16, gpu, pad=0.3), ref.head(90, [700, 33], 128, F16, gpu, pad=0.2), ref.head(40, [3000], 64, BF16, gpu)]
    x, t = [torch.randn(4, 60000, device=gpu).to(BF16)], torch.randint(0, 60000, (4,), device=gpu)
    gs = [torch.randn(c[0].shape[0], device=gpu) for c in cases]
    want = [[v.clone() for v in call(c, g)] for c, g in zip(cases, gs)]
    split = [v.clone() for v in rog.rog_logprob(x, t, top_k=2)]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    got, start = [[] for _ in range(4)], threading.Barrier(4)
    failed = []

    def work(me):
        try:
            with torch.cuda.stream(stream):
                start.wait()
                for _ in range(40):
                    got[me].append(call(cases[me], gs[me]) if me < 3 else list(rog.rog_logprob(x, t, top_k=2)))
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    torch.cuda.synchronize()
    assert not failed, failed
    for mine, right in zip(got, want + [split]):
        for one in mine:
            assert all(torch.equal(a, b) for a, b in zip(one, right))


def test_large_workspaces_go_back(gpu):
    # what a large call needed is torch's again after it, and serves the next tensors
    h, ws, tokens = ref.head(2000, [20000], 256, BF16, gpu)
    one = torch.ones(2000, device=gpu)
    s = rog.rog_linear_logprob(h, ws, tokens)
    out = rog.RogLinearGrad(torch.empty_like(h), [torch.empty_like(ws[0])])
    need = rog.rog_linear_logprob_grad_plan([20000], 2000, 256)["workspace_bytes"]
    assert need > 50 << 20
    before = torch.cuda.memory_allocated()
    rog.rog_linear_logprob_grad(h, ws, tokens, s.lse, s.entropy, one, out=out)
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() == before
