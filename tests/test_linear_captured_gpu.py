"""Captured calls whose outputs the caller passes (the compiled module's way in):
each graph has workspaces of its own, beside eager calls and other graphs."""
from __future__ import annotations

import pytest
import torch

from deterministic_collective_movement_amd import rog
from tests import linear_ref as ref

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


class Step:
    """A score and its gradient into fixed outputs."""

    def __init__(self, case):
        self.h, self.ws, self.tokens = case
        n, dev = self.h.shape[0], self.h.device
        self.score = rog.RogLogprob(*(torch.zeros(n, device=dev) for _ in range(3)), None, None)
        self.grad = rog.RogLinearGrad(torch.zeros_like(self.h), [torch.zeros_like(w) for w in self.ws])
        self.g = torch.linspace(-1, 1, n, device=dev)

    def run(self):
        rog.rog_linear_logprob(self.h, self.ws, self.tokens, out=self.score)
        rog.rog_linear_logprob_grad(self.h, self.ws, self.tokens, self.score.lse, self.score.entropy, self.g, out=self.grad)

    def outputs(self):
        return [*self.score[:3], self.grad.d_hidden, *self.grad.d_weights]

    def clear(self):
        for t in self.outputs():
            t.fill_(7.0)


@pytest.mark.parametrize("n", [5, 90, 300])
def test_captured_into_fixed_outputs(gpu, n):
    step = Step(ref.head(n, [900, 333], 136, BF16, gpu, pad=0.2))
    other = Step(ref.head(400, [2000], 256, BF16, gpu, seed=3))
    step.run()
    want = [t.clone() for t in step.outputs()]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step.run()
    for i in range(4):
        step.clear()
        other.run()
        scratch = torch.full((1 << 24,), 255, dtype=torch.uint8, device=gpu)      # takes what the allocator has at hand
        graph.replay()
        torch.cuda.synchronize()
        del scratch
        assert all(torch.equal(a, b) for a, b in zip(step.outputs(), want)), i


def test_two_graphs_and_eager_calls_at_once(gpu):
    steps = [Step(ref.head(300, [3000, 500], 256, BF16, gpu, seed=1)), Step(ref.head(200, [2500], 192, F16, gpu, seed=2, pad=0.3)),
             Step(ref.head(120, [1800], 128, BF16, gpu, seed=3))]
    for s in steps:
        s.run()
    want = [[t.clone() for t in s.outputs()] for s in steps]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g, s in zip(graphs, steps):
        with torch.cuda.graph(g):
            s.run()
    streams = [torch.cuda.Stream() for _ in range(3)]
    for i in range(5):
        for s in steps:
            s.clear()
        torch.cuda.synchronize()
        for stream, g in zip(streams, graphs):
            with torch.cuda.stream(stream):
                g.replay()
        with torch.cuda.stream(streams[2]):
            steps[2].run()
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            assert all(torch.equal(a, b) for a, b in zip(s.outputs(), w)), i
