"""The gradient of a batch without rows: the weights' are sums over none, zero."""
from __future__ import annotations

import pytest
import torch

from deterministic_collective_movement_amd import rog

pytestmark = pytest.mark.gpu


def inputs(dev, dtype):
    ws = [torch.randn(w, 24, device=dev).to(dtype) for w in (300, 0, 7)]
    none = torch.empty(0, device=dev)
    return torch.empty(0, 24, dtype=dtype, device=dev), ws, torch.empty(0, dtype=torch.int64, device=dev), none


@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_weights_get_zeros(gpu, monkeypatch, compiled, dtype):
    if not compiled:
        monkeypatch.setattr(rog, "_binding", None)
    h, ws, tokens, none = inputs(gpu, dtype)
    # memory that holds something, so that what is not written shows
    full = [torch.full((w.shape[0], 24), 7.0, dtype=dtype, device=gpu) for w in ws]
    del full
    r = rog.rog_linear_logprob_grad(h, ws, tokens, none, none, none)
    assert r.d_hidden.shape == (0, 24)
    assert all(g.shape == w.shape and bool((g == 0).all()) for g, w in zip(r.d_weights, ws))
    # in place, and inside larger matrices whose other elements stay
    wide = [torch.full((w.shape[0] + 1, 40), 7.0, dtype=dtype, device=gpu) for w in ws]
    rog.rog_linear_logprob_grad(h, ws, tokens, none, none, none, none, out=(torch.empty_like(h), [g[:-1, 8:32] for g in wide]))
    for g in wide:
        assert bool((g[:-1, 8:32] == 0).all()) and bool((g[-1] == 7).all()) and bool((g[:, :8] == 7).all()) and bool((g[:, 32:] == 7).all())


def test_on_a_stream_by_name_and_captured(gpu):
    h, ws, tokens, none = inputs(gpu, torch.bfloat16)
    out = rog.RogLinearGrad(torch.empty_like(h), [torch.full_like(w, 7.0) for w in ws])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    rog.rog_linear_logprob_grad(h, ws, tokens, none, none, none, out=out, stream=s)
    s.synchronize()
    assert all(bool((g == 0).all()) for g in out.d_weights)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        rog.rog_linear_logprob_grad(h, ws, tokens, none, none, none, out=out)
    for _ in range(3):
        for g in out.d_weights:
            g.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(bool((g == 0).all()) for g in out.d_weights)


def test_outputs_that_require_gradients(gpu):
    # written like any other output: in no autograd graph
    h, ws, tokens, none = inputs(gpu, torch.bfloat16)
    out = rog.RogLinearGrad(torch.empty_like(h), [torch.full_like(w, 7.0).requires_grad_() for w in ws])
    rog.rog_linear_logprob_grad(h, ws, tokens, none, none, none, out=out)
    assert all(g.is_leaf and bool((g == 0).all()) for g in out.d_weights)


def test_refusals_stay(gpu):
    h, ws, tokens, none = inputs(gpu, torch.bfloat16)
    with pytest.raises(ValueError):
        rog.rog_linear_logprob_grad(h, ws, tokens, none, none, none, out=(torch.empty_like(h), [w[:, :8] for w in ws]))
    with pytest.raises(ValueError):
        rog.rog_linear_logprob_grad(h, ws, tokens, none, none, none, out=(torch.empty_like(h), ws[:2]))
