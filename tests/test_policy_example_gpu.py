"""The policy-step example learns, and repeats bit for bit; the operators under
several host threads, and by both ways through the binding."""
from __future__ import annotations

import importlib.util
import os
import threading

import pytest
import torch

from deterministic_collective_movement_amd import rog

pytestmark = pytest.mark.gpu

EXAMPLE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "policy_step.py")


def _example():
    spec = importlib.util.spec_from_file_location("policy_step", EXAMPLE)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_example_learns_and_repeats(gpu):
    ex = _example()
    rewards, weights = ex.run(steps=20)
    assert sum(rewards[-3:]) / 3 > sum(rewards[:3]) / 3 + 0.1, rewards
    again, same = ex.run(steps=20)
    assert rewards == again and all(torch.equal(a, b) for a, b in zip(weights, same))


def test_host_threads_on_their_own_streams(gpu):
    gen = torch.Generator(device=gpu)
    gen.manual_seed(1)
    x = torch.randn(5, 30011, generator=gen, device=gpu).bfloat16()
    tokens = torch.randint(0, 30011, (5,), generator=gen, device=gpu)
    n = 20001
    logp, old, adv = (torch.randn(n, generator=gen, device=gpu) for _ in range(3))
    want, loss = rog.rog_logprob([x], tokens, 7), rog.rog_policy_loss(logp, old, adv)
    torch.cuda.synchronize()
    bad = []

    def work():
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(40):
                    got, l2 = rog.rog_logprob([x], tokens, 7), rog.rog_policy_loss(logp, old, adv)
                    s.synchronize()
                    if not all(torch.equal(a, b) for a, b in zip(got, want)) or not torch.equal(l2.stats, loss.stats):
                        bad.append("bits")
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad, bad[:3]


def test_both_ways_through_the_binding(gpu):
    """Calls with outputs in hand go through the compiled marshalling, others through Python: the same bits, in graphs too."""
    gen = torch.Generator(device=gpu)
    gen.manual_seed(3)
    x = torch.randn(6, 40007, generator=gen, device=gpu).half()
    shards = [x[:, :20000], x[:, 20000:]]
    tokens = torch.randint(0, 40007, (6,), generator=gen, device=gpu)
    n = 30001
    logp, old, adv, h = (torch.randn(n, generator=gen, device=gpu) for _ in range(4))
    s = torch.cuda.current_stream()
    want = rog.rog_logprob(shards, tokens, 5, 0.9, stream=s)
    d_want = rog.rog_logprob_grad(shards, tokens, want.lse, want.entropy, want.logp, temperature=0.9, stream=s)
    l_want = rog.rog_policy_loss(logp, old, adv, entropy=h, entropy_coef=0.1, stream=s)
    out = tuple(torch.full_like(t, 3) for t in want)
    d_out = [torch.full_like(t, 3) for t in d_want]
    l_out = tuple(torch.full_like(t, 3) for t in l_want)

    def call():
        r = rog.rog_logprob(shards, tokens, 5, 0.9, out=out)
        d = rog.rog_logprob_grad(shards, tokens, r.lse, r.entropy, r.logp, temperature=0.9, out=d_out)
        return r, d, rog.rog_policy_loss(logp, old, adv, entropy=h, entropy_coef=0.1, out=l_out)

    def check():
        torch.cuda.synchronize()
        for got, ref in ((out, want), (d_out, d_want), (l_out, l_want)):
            assert all(torch.equal(a, b) for a, b in zip(got, ref))
            for t in got:
                t.fill_(3)

    r, d, l = call()
    assert r.logp is out[0] and d is d_out and l.stats is l_out[0]
    check()
    call()      # the stream has a workspace by now
    check()
    side = torch.cuda.Stream()
    side.wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for _ in range(3):
        graph.replay()
        check()
        call()
        check()
    with torch.cuda.stream(side):
        call()
    check()


def test_outputs_belong_to_the_stream_that_writes_them(gpu):
    """A call on another stream takes no memory that the current stream has just given back."""
    n = 300000
    x, tokens = torch.randn(3, n, device=gpu), torch.zeros(3, dtype=torch.int64, device=gpu)
    vectors = [torch.randn(n, device=gpu) for _ in range(3)]
    row = torch.randn(3, device=gpu)
    want, d_want, l_want = (rog.rog_logprob([x], tokens), rog.rog_logprob_grad([x], tokens, row, row, row), rog.rog_policy_loss(*vectors))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (side, side.cuda_stream):
        freed = set()
        for shape in ((3,), (n,), (3, n)):
            t = torch.empty(*shape, device=gpu)
            freed.add(t.data_ptr())
            del t
        got = [*rog.rog_logprob([x], tokens, stream=stream)[:3], *rog.rog_logprob_grad([x], tokens, row, row, row, stream=stream),
               *rog.rog_policy_loss(*vectors, stream=stream)[:2]]
        assert not freed & {t.data_ptr() for t in got}
        side.synchronize()
        for a, b in zip(got, [*want[:3], *d_want, *l_want[:2]]):
            assert torch.equal(a, b)
