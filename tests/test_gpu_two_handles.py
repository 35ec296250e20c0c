"""Two handles whose single launches meet on the device: each leaves the other a part of the SMs only.

The tiles of a launch belong to the CTA pairs that run, so either goes on whatever it was given; results and status as alone.
"""
from __future__ import annotations

import pytest
import torch

from muon_newton_schulz_07_b200 import binding as B
from muon_newton_schulz_07_b200.optimizer import MuonStep

pytestmark = pytest.mark.gpu


def values(shape, seed, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(seed)
    return (1e-2 * torch.randn(shape, generator=gen)).to("cuda", dtype)


@pytest.mark.parametrize("mode", ["half", "fast"])
@pytest.mark.parametrize("shapes", [([(7, 331, 1003)], [(2, 512, 2048)]), ([(48, 512, 768)], [(300, 260), (40, 768, 768)])], ids=str)
def test_two_single_launches_at_once(mode, shapes):
    ops = [MuonStep(s, mode=mode, schedule="fused") for s in shapes]
    X = [[values(s, 10 * k + i) for i, s in enumerate(l)] for k, l in enumerate(shapes)]
    want = [[torch.empty_like(x) for x in l] for l in X]
    for op, x, w in zip(ops, X, want):
        op.orthogonalize(x, w)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    got = [[[torch.empty_like(x) for x in l] for _ in range(20)] for l in X]
    torch.cuda.synchronize()
    for t in range(20):
        for op, x, o, st in zip(ops, X, got, streams):
            op.orthogonalize(x, o[t], stream=st)
    torch.cuda.synchronize()
    for op, w, o in zip(ops, want, got):
        assert op.status() == B.MUON_OK
        for one in o:
            assert all(torch.equal(a, b) for a, b in zip(one, w))
        op.close()


@pytest.mark.parametrize("shapes", [[(300, 260)], [(7, 331, 1003)], [(20, 768, 768)], [(1024, 1024), (300, 3000), (260, 700)]], ids=str)
@pytest.mark.parametrize("k", [1, 2, 7])
def test_every_tile_is_done_once(shapes, k):
    """Against the launches of one stage each, where no tile waits; replayed from a graph, where the counters start again."""
    outs = []
    for schedule in ("staged", "fused", "split"):
        op = MuonStep(shapes, mode="half", schedule=schedule)
        X = [values(s, i) for i, s in enumerate(shapes)]
        O = [torch.empty_like(x) for x in X]
        op.orthogonalize(X, O, ns_steps=k)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            op.orthogonalize(X, O, ns_steps=k)
        for _ in range(3):
            for o in O:
                o.zero_()
            graph.replay()
            torch.cuda.synchronize()
            outs.append([o.clone() for o in O])
        assert op.status() == B.MUON_OK
        del graph
        op.close()
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


@pytest.mark.parametrize("mode", ["half", "fast"])
def test_a_single_launch_beside_work_that_stays(mode):
    """On-chip iterations hold more than half of the SMs for many times as long as the other handle's launch takes, and
    that launch waits for none of them."""
    long = MuonStep([(40, 128, 1024)], mode="half")
    held = [values((40, 128, 1024), 3)]
    held_out = [torch.empty_like(held[0])]
    shape = (7, 331, 1003)
    op = MuonStep([shape], mode=mode, schedule="fused")
    x = [values(shape, 4)]
    want, got = [torch.empty_like(x[0])], [torch.empty_like(x[0])]
    op.orthogonalize(x, want)
    long.orthogonalize(held, held_out, ns_steps=64)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    ended = torch.cuda.Event()
    torch.cuda.synchronize()
    for _ in range(40):
        long.orthogonalize(held, held_out, ns_steps=64, stream=a)
    ended.record(a)
    for _ in range(3):
        op.orthogonalize(x, got, stream=b)
    b.synchronize()
    assert not ended.query()
    assert torch.equal(got[0], want[0])
    torch.cuda.synchronize()
    assert op.status() == B.MUON_OK and long.status() == B.MUON_OK
    op.close()
    long.close()
