"""step_from_host's device buffers: blocks that the allocator takes from, and gives to, others while streams are at work."""
from __future__ import annotations

import pytest
import torch

from muon_newton_schulz_07_b200 import binding as B
from muon_newton_schulz_07_b200.optimizer import MuonStep

pytestmark = pytest.mark.gpu

SHAPES = [(512, 768), (2, 300, 256)]


def tensors():
    gen = torch.Generator().manual_seed(3)
    G = [(1e-2 * torch.randn(s, generator=gen)).to(torch.bfloat16).pin_memory() for s in SHAPES]
    W = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in SHAPES]
    return W, G, [torch.zeros_like(w) for w in W]


@pytest.mark.parametrize("mode", ["fast", "half"])
def test_blocks_whose_last_work_is_still_queued(mode):
    op = MuonStep(SHAPES, mode=mode)
    W, G, M = tensors()
    torch.cuda.synchronize()
    old = [torch.full(s, 3.0, dtype=torch.bfloat16, device="cuda") for s in SHAPES * 2]
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    kept = [t.clone() for t in old]                     # after the sleep
    del old                                             # and their blocks are free for the buffers
    op.step_from_host(W, G, M)
    torch.cuda.synchronize()
    assert all(bool((t == 3).all()) for t in kept)
    want = [torch.zeros_like(w) for w in W]
    op(want, [g.cuda() for g in G], [torch.zeros_like(w) for w in W])
    assert op.status() == B.MUON_OK
    assert all(torch.equal(a, b) for a, b in zip(W, want))
    op.close()


@pytest.mark.parametrize("mode", ["fast", "half"])
def test_buffers_outlive_the_step_on_another_stream(mode):
    op = MuonStep(SHAPES, mode=mode)
    W, G, M = tensors()
    op.step_from_host(W, G, M)                          # (buffers of the current stream)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
    op.step_from_host(W, G, M, stream=side)
    at = {t.data_ptr() for t in op._gbuf[0] + op._gbuf[1]}
    op._gbuf = None
    taken = [torch.empty(s, dtype=torch.bfloat16, device="cuda") for s in SHAPES * 4]
    assert not side.query() and not at & {t.data_ptr() for t in taken}
    torch.cuda.synchronize()
    op.close()
