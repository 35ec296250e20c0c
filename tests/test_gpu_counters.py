"""What a handle keeps in its workspace between calls: the fill at its creation against work on other streams, counters that an
earlier call left behind, the status word.

The results are compared bit for bit with those of a handle that nothing ran beside.
"""
from __future__ import annotations

import pytest
import torch

from muon_newton_schulz_07_b200 import binding as B
from muon_newton_schulz_07_b200.optimizer import MuonStep, QuantizedState

pytestmark = pytest.mark.gpu

SHAPES = [(3, 64, 96), (300, 256), (2, 512, 768)]


def values(shape, seed, dtype=torch.bfloat16):
    gen = torch.Generator().manual_seed(seed)
    return (1e-2 * torch.randn(shape, generator=gen)).to("cuda", dtype)


def tensors():
    """W, G, U and a state of one set of values."""
    G = [values(s, 10 + i) for i, s in enumerate(SHAPES)]
    state = QuantizedState(SHAPES)
    state.write([values(s, 20 + i) for i, s in enumerate(SHAPES)])
    return [values(s, 30 + i) for i, s in enumerate(SHAPES)], G, [torch.empty_like(g) for g in G], state


def calls(op, W, G, U, state):
    """Momentum, a step and the orthogonaliser, twice: everything that they write, the norms with it."""
    out = []
    for t in range(2):
        out.append(op.momentum(G, state, U, seed=2 * t))
        out += [u.clone() for u in U]
        op(W, G, state, seed=2 * t + 1)
        out += [op.norms()] + [w.clone() for w in W]
        op.orthogonalize(G, U)
        out += [op.norms()] + [u.clone() for u in U]
    return out + [q.clone() for q in state.codes] + [s.clone() for s in state.scales]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b, strict=True))


def alone():
    op = MuonStep(SHAPES, mode="half")
    got = calls(op, *tensors())
    torch.cuda.synchronize()
    assert op.status() == B.MUON_OK
    op.close()
    return got


def test_a_handle_made_while_the_default_stream_is_busy():
    """The workspace is filled before muon_create returns, whatever else the device has to do."""
    want = alone()
    made = tensors()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)                      # a tenth of a second on the default stream
    with torch.cuda.stream(side):
        op = MuonStep(SHAPES, mode="half")
        got = calls(op, *made)
    torch.cuda.synchronize()
    assert op.status() == B.MUON_OK
    assert same(got, want)
    op.close()


def test_a_workspace_whose_block_is_still_in_use():
    """A block that the allocator hands over may still be written by the stream it comes from."""
    want = alone()
    nbytes = B.muon_workspace_size([(s[-2], s[-1]) for s in SHAPES for _ in range(s[0] if len(s) == 3 else 1)],
                                   B.MUON_BF16, B.MUON_MODE_HALF) + 1024
    made = tensors()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        before = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
        torch.cuda._sleep(200_000_000)
        before.fill_(1)
        del before
        op = MuonStep(SHAPES, mode="half")
        got = calls(op, *made)
    torch.cuda.synchronize()
    assert op.status() == B.MUON_OK
    assert same(got, want)
    op.close()


def test_status_is_read_and_cleared_on_its_own_stream():
    op = MuonStep(SHAPES, mode="half")
    side = torch.cuda.Stream()
    B.muon_selftest_timeout(op.handle, 10_000, side.cuda_stream)    # a kernel's first launch loads it, which waits for the device
    assert op.status(side) == B.MUON_ERR_TIMEOUT
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)
    busy = torch.cuda.Event()
    busy.record()
    assert op.status(side) == B.MUON_OK
    for _ in range(3):                                  # recorded, read, cleared: and recorded again right after
        B.muon_selftest_timeout(op.handle, 10_000, side.cuda_stream)
        assert op.status(side) == B.MUON_ERR_TIMEOUT
    assert op.status(side) == B.MUON_OK
    assert not busy.query()                             # without a wait for the default stream
    torch.cuda.synchronize()
    op.close()


def spoil(op):
    """Everything in a handle's workspace but the status word, as a call that overlapped another might leave the counters."""
    at = op._ws_ptr - op._ws.data_ptr()
    op._ws[at + 1024:at + op.workspace_bytes].fill_(0x11)


@pytest.mark.parametrize("schedule", ["auto", "staged", "fused"])
def test_what_a_call_leaves_behind_does_not_reach_the_next(schedule):
    want = alone()
    op = MuonStep(SHAPES, mode="half", schedule=schedule)
    spoil(op)
    assert same(calls(op, *tensors()), want)
    W, G, U, state = tensors()
    V = [torch.empty_like(u) for u in U]
    op.orthogonalize(G, V)
    for call in (lambda: op.momentum(G, state, U, seed=1), lambda: op(W, G, state, seed=2), lambda: op.orthogonalize(G, U)):
        spoil(op)
        call()
    assert same(U, V)
    assert op.status() == B.MUON_OK
    op.close()


def test_a_captured_call_clears_its_counters():
    op = MuonStep(SHAPES, mode="half")
    want = alone()
    made, back = tensors(), tensors()
    W, G, U, state = made
    for _ in range(2):
        calls(op, *made)                                # (what a capture may not load)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls(op, *made)
    for _ in range(2):
        for a, b in zip(W + state.codes + state.scales, back[0] + back[3].codes + back[3].scales):
            a.copy_(b)
        spoil(op)
        graph.replay()
        torch.cuda.synchronize()
        assert same(got, want)
    assert op.status() == B.MUON_OK
    del graph
    op.close()


@pytest.mark.parametrize("how", ["stream=", "current", "graph"])
@pytest.mark.parametrize("call", ["orthogonalize", "step", "momentum"])
def test_a_workspace_outlives_the_work_on_another_stream(call, how):
    """A handle that goes while another stream's work is queued: its block is not handed out before that is done."""
    op = MuonStep(SHAPES, mode="half")
    W, G, U, state = tensors()

    def run(**kw):
        if call == "orthogonalize":
            op.orthogonalize(G, U, **kw)
        elif call == "step":
            op(W, G, state, **kw)
        else:
            op.momentum(G, state, U, **kw)

    run()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    if how == "graph":
        with torch.cuda.graph(graph, stream=side):
            run()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)
        if how == "graph":
            graph.replay()
        elif how == "current":
            run()
    if how == "stream=":
        run(stream=side)
    at, nbytes = op._ws.data_ptr(), op._ws.numel()
    op.close()
    op._ws = None
    taken = [torch.empty(nbytes, dtype=torch.uint8, device="cuda") for _ in range(3)]
    assert not side.query() and at not in [t.data_ptr() for t in taken]
    torch.cuda.synchronize()
    del graph
