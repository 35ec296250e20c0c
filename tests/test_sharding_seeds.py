"""ShardedMuon with an 8-bit state: the seeds of its stochastic rounding (CPU, the local step injected)."""
from __future__ import annotations

import pytest
import torch

from muon_newton_schulz_07_b200 import binding as B
from muon_newton_schulz_07_b200.optimizer import MuonStep, QuantizedState
from muon_newton_schulz_07_b200.sharding import ShardedMuon


def test_every_rank_rounds_with_random_bits_of_its_own():
    """Stochastic rounding keys its bits by the seed and the matrix's place in the call, and every rank's call starts at place
    0: the seed has to differ by rank, and two steps on two ranks may not meet either."""
    shapes = [(8, 8)] * 6
    seen = {}
    for rank in range(3):
        got = []
        sh = ShardedMuon(shapes, rank, 3, local_step=lambda W, G, M, **hp: got.append(hp))
        sh.exchange = lambda W: None
        sh.reduce_gradients = lambda G: [G[i] for i in sh.owned]
        T = [torch.zeros(s) for s in shapes]
        for t in range(200):
            sh.step(T, T, None, seed=t, lr=0.1)
        sh.step_local_grads(T, T, None, seed=200)
        sh.step(T, T, None, lr=0.1)
        sh.step(T, T, None, seed=None)
        assert all(hp["lr"] == 0.1 for hp in got[:200]) and "seed" not in got[201] and got[202]["seed"] is None
        seen[rank] = [hp["seed"] & 0xFFFFFFFF for hp in got[:201]]
        assert len(set(seen[rank])) == 201
    assert seen[0] == list(range(201))                   # one rank alone: the caller's seeds
    assert len(set(seen[0] + seen[1] + seen[2])) == 3 * 201


@pytest.mark.gpu
def test_sharded_steps_on_an_8_bit_state():
    """Every rank's step on the matrices it owns, one rank after the other: those of a handle with these matrices and that
    seed, and different codes where two ranks hold the same matrix."""
    shapes = [(64, 96), (300, 256)] * 2
    gen = torch.Generator().manual_seed(1)
    G = [(1e-2 * torch.randn(s, generator=gen)).to("cuda", torch.bfloat16) for s in shapes[:2]] * 2
    codes = {}
    for rank in range(2):
        sh = ShardedMuon(shapes, rank, 2, local_step=lambda *a, **hp: op(*a, **hp))
        sh.exchange = lambda W: None
        own = [shapes[i] for i in sh.owned]
        op = MuonStep(own, mode="half")
        W = [torch.zeros_like(g) for g in G]
        state = QuantizedState(own)
        for t in range(3):
            sh.step(W, G, state, lr=0.02, seed=t)
        ref, V = QuantizedState(own), [torch.zeros_like(G[i]) for i in sh.owned]
        for t in range(3):
            op(V, [G[i] for i in sh.owned], ref, lr=0.02, seed=t + rank * 0x9E3779B1)
        assert op.status() == B.MUON_OK
        assert all(torch.equal(W[i], v) for i, v in zip(sh.owned, V))
        assert all(torch.equal(a, b) for a, b in zip(state.codes, ref.codes))
        codes[rank] = {shapes[i]: q for i, q in zip(sh.owned, state.codes)}
        op.close()
    for s in set(codes[0]) & set(codes[1]):
        assert not torch.equal(codes[0][s], codes[1][s])
    assert set(codes[0]) & set(codes[1])
