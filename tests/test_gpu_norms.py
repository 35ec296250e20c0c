"""The Frobenius norms of MUON_MODE_HALF: of matrices of many tiles, in work that grows with their size.

A norm adds up squares rounded to fp32 in partial sums of at most 40 terms in sequence (a thread's 32, eight warps; then the
parts of a thread, averaged over 256 of them): its relative error stays below 64 * 2^-24.
"""
from __future__ import annotations

import pytest
import torch

from muon_newton_schulz_07_b200 import binding as B
from muon_newton_schulz_07_b200.optimizer import MuonStep, QuantizedState

pytestmark = pytest.mark.gpu

NORM = 64 * 2.0 ** -24


def normal(shape, seed, dtype=torch.bfloat16):
    gen = torch.Generator("cuda").manual_seed(seed)
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen)


@pytest.mark.parametrize("shape", [(130, 300), (2, 200, 40_000), (150_000, 260), (4096, 4096)], ids=str)
def test_norms_of_many_parts(shape):
    op = MuonStep([shape], mode="half")
    X = normal(shape, 1)
    X[..., 0, :7] *= 100
    want = X.double().flatten(-2).norm(dim=-1).reshape(-1)
    out, u = torch.empty_like(X), torch.empty_like(X)
    op.orthogonalize([X], [out], ns_steps=1)
    got = [op.norms()]
    for _ in range(3):                                  # the counters start again with every call
        op.orthogonalize([X], [out], ns_steps=1)
        got.append(op.norms())
    got.append(op.momentum([X], QuantizedState([shape]), [u], beta=0.0))
    for g in got:
        assert bool(((g.double() - want).abs() <= NORM * want).all())
    # one iteration with (1, 0, 0) leaves the normalised matrix: two roundings to fp16 and one to bf16
    op.orthogonalize([X], [out], abc=(1.0, 0.0, 0.0), ns_steps=1)
    ref = X.double() / (want.reshape(-1, 1, 1) if X.dim() == 3 else want)
    err = (out.double() - ref).flatten(-2).norm(dim=-1)
    assert bool((err <= 2.0 ** -9 + 2.0 ** -10).all())
    assert op.status() == B.MUON_OK
    op.close()


def front_ms(shape):
    """The norms and X0 of one call, the best of five."""
    op = MuonStep([shape], mode="half")
    X = normal(shape, 2)
    best = 1e9
    for _ in range(5):
        B.muon_profile_begin(op.handle, 1)
        op.orthogonalize([X], [X], ns_steps=1)
        best = min(best, B.muon_profile_end(op.handle)["momentum_norm"][0])
    op.close()
    return best


def test_the_norms_work_grows_with_the_matrix():
    """Eight times the tiles: eight times the time, where work that grew with their square would take far more."""
    small, large = front_ms((1024, 1 << 17)), front_ms((1024, 1 << 20))
    assert large <= 12 * small, (small, large)
