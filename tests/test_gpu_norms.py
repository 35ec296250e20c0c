"""The Frobenius norms of MUON_MODE_HALF: of matrices of many tiles, in work that grows with their size, and of matrices
whose squares fp32 has no values for.

A norm adds up squares rounded to fp32 in partial sums of at most 40 terms in sequence (a thread's 32, eight warps; then the
parts of a thread, averaged over 256 of them): its relative error stays below 64 * 2^-24.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from muon_newton_schulz_07_b200 import binding as B
from muon_newton_schulz_07_b200.optimizer import MuonStep, QuantizedState

from helpers import rel_fro, to_f64

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


# On chip: one CTA, one matrix in two column ranges, clusters; one 256 x 256 tile; tiles; many tiles
SHAPES = [(3, 64, 96), (5, 64, 768), (2, 128, 2048), (100, 333), (700, 64), (2, 200, 250), (331, 503), (512, 1024)]
SIZES = [2.0 ** -98, 2.0 ** -83, 2.0 ** -48, 2.0 ** 49, 2.0 ** 67, 2.0 ** 110]
DIRECTION = 2.5e-3          # fp16 operands: an eighth of the 2e-2 that bf16 operands are held to


def direction(x):
    return O.newton_schulz(np.asarray(x, np.float64), 5, O.QUINTIC, 0.0)


def each(t):
    a = to_f64(t)
    return list(a) if a.ndim == 3 else [a]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_matrices_of_any_size(shape, dtype):
    """Finite matrices whose squares fp32 has no values for, far too large or too small (eps = 0), on every path."""
    op = MuonStep([shape], mode="half")
    base = normal(shape, 3, torch.float32)
    out = torch.empty_like(base)
    for size in SIZES:
        x = (base * size).to(dtype)
        op.orthogonalize([x], [out], eps=0.0)
        norms = op.norms().double().cpu().numpy()
        for e, (a, o) in enumerate(zip(each(x), each(out))):
            n = np.linalg.norm(a)
            assert abs(norms[e] - n) <= NORM * n, (size, norms[e], n)
            assert rel_fro(o, direction(a)) <= DIRECTION, size
    assert op.status() == B.MUON_OK
    op.close()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_norm_beyond_fp32(shape):
    """Entries near the largest fp32 value: the norm, as fp32, is infinite, and the direction is what it is."""
    op = MuonStep([shape], mode="half")
    x = normal(shape, 3, torch.float32).clamp(-3.9, 3.9) * 2.0 ** 126
    x += 2.0 ** 126 * x.sign()                          # entries from a quarter of the largest value
    x = x.clamp(-3.4e38, 3.4e38)
    out = torch.empty_like(x)
    op.orthogonalize([x], [out])
    assert bool(torch.isinf(op.norms()).all())
    for a, o in zip(each(x), each(out)):
        assert rel_fro(o, direction(a)) <= DIRECTION
    op.close()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_sizes_mixed_in_one_matrix(shape):
    """One value far beyond the others', rows of values far below them, and zeros."""
    op = MuonStep([shape], mode="half")
    for top in (1.0, 2.0 ** 70):
        x = normal(shape, 4, torch.float32)
        x[..., 1, :] *= 2.0 ** -70
        x[..., 2, :] = 0
        x[..., 3, 5] = top
        out = torch.empty_like(x)
        op.orthogonalize([x], [out], ns_steps=0)        # X0 by itself, rounded to fp16
        for a, o, n in zip(each(x), each(out), op.norms().double().cpu().numpy()):
            want = np.linalg.norm(a)
            assert abs(n - want) <= NORM * want
            assert np.all(np.abs(o - a / want) <= (2.0 ** -11 + 2.0 ** -17) * np.abs(a / want) + 2.0 ** -36)
    op.close()


@pytest.mark.parametrize("shape", [(3, 64, 96), (5, 60, 770), (2, 128, 2048), (331, 503), (512, 1024)], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_steps_on_gradients_of_any_size(shape, dtype):
    """W takes the direction whatever the gradient's size: with a dense momentum, and with an 8-bit one.

    The 8-bit state starts at zero, so that m = 0 and u = (1 - beta) (1 + beta) g exactly but for fp32 roundings: the
    direction is g's.
    """
    op = MuonStep([shape], dtype=dtype, mode="half")
    base = normal(shape, 5, torch.float32)
    r, c = shape[-2:]
    scale = O.shape_scale(r, c)
    for size in SIZES:
        g = (base * size).to(dtype)
        u = torch.empty_like(g)
        want = [direction(a) for a in each(g)]
        for m in ([torch.zeros_like(g)], QuantizedState([shape], fmt="e4m3")):
            w = torch.zeros_like(g)
            op([w], [g], m, lr=1.0, beta=0.5, eps=0.0)
            norms = op.norms().double().cpu().numpy()
            for a, b, o, n in zip(each(g), each(w), want, norms):
                assert rel_fro(-b / scale, o) <= DIRECTION + torch.finfo(dtype).eps / 2, size
                ref = 0.75 * np.linalg.norm(a)
                assert abs(n - ref) <= NORM * ref, size
        got = op.momentum([g], QuantizedState([shape]), [u], beta=0.5).double().cpu().numpy()
        for a, n in zip(each(g), got):
            ref = 0.75 * np.linalg.norm(a)              # (of u as it is stored, rounded once, where fp32 has no squares)
            assert abs(n - ref) <= (NORM + torch.finfo(dtype).eps / 2) * ref, size
    assert op.status() == B.MUON_OK
    op.close()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_what_is_not_finite_is_nan(shape):
    op = MuonStep([shape], mode="half")
    for bad in (float("inf"), float("nan")):
        x = normal(shape, 6, torch.float32)
        x[..., 4, 3] = bad
        out = torch.empty_like(x)
        for k in (0, 5):
            op.orthogonalize([x], [out], ns_steps=k)
            assert bool(torch.isnan(out).all())
            assert not bool(torch.isfinite(op.norms()).any())
    op.close()
