"""Stochastic rounding at places past 2^33 of a matrix, where the pairs of values pass 2^32: the formula's bits on every path."""
from __future__ import annotations

import numpy as np
import pytest
import torch

import state_reference as R
from muon_newton_schulz_07_b200.optimizer import QuantizedState

pytestmark = pytest.mark.gpu

SEED = 77


def bits(first, shape):
    place = np.arange(first, first + shape[0] * shape[1], dtype=np.uint64)
    key = R.mixed(R.mixed(np.uint64(SEED)) ^ np.uint64(0))
    pair = R.mixed((place >> np.uint64(1)) + key)
    return ((pair >> (np.uint64(16) * (place & np.uint64(1)))) & np.uint64(0xFFFF)).reshape(shape)


# whole blocks back to back; rows of multiples of 4 (the pairs pass 2^32 in the middle of a row); single values
@pytest.mark.parametrize("cols", [32_768, 32_764, 32_765])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_places_beyond_32_bits_of_pairs(cols, fmt, monkeypatch):
    edge = (1 << 33) // cols                            # the row that place 2^33 is in, or starts
    shape = (edge + 4, cols)
    x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator("cuda").manual_seed(cols)
    x[edge - 2:].normal_(generator=gen)
    state = QuantizedState([shape], fmt=fmt)
    state.write([x], seed=SEED)
    monkeypatch.setattr(R, "random_bits", lambda seed, matrix, rows, c: bits((edge - 2) * cols, (rows, c)))
    q, s = R.encode(x[edge - 2:].float().cpu().numpy(), fmt, SEED)
    assert np.array_equal(state.codes[0][edge - 2:].float().cpu().numpy(), q)
    assert np.array_equal(state.scales[0][edge - 2:].cpu().numpy(), s)
