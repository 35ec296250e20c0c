"""CPU checks around the 8-bit state: the reference formula against bounds that follow from the definition, and
the refusals of the entry points that need no device."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

import state_reference as R
from muon_newton_schulz_07_b200 import binding as B
from muon_newton_schulz_07_b200 import build as build_mod


@pytest.fixture(scope="module", autouse=True)
def built_library():
    build_mod.build()
    return B.lib()


def values(rows, cols, seed=0):
    rng = np.random.default_rng(seed)
    return (rng.standard_normal((rows, cols)) * np.where(rng.random((rows, cols)) < 0.01, 100.0, 1.0)).astype(np.float32)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("seed", [None, 7])
def test_rounding_stays_within_a_step(fmt, seed):
    """To nearest the value is off by at most half a spacing of the codes, stochastic by less than a whole one; the fp32
    arithmetic of y = x * (T / t) and of the product with the scale adds a few 2^-24 of the value."""
    x = values(5, 300)
    q, s = R.encode(x, fmt, seed)
    s64 = R.spread(s, 300).astype(np.float64)
    y = np.abs(x.astype(np.float64)) / s64
    spacing = np.ones_like(y) if fmt == "int8" else np.exp2(np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
    err = np.abs(q * s64 - x)
    assert np.all(err <= spacing * s64 * (0.5 if seed is None else 1.0) + 8 * 2.0 ** -24 * np.abs(x))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_stochastic_rounding_is_unbiased(fmt):
    """The mean over n seeds of a value rounded up with probability p has standard deviation at most spacing / (2 sqrt n);
    six of them, and the 2^-17 of a spacing that 16 bits leave out."""
    x = values(2, 256, 3)
    n = 400
    mean = np.zeros(x.shape)
    for seed in range(n):
        q, s = R.encode(x, fmt, seed)
        mean += q * R.spread(s, 256).astype(np.float64) / n
    s64 = R.spread(s, 256).astype(np.float64)
    y = np.abs(x.astype(np.float64)) / s64
    # the spacing above y counts: next to a power of two the two neighbours lie in different binades
    spacing = np.ones_like(y) if fmt == "int8" else np.exp2(np.floor(np.log2(np.maximum(y, 2.0 ** -6))) - 3)
    bound = spacing * s64 * (6 * 0.5 / np.sqrt(n) + 2.0 ** -16) + 8 * 2.0 ** -24 * np.abs(x)
    # the largest value of a block sits on the last code and cannot round above it
    assert np.all(np.abs(mean - x) <= bound)


def test_random_bits_are_even():
    bits = R.random_bits(11, 2, 512, 512).astype(np.float64) / 2 ** 16
    n = bits.size
    assert abs(bits.mean() - 0.5) < 6 * np.sqrt(1 / 12 / n)
    flat = bits.ravel() - 0.5
    for lag in (1, 2, 3, 128, 512):  # a product of two even numbers has variance 1/144
        assert abs(np.mean(flat[lag:] * flat[:-lag])) < 6 / 12 / np.sqrt(n)
    other = R.random_bits(11, 3, 512, 512).astype(np.float64).ravel() / 2 ** 16 - 0.5
    assert abs(np.mean(flat * other)) < 6 / 12 / np.sqrt(n)


def test_blocks_without_a_size():
    x = np.zeros((4, 130), np.float32)
    x[1, :128] = 2.0 ** -101
    x[2, 129] = np.inf
    x[3, 3] = np.nan
    for fmt in ("int8", "e4m3"):
        q, s = R.encode(x, fmt)
        assert np.all(q == 0) and np.all(s[:2] == 0)
        assert s[2, 0] == 0 and np.isnan(s[2, 1]) and np.isnan(s[3, 0]) and s[3, 1] == 0


# ------------------------------------------------------------------ refusals, before anything touches a device

VIEW = dict(data=4096, count=2, batch_stride=8 * 256, row_stride=256, col_stride=1, dtype=B.MUON_BF16)
STATE = dict(codes=4096, scales=4096, count=2, rows=8, cols=256)


def view(**kw):
    return B.views([tuple({**VIEW, **kw}.values())])


def state(**kw):
    return B.states([tuple({**STATE, **kw}.values())])


@pytest.mark.parametrize("bad_view, bad_state, code", [
    (dict(data=None), {}, B.MUON_ERR_INVALID_ARG),
    (dict(data=4097), {}, B.MUON_ERR_INVALID_ARG),
    (dict(dtype=9), {}, B.MUON_ERR_INVALID_ARG),
    (dict(count=3), {}, B.MUON_ERR_INVALID_ARG),
    (dict(row_stride=-256), {}, B.MUON_ERR_INVALID_ARG),
    (dict(col_stride=2), {}, B.MUON_ERR_UNSUPPORTED),
    ({}, dict(codes=None), B.MUON_ERR_INVALID_ARG),
    ({}, dict(scales=None), B.MUON_ERR_INVALID_ARG),
    ({}, dict(scales=4098), B.MUON_ERR_INVALID_ARG),
    ({}, dict(rows=0), B.MUON_ERR_INVALID_ARG),
    ({}, dict(cols=-1), B.MUON_ERR_INVALID_ARG),
    ({}, dict(rows=2 ** 30, cols=512), B.MUON_ERR_UNSUPPORTED),
    ({}, dict(rows=2 ** 40), B.MUON_ERR_UNSUPPORTED),
])
def test_state_calls_refuse(bad_view, bad_state, code):
    for call in (lambda: B.muon_state_quantize(view(**bad_view), state(**bad_state), 1, B.MUON_STATE_INT8, None, 0),
                 lambda: B.muon_state_dequantize(state(**bad_state), view(**bad_view), 1, B.MUON_STATE_E4M3, 0)):
        with pytest.raises(B.MuonError) as e:
            call()
        assert e.value.code == code


def test_overlapping_output_and_formats_refused():
    with pytest.raises(B.MuonError) as e:  # rows that overlap may be read but not written
        B.muon_state_dequantize(state(), view(row_stride=100), 1, B.MUON_STATE_INT8, 0)
    assert e.value.code == B.MUON_ERR_INVALID_ARG
    for n, fmt in ((-1, 0), (1, 2)):
        with pytest.raises(B.MuonError) as e:
            B.muon_state_quantize(view(), state(), n, fmt, None, 0)
        assert e.value.code == B.MUON_ERR_INVALID_ARG
    B.muon_state_quantize(None, None, 0, B.MUON_STATE_INT8, None, 0)   # nothing to do
    lib = B.lib()
    assert lib.muon_state_quantize(None, None, 1, 0, None, None) == B.MUON_ERR_INVALID_ARG
    two = B.views([tuple(VIEW.values()), tuple({**VIEW, "dtype": B.MUON_FP32}.values())])
    with pytest.raises(B.MuonError):  # one type a call
        B.muon_state_quantize(two, B.states([tuple(STATE.values())] * 2), 2, 0, None, 0)


def test_null_handles_refused():
    lib, hp = B.lib(), B.make_hparams()
    assert lib.muon_orthogonalize_views(None, view(), view(), 1, ctypes.byref(hp), None) == B.MUON_ERR_INVALID_ARG
    assert lib.muon_set_coefficients(None, None, 0) == B.MUON_ERR_INVALID_ARG
    assert lib.muon_momentum_state(None, view(), state(), view(), 1, 0, ctypes.byref(hp), None, None) == B.MUON_ERR_INVALID_ARG
    assert lib.muon_step_state(None, view(), view(), state(), 1, 0, ctypes.byref(hp), None, None) == B.MUON_ERR_INVALID_ARG


def test_half_workspace():
    """Groups of at most 128 rows and 4096 columns need no operand buffers, the others the same as with bf16 operands."""
    few = B.muon_workspace_size([(64, 768)], B.MUON_BF16, B.MUON_MODE_HALF)
    assert few < B.muon_workspace_size([(64, 768)], B.MUON_BF16, B.MUON_MODE_FAST)
    for dtype in (B.MUON_BF16, B.MUON_FP32):
        assert B.muon_workspace_size([(512, 768)], dtype, B.MUON_MODE_HALF) == \
            B.muon_workspace_size([(512, 768)], dtype, B.MUON_MODE_FAST)
    with pytest.raises(B.MuonError):
        B.muon_workspace_size([(512, 768)], B.MUON_FP16, B.MUON_MODE_HALF)


def test_one_place_written_twice_is_refused():
    two = lambda make, a, b: make([tuple(a.values()), tuple(b.values())])  # noqa: E731
    for codes, scales in ((4096, 8192), (8192, 4096)):   # codes, or scales, shared by two states
        other = {**STATE, "codes": codes, "scales": scales}
        with pytest.raises(B.MuonError) as e:
            B.muon_state_quantize(two(B.views, VIEW, VIEW), two(B.states, {**STATE, "scales": 12288 if codes == 4096 else 4096}, other), 2,
                                  B.MUON_STATE_INT8, None, 0)
        assert e.value.code == B.MUON_ERR_INVALID_ARG
    with pytest.raises(B.MuonError) as e:                # read back into one tensor twice
        B.muon_state_dequantize(two(B.states, STATE, {**STATE, "codes": 1 << 20}), two(B.views, VIEW, VIEW), 2, B.MUON_STATE_INT8, 0)
    assert e.value.code == B.MUON_ERR_INVALID_ARG
