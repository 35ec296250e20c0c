"""The 8-bit state's definition in elementary NumPy steps: fp32 where the definition rounds each operation to fp32 (the
codes), float64 where it does not (the bounds).  Written from the formulas, shared by the CPU and GPU tests."""
from __future__ import annotations

import numpy as np

BLOCK = 128
TOP = {"int8": np.float32(127.0), "e4m3": np.float32(448.0)}


def mixed(h):
    h = np.asarray(h, np.uint64) & 0xFFFFFFFF
    for shift, factor in ((16, 0x6A09E667), (15, 0xBB67AE85), (16, 1)):
        h = h ^ (h >> np.uint64(shift))
        h = (h * np.uint64(factor)) & np.uint64(0xFFFFFFFF)
    return h


def random_bits(seed, matrix, rows, cols):
    place = np.arange(rows * cols, dtype=np.uint64)
    key = mixed(mixed(np.uint64(seed & 0xFFFFFFFF)) ^ np.uint64(matrix))
    pair = mixed((place >> np.uint64(1)) + key)
    return ((pair >> (np.uint64(16) * (place & np.uint64(1)))) & np.uint64(0xFFFF)).reshape(rows, cols)


def e4m3_grid(y):
    """y (fp32, |y| <= 448 and a little) to the nearest e4m3 value, ties to even."""
    a = np.abs(y).astype(np.float64)
    step = np.exp2(np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.copysign(np.minimum(np.rint(a / step) * step, 448.0), y)


def encode(x, fmt, seed=None, matrix=0):
    """(values the codes stand for before scaling, scales) of one rows x cols fp32 matrix."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    bits = None if seed is None else random_bits(seed, matrix, rows, cols)
    q = np.zeros((rows, cols), np.float64)
    scales = np.zeros((rows, -(-cols // BLOCK)), np.float32)
    for b in range(scales.shape[1]):
        at = slice(b * BLOCK, min(cols, (b + 1) * BLOCK))
        part = x[:, at]
        top = np.abs(part).max(axis=1)
        bad = ~np.isfinite(part).all(axis=1)
        live = ~bad & (top >= np.float32(2.0 ** -100))
        safe = np.where(live, top, np.float32(1))
        mul = np.where(live, TOP[fmt] / safe, np.float32(0)).astype(np.float32)
        scales[:, b] = np.where(bad, np.float32(np.nan), np.where(live, safe / TOP[fmt], np.float32(0)))
        y = (np.where(live[:, None], part, np.float32(0)) * mul[:, None]).astype(np.float32)
        if bits is None:
            q[:, at] = np.clip(np.rint(y), -127, 127) if fmt == "int8" else e4m3_grid(y)
            continue
        u = (bits[:, at].astype(np.float32) * np.float32(2.0 ** -16)).astype(np.float32)
        if fmt == "int8":
            q[:, at] = np.clip(np.floor((y + u).astype(np.float32)), -127, 127)
            continue
        a = np.abs(y)
        cut = (a.view(np.uint32).astype(np.uint64) + (bits[:, at] << np.uint64(4))) & np.uint64(0xFFF00000)
        normal = cut.astype(np.uint32).view(np.float32)
        small = np.floor((a * np.float32(512) + u).astype(np.float32)) * 2.0 ** -9
        q[:, at] = np.copysign(np.minimum(np.where(a >= 2.0 ** -6, normal, small), 448.0), y)
    return q, scales


def spread(scales, cols):
    return np.repeat(scales, BLOCK, axis=1)[:, :cols]


def decode(q, scales):
    """fp32 values: one product of a code and its scale."""
    with np.errstate(invalid="ignore"):
        return (q.astype(np.float32) * spread(scales, q.shape[1])).astype(np.float32)


def momentum(m, g, beta, nesterov):
    """(m1, u) in fp32, every operation rounded by itself."""
    beta = np.float32(beta)
    rest = np.float32(1) - beta
    g = (np.asarray(g, np.float32) * rest).astype(np.float32)
    m1 = ((np.asarray(m, np.float32) * beta).astype(np.float32) + g).astype(np.float32)
    u = (g + (m1 * beta).astype(np.float32)).astype(np.float32) if nesterov else m1
    return m1, u
