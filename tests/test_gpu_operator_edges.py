"""Views, 8-bit state and HALF steps where calls meet: offsets beyond 32 bits, graphs that share a handle, gradients that are
not finite, long lists, padding, and lists that would race.

Tolerances are those of test_gpu_half.py (direction) and test_gpu_state.py (codes, scales and U bit for bit).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
import state_reference as R
from muon_newton_schulz_07_b200 import binding as B
from muon_newton_schulz_07_b200.optimizer import QUINTIC, MuonStep, QuantizedState

from helpers import rel_fro, to_f64

pytestmark = pytest.mark.gpu

DIRECTION = 2.5e-3          # an eighth of the 2e-2 that bf16 operands are held to
BF16 = 2.0 ** -8


def values(shape, seed, dtype=torch.bfloat16):
    return torch.from_numpy(1e-2 * np.random.default_rng(seed).standard_normal(shape)).to("cuda", dtype)


def f32(t):
    return t.detach().float().cpu().numpy()


def direction(x):
    return O.newton_schulz(np.asarray(x, np.float64), 5, O.QUINTIC, 1e-7)


def test_lists_that_would_race_are_refused():
    shapes = [(64, 64), (64, 64), (200, 300)]
    op = MuonStep(shapes, mode="half")
    a = [values(s, i) for i, s in enumerate(shapes)]
    o = [torch.empty_like(x) for x in a]
    state = QuantizedState(shapes)
    twice = QuantizedState(shapes)
    twice.codes[1] = twice.codes[0]
    shared = QuantizedState(shapes)
    shared.scales[1] = shared.scales[0]
    calls = [lambda: op.orthogonalize(a, [o[0], o[0], o[2]]),          # an output twice
             lambda: op.orthogonalize(a, [a[1], a[0], o[2]]),          # a list given back in another order
             lambda: op.orthogonalize(a, [a[0].mT, o[1], o[2]]),       # in place, but transposed
             lambda: op.orthogonalize(a, [a[0].view(torch.float16), o[1], o[2]]),
             lambda: op.momentum(a, state, [o[0], o[0], o[2]]),
             lambda: op.momentum(a, state, [a[1], a[0], o[2]]),
             lambda: op.momentum(a, twice, o),
             lambda: op.momentum(a, shared, o),
             lambda: op([o[0], o[0], o[2]], a, state),
             lambda: op(o, a, twice),
             lambda: op([o[0], o[0], o[2]], a, [torch.zeros_like(x) for x in a]),
             lambda: op(o, a, [o[1], torch.zeros_like(o[1]), torch.zeros_like(o[2])]),
             lambda: twice.write(a),
             lambda: shared.write(a),
             lambda: state.read([o[0], o[0], o[2]])]
    for i, call in enumerate(calls):
        with pytest.raises(B.MuonError) as e:
            call()
        assert e.value.code == B.MUON_ERR_INVALID_ARG, i
    with pytest.raises(ValueError):                                     # a list that has lost an entry
        state.codes.pop()
        state.write(a)
    op.orthogonalize([a[0], a[0], a[2]], o)                             # an input may come twice
    assert torch.equal(o[0], o[1]) and rel_fro(to_f64(o[0]), direction(to_f64(a[0]))) <= DIRECTION + BF16
    op.close()


@pytest.mark.parametrize("shape", [(3, 64, 768), (3, 320, 512), (3, 100, 333)], ids=str)
def test_offsets_beyond_32_bits(shape):
    far = (1_100_000_000, shape[2], 1)                                  # the last matrix starts past 2^31 elements
    src = torch.empty(2 * far[0] + shape[1] * shape[2], dtype=torch.bfloat16, device="cuda")
    dst = torch.empty_like(src)
    x, o = src.as_strided(shape, far), dst.as_strided(shape, far)
    x.copy_(values(shape, 1))
    op = MuonStep([shape], mode="half")
    op.orthogonalize([x], [o])
    for e in range(3):
        assert rel_fro(to_f64(o[e].contiguous()), direction(to_f64(x[e].contiguous()))) <= DIRECTION + BF16
    state, ref = QuantizedState([shape]), QuantizedState([shape])
    m = x.contiguous()
    state.write([x], seed=3)
    ref.write([m], seed=3)
    assert torch.equal(state.codes[0], ref.codes[0]) and torch.equal(state.scales[0], ref.scales[0])
    state.read([o])
    back = torch.empty_like(m)
    ref.read([back])
    assert torch.equal(o, back)
    u = torch.empty_like(m)
    op.momentum([x], state, [o], seed=4)
    op.momentum([m], ref, [u], seed=4)
    assert torch.equal(o, u) and torch.equal(state.codes[0], ref.codes[0])
    w = values(shape, 2)
    o.copy_(w)
    op([o], [x], state, seed=5, weight_decay=0.1)
    op([w], [m], ref, seed=5, weight_decay=0.1)
    assert torch.equal(o, w) and torch.equal(state.codes[0], ref.codes[0])
    assert op.status() == B.MUON_OK
    op.close()


def test_rows_and_columns_far_apart():
    ld = 40_000_000                                                     # 64 of them pass 2^31 elements
    buf = torch.empty(63 * ld + 1024, dtype=torch.bfloat16, device="cuda")
    for m, n in ((64, 768), (64, 40)):
        for by_rows in (True, False):
            shape = (m, n) if by_rows else (n, m)
            x = buf.as_strided(shape, (ld, 1) if by_rows else (1, ld))
            x.copy_(values(shape, 3))
            want = direction(to_f64(x.contiguous()))
            op = MuonStep([shape], mode="half")
            out = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
            op.orthogonalize([x], [out])
            assert rel_fro(to_f64(out), want) <= DIRECTION + BF16
            op.orthogonalize([x], [x])                                  # in place
            assert torch.equal(x, out)
            op.close()


def test_a_state_beyond_32_bits():
    shape = (2, 40_000, 32_768)                                         # 2.6 G codes, the second matrix past 2^30
    gen = torch.Generator("cuda").manual_seed(1)
    x = torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(generator=gen)
    state = QuantizedState([shape])
    state.write([x])
    out = torch.empty_like(x)
    state.read([out])
    for e, rows in ((0, slice(0, 3)), (0, slice(39_998, 40_000)), (1, slice(0, 2)), (1, slice(39_997, 40_000))):
        q, s = R.encode(f32(x[e, rows]), "int8")                        # to nearest: a row by itself
        assert np.array_equal(f32(state.codes[0][e, rows].float()), q) and np.array_equal(f32(state.scales[0][e, rows]), s)
        v = torch.from_numpy(np.ascontiguousarray(R.decode(q, s), dtype=np.float32)).to(torch.bfloat16)
        assert torch.equal(out[e, rows].cpu(), v)
    # everywhere: half a code (and the fp32 rounding of up to 127 codes), then bf16's half step of what is read back
    scale = state.scales[0][1].repeat_interleave(128, -1)
    bound = scale * (0.5 * (1 + BF16) + 2.0 ** -14) + x[1].float().abs() * BF16
    assert bool(((out[1].float() - x[1].float()).abs() <= bound).all())


def test_two_graphs_share_a_handle():
    shapes = [(12, 64, 96), (300, 256), (400, 512)]
    op = MuonStep(shapes, mode="half")
    sets = [[values(s, 10 * k + i) for i, s in enumerate(shapes)] for k in range(2)]
    outs = [[torch.empty_like(x) for x in X] for X in sets]
    eager = [[torch.empty_like(x) for x in X] for X in sets]
    for X, E in zip(sets, eager):
        op.orthogonalize(X, E)
    graphs = []
    for X, out in zip(sets, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            op.orthogonalize(X, out)
        graphs.append(g)
    for order in ((0, 1, 0), (1, 0, 0), (1, 1, 0)):                     # in turn, on one stream
        for out in outs:
            for o in out:
                o.zero_()
        for k in order:
            graphs[k].replay()
        torch.cuda.synchronize()
        for k in set(order):
            assert all(torch.equal(a, b) for a, b in zip(outs[k], eager[k]))
    del graphs
    op.close()


def test_a_captured_step_replays():
    shapes = [(3, 64, 96), (300, 256)]
    op = MuonStep(shapes, mode="half")
    G = [values(s, i) for i, s in enumerate(shapes)]
    W = [values(s, 20 + i) for i, s in enumerate(shapes)]
    W2 = [w.clone() for w in W]
    a, b = QuantizedState(shapes), QuantizedState(shapes)
    op(W2, G, b, seed=7)                                                # eager, three times with the captured seed
    for _ in range(2):
        op(W2, G, b, seed=7)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        op(W, G, a, seed=7)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    for x, y in zip(W + a.codes + a.scales, W2 + b.codes + b.scales):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    del g
    op.close()


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("shape", [(4, 64, 96), (4, 130, 260), (4, 320, 512)], ids=str)
def test_a_bad_gradient_stays_alone(shape, bad):
    op = MuonStep([shape], mode="half")
    G = values(shape, 1)
    W = [values(shape, 2)]
    good = [W[0].clone()]
    a, b = QuantizedState([shape], fmt="e4m3"), QuantizedState([shape], fmt="e4m3")
    op(good, [G], b, seed=1)
    G[2, 5, 7] = bad
    op(W, [G], a, seed=1)
    assert op.status() == B.MUON_OK
    assert torch.isnan(W[0][2]).all()
    back = [torch.empty_like(G)]
    a.read(back)
    assert torch.isnan(back[0][2, 5, : min(128, shape[2])]).all() and int(torch.isnan(back[0]).sum()) == min(128, shape[2])
    for e in (0, 1, 3):
        assert torch.equal(W[0][e], good[0][e])
        assert torch.equal(a.codes[0][e].view(torch.uint8), b.codes[0][e].view(torch.uint8))
        assert torch.equal(a.scales[0][e], b.scales[0][e])
    op.close()


def test_more_states_than_a_launch_takes():
    rng = np.random.default_rng(5)
    shapes = [(int(rng.integers(1, 40)), int(rng.choice([4, 12, 100, 128, 129, 256, 1000]))) for _ in range(101)]
    X = [values(s, 100 + i) for i, s in enumerate(shapes)]
    state = QuantizedState(shapes, fmt="e4m3")
    state.write(X, seed=9)
    op = MuonStep(shapes, mode="half")
    U = [torch.empty_like(x) for x in X]
    before = [(f32(q.float()), f32(s)) for q, s in zip(state.codes, state.scales)]
    norms = op.momentum(X, state, U, beta=0.5, seed=11)
    for i, x in enumerate(X):
        q0, s0 = R.encode(f32(x), "e4m3", 9, i)
        assert np.array_equal(before[i][0], q0) and np.array_equal(before[i][1], s0), shapes[i]
        m1, u = R.momentum(R.decode(q0.astype(np.float64), s0), f32(x), 0.5, True)
        q, s = R.encode(m1, "e4m3", 11, i)
        assert np.array_equal(f32(state.codes[i].float()), q) and np.array_equal(f32(state.scales[i]), s), shapes[i]
        want = float(np.linalg.norm(u.astype(np.float64)))
        assert abs(float(norms[i]) - want) <= 40 * 2.0 ** -24 * want
    op.close()


@pytest.mark.parametrize("schedule", ["staged", "fused"])
@pytest.mark.parametrize("mode", ["half", "fast"])
def test_slices_of_padding(mode, schedule):
    """Rows and columns one beyond, and one short of, the slices of 64 that the products run over."""
    shapes = [(193, 300), (257, 321), (320, 705), (449, 450), (700, 255)]
    op = MuonStep(shapes, mode=mode, schedule=schedule)
    X = [values(s, 30 + i) for i, s in enumerate(shapes)]
    Os = [torch.empty_like(x) for x in X]
    op.orthogonalize(X, Os)
    assert op.status() == B.MUON_OK
    for x, o in zip(X, Os):
        assert rel_fro(to_f64(o), direction(to_f64(x))) <= (DIRECTION if mode == "half" else 2e-2) + BF16, tuple(x.shape)
    op.close()
