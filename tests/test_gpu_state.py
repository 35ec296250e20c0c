"""8-bit state on the GPU: writing, reading back, the momentum on it, and a step on it.

The kernels round every fp32 operation of the definition by itself, so codes, scales, U and the values read
back are compared bit for bit with the fp32 formula (state_reference.py); its own bounds are tested on the CPU.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
import state_reference as R
from muon_newton_schulz_07_b200 import binding as B
from muon_newton_schulz_07_b200.optimizer import MuonStep, QuantizedState

from helpers import rel_fro, to_f64

pytestmark = pytest.mark.gpu

DTYPES = [torch.bfloat16, torch.float16, torch.float32]
SHAPES = [(1, 1), (1, 7), (3, 128), (5, 129), (70, 256), (64, 1100), (2, 3, 40), (9, 1, 130), (3, 65, 384), (1, 70001)]


def random(shape, dtype, seed=0, heavy=True):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape)
    if heavy:
        x = x * np.where(rng.random(shape) < 0.02, 100.0, 1.0)
    return torch.from_numpy(x * 1e-2).to("cuda", dtype)


def matrices(t):
    """fp32 NumPy matrices of a tensor that is one matrix or a stack."""
    a = t.detach().float().cpu().numpy()
    return list(a) if a.ndim == 3 else [a]


def codes_of(state, i):
    return matrices(state.codes[i].float())


def same(a, b):
    return np.array_equal(np.asarray(a, np.float64), np.asarray(b, np.float64), equal_nan=True)


def rounded(a, dtype):
    return matrices(torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(dtype))[0]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("seed", [None, 12345, -1])
@pytest.mark.parametrize("dtype", DTYPES)
def test_write_and_read_back(fmt, seed, dtype):
    X = [random(s, dtype, i) for i, s in enumerate(SHAPES)]
    state = QuantizedState(SHAPES, fmt=fmt)
    state.write(X, seed=seed)
    outs = {}
    for out_dtype in DTYPES:
        outs[out_dtype] = [torch.empty(s, dtype=out_dtype, device="cuda") for s in SHAPES]
        state.read(outs[out_dtype])
    torch.cuda.synchronize()
    matrix = 0
    for i, x in enumerate(X):
        for e, m in enumerate(matrices(x)):
            q, s = R.encode(m, fmt, seed, matrix)
            matrix += 1
            assert same(codes_of(state, i)[e], q), (SHAPES[i], e)
            assert same(matrices(state.scales[i])[e], s), (SHAPES[i], e)
            v = R.decode(q, s)
            for out_dtype in DTYPES:
                assert same(matrices(outs[out_dtype][i])[e], rounded(v, out_dtype)), (SHAPES[i], e, out_dtype)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_blocks_without_a_size_and_edges(fmt):
    x = torch.zeros(6, 200, device="cuda")
    x[1] = 2.0 ** -101
    x[2, 5] = float("inf")
    x[3, 150] = float("nan")
    x[4] = torch.linspace(-1, 1, 200, device="cuda") * 3e38
    x[5] = torch.linspace(-1, 1, 200, device="cuda") * 2.0 ** -99
    state = QuantizedState([(6, 200)], fmt=fmt)
    for seed in (None, 3):
        state.write([x], seed=seed)
        q, s = R.encode(x.cpu().numpy(), fmt, seed)
        assert same(codes_of(state, 0)[0], q) and same(matrices(state.scales[0])[0], s)
        out = torch.empty(6, 200, device="cuda")
        state.read([out])
        assert same(matrices(out)[0], R.decode(q, s))
        assert torch.isnan(out[2, :128]).all() and torch.isnan(out[3, 128:]).all() and (out[:2] == 0).all()


def test_strided_rows_and_misaligned_pointers():
    wide = random((6, 3 * 130 + 8), torch.bfloat16)
    x = wide[:, 3:133]                                   # rows 398 apart, base not 16-byte aligned
    stack = random((40, 4 * 64), torch.bfloat16, 1).view(40, 4, 64).transpose(0, 1)   # column slices
    state = QuantizedState([(6, 130), (4, 40, 64)], fmt="e4m3")
    state.write([x, stack])
    out_wide = torch.full_like(wide, 7.0)
    out_stack = torch.full((40, 4 * 64), 7.0, dtype=torch.bfloat16, device="cuda")
    state.read([out_wide[:, 3:133], out_stack.view(40, 4, 64).transpose(0, 1)])
    for e, m in enumerate([x.contiguous()] + list(stack.contiguous())):
        q, s = R.encode(matrices(m)[0], "e4m3")
        got = out_wide[:, 3:133] if e == 0 else out_stack.view(40, 4, 64)[:, e - 1]
        assert same(matrices(got.contiguous())[0], rounded(R.decode(q, s), torch.bfloat16))
    assert (out_wide[:, :3] == 7).all() and (out_wide[:, 133:] == 7).all()   # around the view: as it was


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("seed", [None, 99])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mode", ["half", "fast"])
def test_momentum(fmt, seed, dtype, mode):
    shapes = [(5, 129), (3, 64, 256), (1, 1), (33, 1000), (700, 16)]
    step = MuonStep(shapes, dtype=dtype, mode=mode)
    state = QuantizedState(shapes, fmt=fmt)
    state.write([random(s, dtype, 50 + i) for i, s in enumerate(shapes)])
    for t, nesterov in enumerate([True, False, True]):
        G = [random(s, dtype, 10 * t + i) for i, s in enumerate(shapes)]
        before = [(matrices(q.float()), matrices(s)) for q, s in zip(state.codes, state.scales)]
        U = [torch.empty_like(g) for g in G] if t < 2 else G           # U may be G
        Gm = [matrices(g) for g in G]
        norms = step.momentum(G, state, U, beta=0.9, nesterov=nesterov, seed=None if seed is None else seed + t)
        torch.cuda.synchronize()
        matrix = 0
        for i in range(len(shapes)):
            for e, g in enumerate(Gm[i]):
                m = R.decode(before[i][0][e].astype(np.float64), before[i][1][e])
                m1, u = R.momentum(m, g, 0.9, nesterov)
                q, s = R.encode(m1, fmt, None if seed is None else seed + t, matrix)
                assert same(matrices(U[i])[e], rounded(u, dtype)), (shapes[i], e, t)
                assert same(codes_of(state, i)[e], q) and same(matrices(state.scales[i])[e], s), (shapes[i], e, t)
                # a sum of N squares in fp32, in parts: at most about log2(N) + 40 roundings a term, half of that
                # in the root, each 2^-24
                want = float(np.linalg.norm(u.astype(np.float64)))
                assert abs(float(norms[matrix]) - want) <= 40 * 2.0 ** -24 * want
                matrix += 1
    step.close()


def exact_step(w, g, m, hp, fmt):
    m1, u = R.momentum(m, g, hp.beta, hp.nesterov)
    o = O.newton_schulz(u.astype(np.float64), hp.ns_steps, hp.abc, hp.eps)
    return (1 - hp.lr * hp.weight_decay) * w - hp.lr * O.shape_scale(*w.shape) * o, o, m1


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_steps_on_quantized_momentum(dtype, fmt):
    """Three steps as a trainer makes them: write the state once, step, read it back.  Each is compared with the float64
    step from the state the GPU had before it.  The direction's budget is an eighth of the 2e-2 that bf16 operands are
    held to (fp16's step is an eighth of bf16's; U is rounded once, to fp16); then W's own rounding."""
    shapes = [(96, 64), (3, 64, 256), (130, 300), (512, 256), (40, 40)]
    step = MuonStep(shapes, dtype=dtype, mode="half")
    state = QuantizedState(shapes, fmt=fmt)
    state.write([random(s, dtype, 70 + i, heavy=False) for i, s in enumerate(shapes)], seed=1)
    W = [random(s, dtype, 90 + i, heavy=False) for i, s in enumerate(shapes)]
    hp = O.Hyper(lr=0.02, beta=0.95, weight_decay=0.1, eps=1e-7, nesterov=True, ns_steps=5)
    direction = 2.5e-3
    eps = torch.finfo(dtype).eps / 2
    for t in range(3):
        G = [random(s, dtype, 1000 * t + i) for i, s in enumerate(shapes)]
        W0 = [matrices(w) for w in W]
        M0 = [[R.decode(q.astype(np.float64), s) for q, s in zip(codes_of(state, i), matrices(state.scales[i]))]
              for i in range(len(shapes))]
        step(W, G, state, lr=hp.lr, beta=hp.beta, weight_decay=hp.weight_decay, seed=5 + t)
        assert step.status() == B.MUON_OK
        matrix = 0
        for i in range(len(shapes)):
            for e, g in enumerate(matrices(G[i])):
                w1, o, m1 = exact_step(W0[i][e].astype(np.float64), g, M0[i][e], hp, fmt)
                scale = hp.lr * O.shape_scale(*w1.shape)
                err = np.linalg.norm(matrices(W[i])[e] - w1)
                assert err <= direction * scale * np.linalg.norm(o) + eps * np.linalg.norm(w1), (shapes[i], e, t)
                q, s = R.encode(m1, fmt, 5 + t, matrix)
                assert same(codes_of(state, i)[e], q) and same(matrices(state.scales[i])[e], s)
                matrix += 1
    step.close()


def test_step_state_equals_its_parts():
    """The step is its parts in order: momentum into U, the orthogonaliser on U, the parameter write."""
    shapes = [(64, 768), (300, 512)]
    step = MuonStep(shapes, mode="half")
    G = [random(s, torch.bfloat16, i) for i, s in enumerate(shapes)]
    a, b = QuantizedState(shapes), QuantizedState(shapes)
    for s in (a, b):
        s.write(G, seed=4)
    W = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in shapes]
    step(W, G, a, lr=1.0, seed=6)
    U = [torch.empty_like(g) for g in G]
    O_ = [torch.empty_like(g) for g in G]
    step.momentum(G, b, U, seed=6)
    step.orthogonalize(U, O_)
    for w, o, x, y in zip(W, O_, a.codes + a.scales, b.codes + b.scales):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
        # momentum() rounds U to bf16 (the bf16 budget of the direction), the step does not; then both results to bf16
        assert rel_fro(-to_f64(w), to_f64(o)) <= 2e-2 + 2 * 2.0 ** -8
    step.close()


def test_captured_write_and_read():
    shapes = [(33, 300)]
    x = random(shapes[0], torch.bfloat16)
    state, out = QuantizedState(shapes), torch.empty(shapes[0], dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        state.write([x], seed=3)
        state.read([out])
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        state.write([x], seed=3)
        state.read([out])
    x.copy_(random(shapes[0], torch.bfloat16, 5))
    graph.replay()
    torch.cuda.synchronize()
    q, s = R.encode(matrices(x)[0], "int8", 3)
    assert same(matrices(out)[0], rounded(R.decode(q, s), torch.bfloat16))


def test_refusals():
    shapes = [(8, 256)]
    step, state = MuonStep(shapes, mode="half"), QuantizedState(shapes)
    g = [torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")]
    with pytest.raises(ValueError):
        QuantizedState(shapes, fmt="int4")
    with pytest.raises(ValueError):
        state.write([g[0].t().contiguous().t()])             # stored by columns
    with pytest.raises(ValueError):
        state.write([g[0].double()])
    with pytest.raises(ValueError):
        state.write([g[0].cpu()])
    with pytest.raises(ValueError):
        state.write([])
    with pytest.raises(ValueError):
        step(g, g, QuantizedState([(256, 8)]))
    with pytest.raises(ValueError):
        step(g, g, g, seed=1)                                 # nothing to round
    with pytest.raises(ValueError):
        MuonStep(shapes)(g, g, state)                         # bf16 operands: no 8-bit momentum
    with pytest.raises(ValueError):
        step.momentum([g[0].float()], state, g)
    state.codes[0] = torch.zeros(8, 255, dtype=torch.int8, device="cuda")
    with pytest.raises(ValueError):
        state.read(g)
    with pytest.raises(B.MuonError) as e:  # a state of another shape, past the Python checks
        ok = QuantizedState([(8, 128)])
        B.muon_momentum_state(step.handle, B.views([(g[0].data_ptr(), 1, 0, 256, 1, B.MUON_BF16)]), ok._states(),
                              B.views([(g[0].data_ptr(), 1, 0, 256, 1, B.MUON_BF16)]), 1, 0, B.make_hparams(), None, 0)
    assert e.value.code == B.MUON_ERR_INVALID_ARG
    step.close()
