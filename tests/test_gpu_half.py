"""fp16 operands (mode "half"): the orthogonaliser on views and the dense step, against the float64 oracle.

Tolerance of the direction: the bf16 path is held to 2e-2 for the same four roundings an iteration; fp16's
half step, 2^-11, is an eighth of bf16's 2^-8, so 2.5e-3, plus half a step of the type O is stored in.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from muon_newton_schulz_07_b200 import binding as B
from muon_newton_schulz_07_b200.optimizer import QUINTIC, MuonStep

from helpers import assert_m1_elementwise, rel_fro, to_f64

pytestmark = pytest.mark.gpu

SETTLE = (15 / 8, -10 / 8, 3 / 8)
ITERATION = 2.5e-3


def iterate(x, abc, eps=1e-7):
    """The oracle's iteration with one coefficient triple each."""
    x = np.asarray(x, np.float64)
    flip = x.shape[0] > x.shape[1]
    x = x.T if flip else x
    x = x / (np.linalg.norm(x) + eps)
    for a, b, c in abc:
        g = x @ x.T
        x = a * x + (b * g + c * g @ g) @ x
    return x.T if flip else x


def test_the_iteration_used_here_is_the_oracles():
    x = np.random.default_rng(0).standard_normal((20, 9))
    assert rel_fro(iterate(x, [QUINTIC] * 5), O.newton_schulz(x, 5, O.QUINTIC, 1e-7)) < 1e-12


def random(shape, dtype, seed=0, kind="rows"):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal(shape)
    if kind == "rows":
        x = x * 10.0 ** rng.uniform(-4, -2, shape[:-1] + (1,))
    elif kind == "heavy":
        x = 1e-3 * x * np.where(rng.random(shape) < 0.01, 100.0, 1.0)
    return torch.from_numpy(x).to("cuda", dtype)


def matrices(t):
    a = to_f64(t)
    return list(a) if a.ndim == 3 else [a]


def tolerance(dtype):
    return ITERATION + torch.finfo(dtype).eps / 2


def check(shapes, X, Os, abc, op, what=""):
    assert op.status() == B.MUON_OK
    norms = op.norms().cpu().numpy()
    at = 0
    for s, x, o in zip(shapes, X, Os):
        for e, (a, b) in enumerate(zip(matrices(x), matrices(o))):
            want = iterate(a, abc)
            assert np.isfinite(b).all(), (s, e, what)
            err = rel_fro(b, want)
            assert err <= tolerance(o.dtype), (s, e, what, err)
            n = np.linalg.norm(a)
            assert abs(norms[at] - n) <= 40 * 2.0 ** -24 * n, (s, e, what)
            at += 1


ON_CHIP = [(1, 1), (1, 7), (7, 1), (5, 3), (8, 64), (64, 768), (128, 128), (100, 333), (333, 100), (17, 769), (128, 1024),
           (31, 2000), (4096, 128), (3, 4096), (128, 700), (2, 1441), (60, 8000), (25, 626), (16, 20001), (64, 1600),
           (33, 4000), (5, 60001)]
TILED = [(129, 130), (256, 256), (155, 221), (331, 503), (640, 256), (256, 1024), (100, 4097), (300, 1), (5000, 2)]


@pytest.mark.parametrize("shape", ON_CHIP, ids=str)
@pytest.mark.parametrize("kind", ["plain", "rows", "heavy"])
def test_one_matrix_on_chip(shape, kind):
    op = MuonStep([shape], mode="half")
    X, Os = [random(shape, torch.bfloat16, 1, kind)], [torch.empty(shape, dtype=torch.bfloat16, device="cuda")]
    op.orthogonalize(X, Os)
    check([shape], X, Os, [QUINTIC] * 5, op)
    op.close()


@pytest.mark.parametrize("stack", [(2, 64, 64), (12, 64, 768), (300, 20, 70), (37, 128, 256), (700, 1, 9), (200, 3, 500),
                                   (60, 1536, 128), (5, 33, 3000), (320, 64, 128), (9, 25, 626), (32, 11, 993), (50, 4000, 16), (200, 64, 768)], ids=str)
def test_stacks_on_chip(stack):
    op = MuonStep([stack], mode="half")
    X, Os = [random(stack, torch.bfloat16, 2)], [torch.empty(stack, dtype=torch.bfloat16, device="cuda")]
    op.orthogonalize(X, Os, abc=[QUINTIC] * 3 + [SETTLE] * 2)
    check([stack], X, Os, [QUINTIC] * 3 + [SETTLE] * 2, op)
    op.close()


@pytest.mark.parametrize("shape", TILED, ids=str)
def test_one_matrix_tiled(shape):
    op = MuonStep([shape], mode="half")
    for dtype in (torch.bfloat16, torch.float32):
        X, Os = [random(shape, dtype, 3)], [torch.empty(shape, dtype=dtype, device="cuda")]
        op.orthogonalize(X, Os)
        check([shape], X, Os, [QUINTIC] * 5, op, dtype)
    op.close()


def layouts(t):
    """The same values stored by rows, with padding, by columns, and as a misaligned slice."""
    yield "rows", t.contiguous()
    wide = torch.zeros(t.shape[:-1] + (t.shape[-1] + 8,), dtype=t.dtype, device=t.device)
    wide[..., :t.shape[-1]] = t
    yield "padded rows", wide[..., :t.shape[-1]]
    yield "columns", t.mT.contiguous().mT
    off = torch.zeros(t.shape[:-1] + (t.shape[-1] + 3,), dtype=t.dtype, device=t.device)
    off[..., 1:-2] = t
    yield "odd slice", off[..., 1:-2]
    if t.dim() == 3:
        yield "column slices", t.transpose(0, 1).contiguous().transpose(0, 1)


@pytest.mark.parametrize("shape", [(3, 64, 96), (3, 96, 64), (40, 200), (2, 256, 320), (2, 320, 256), (260, 130)], ids=str)
def test_layouts_and_types(shape):
    op = MuonStep([shape], mode="half")
    abc = [QUINTIC] * 4
    want = None
    for xt in (torch.bfloat16, torch.float16, torch.float32):
        base = random(shape, xt, 4, "plain")
        for xn, x in layouts(base):
            for ot in (torch.bfloat16, torch.float16, torch.float32):
                for on, o in layouts(torch.full(shape, 9.0, dtype=ot, device="cuda")):
                    if on != "rows" and xn != "rows" and (xt != torch.bfloat16 or ot != torch.bfloat16):
                        continue
                    op.orthogonalize([x], [o], abc=QUINTIC, ns_steps=4)
                    assert op.status() == B.MUON_OK
                    for a, b in zip(matrices(base), matrices(o)):
                        assert rel_fro(b, iterate(a, abc)) <= tolerance(ot), (xt, xn, ot, on)
    op.close()


def test_output_around_a_view_is_left_alone():
    for shape in [(64, 96), (200, 160)]:
        for off in (1, 8):
            op = MuonStep([shape], mode="half")
            big = torch.full((shape[0] + 2, shape[1] + 16), 5.0, dtype=torch.bfloat16, device="cuda")
            op.orthogonalize([random(shape, torch.bfloat16)], [big[1:-1, off:off + shape[1]]])
            torch.cuda.synchronize()
            inside = torch.zeros_like(big, dtype=torch.bool)
            inside[1:-1, off:off + shape[1]] = True
            assert (big[~inside] == 5).all() and torch.isfinite(big).all()
            op.close()


def test_in_place_and_mixed_sets():
    """Matrices that run on chip and tiled ones in one call, tall and wide in one group, O written over X."""
    shapes = [(64, 768), (512, 256), (4, 256, 512), (768, 64), (300, 200), (130, 70), (200, 300), (2, 640, 1024)]
    op = MuonStep(shapes, mode="half")
    X = [random(s, torch.bfloat16, i) for i, s in enumerate(shapes)]
    ref = [x.clone() for x in X]
    Os = [torch.empty_like(x) for x in X]
    op.orthogonalize(X, Os)
    check(shapes, ref, Os, [QUINTIC] * 5, op)
    assert all(torch.equal(a, b) for a, b in zip(X, ref))
    op.orthogonalize(X, X)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(X, Os))
    op.close()


def test_more_views_and_groups_than_a_launch_takes():
    shapes = [(130 + 2 * (i % 9), 300) for i in range(110)] + [(16, 40 + i % 2) for i in range(150)]
    op = MuonStep(shapes, mode="half")
    X = [random(s, torch.bfloat16, i) for i, s in enumerate(shapes)]
    Os = [torch.empty_like(x) for x in X]
    op.orthogonalize(X, Os)
    check(shapes, X, Os, [QUINTIC] * 5, op)
    op.close()


@pytest.mark.parametrize("shape", [(16, 40), (64, 900), (128, 256), (200, 256)], ids=str)
def test_a_bad_matrix_stays_alone(shape):
    """Not finite, zero and diverging matrices of a stack: the others come out as without them, bit for bit."""
    n = 24
    op = MuonStep([(n,) + shape], mode="half")
    x = random((n,) + shape, torch.float32, 6, "plain")
    good, out = torch.empty_like(x), torch.empty_like(x)
    op.orthogonalize([x], [good])
    bad = x.clone()
    bad[3, 1, 2] = float("nan")
    bad[7, 0, 0] = float("inf")
    bad[8] = 0
    op.orthogonalize([bad], [out])
    assert op.status() == B.MUON_OK
    for e in range(n):
        if e in (3, 7):
            assert torch.isnan(out[e]).all()
        elif e == 8:
            assert (out[e] == 0).all()
        else:
            assert torch.equal(out[e], good[e]), e
    op.orthogonalize([x], [out])              # and nothing stays behind in the workspace
    assert torch.equal(out, good)
    # a polynomial that sends singular value 1 past fp16's range and shrinks those of the others (0.41 at most)
    flat = x.clone()
    flat[5] = 0
    flat[5, :, 0] = 1.0                       # rank one: its singular value is 1
    steep = [(0.1, 0.0, 8.0)] * 3
    op.orthogonalize([flat], [out], abc=steep)
    kept = torch.empty_like(x)
    op.orthogonalize([x], [kept], abc=steep)
    assert not torch.isfinite(out[5]).any()
    assert all(torch.equal(out[e], kept[e]) for e in range(n) if e != 5)
    op.close()


@pytest.mark.parametrize("shape", [(3, 64, 100), (200, 300)], ids=str)
def test_no_iterations_and_eps(shape):
    op = MuonStep([shape], mode="half")
    x = random(shape, torch.float32, 8, "plain")
    o = torch.empty_like(x)
    op.orthogonalize([x], [o], ns_steps=0)
    for a, b in zip(matrices(x), matrices(o)):  # X0 itself: one rounding to fp16 (and a few to fp32)
        assert np.all(np.abs(b - a / (np.linalg.norm(a) + 1e-7)) <= (2.0 ** -11 + 2.0 ** -20) * np.abs(b) + 2.0 ** -36)
    z = torch.zeros_like(x)
    for eps in (1e-7, 0.0):
        op.orthogonalize([z], [o], eps=eps)
        assert (o == 0).all()
    tiny = x * 1e-12                             # a norm far below the usual, eps below it
    op.orthogonalize([tiny], [o], eps=0.0)
    for a, b in zip(matrices(x), matrices(o)):
        assert rel_fro(b, iterate(a, [QUINTIC] * 5, 0.0)) <= tolerance(torch.float32)
    op.close()


def test_coefficients_per_iteration():
    shapes = [(40, 100), (200, 300)]
    op = MuonStep(shapes, mode="half")
    X = [random(s, torch.float32, i, "plain") for i, s in enumerate(shapes)]
    a, b = ([torch.empty_like(x) for x in X] for _ in range(2))
    op.orthogonalize(X, a, abc=[QUINTIC] * 5)
    op.orthogonalize(X, b)                        # back to one triple
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    abc = [(3.0, -3.2, 1.1), QUINTIC, SETTLE, (1.5, -0.5, 0.0)]
    op.orthogonalize(X, a, abc=abc)
    for x, o in zip(X, a):
        assert rel_fro(to_f64(o), iterate(to_f64(x), abc)) <= tolerance(torch.float32)
    B.muon_set_coefficients(op.handle, abc)
    with pytest.raises(B.MuonError) as e:
        B.muon_orthogonalize_views(op.handle, B.views([(x.data_ptr(), 1, 0, x.shape[1], 1, B.MUON_FP32) for x in X]),
                                   B.views([(x.data_ptr(), 1, 0, x.shape[1], 1, B.MUON_FP32) for x in a]), 2,
                                   B.make_hparams(ns_steps=5), 0)
    assert e.value.code == B.MUON_ERR_INVALID_ARG  # five iterations, four triples
    op.close()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dense_step(dtype):
    """muon_step on a "half" handle: M1 element by element, W from the direction."""
    shapes = [(64, 300), (512, 256), (256, 512), (131, 77), (2, 96, 640)]
    op = MuonStep(shapes, dtype=dtype, mode="half")
    W, G, M = ([random(s, dtype, 10 * k + i, "plain") for i, s in enumerate(shapes)] for k in range(3))
    pre = [[matrices(t) for t in (w, g, m)] for w, g, m in zip(W, G, M)]
    hp = O.Hyper(lr=0.02, beta=0.95, weight_decay=0.1, eps=1e-7, nesterov=True, ns_steps=5)
    op(W, G, M, lr=0.02, weight_decay=0.1)
    assert op.status() == B.MUON_OK
    for i in range(len(shapes)):
        for e, (w0, g0, m0) in enumerate(zip(*pre[i])):
            W1, M1, Or = O.muon_step(w0, g0, m0, hp)
            assert_m1_elementwise(matrices(M[i])[e], M1, m0, g0, dtype)
            scale = hp.lr * O.shape_scale(*w0.shape)
            err = np.linalg.norm(matrices(W[i])[e] - W1)
            budget = ITERATION * scale * np.linalg.norm(Or)
            assert err <= budget + torch.finfo(dtype).eps / 2 * np.linalg.norm(W1), (shapes[i], e)
    op.close()


@pytest.mark.parametrize("shapes", [[(64, 300), (512, 256), (131, 77)], [(512, 512)], [(300, 256)] * 3, [(20, 30)]], ids=str)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_launches_are_counted(shapes, dtype):
    op = MuonStep(shapes, dtype=dtype, mode="half")
    W, G, M = ([random(s, dtype, i, "plain") for i, s in enumerate(shapes)] for _ in range(3))
    for k in (0, 1, 4):
        B.muon_profile_begin(op.handle, 1)
        op(W, G, M, ns_steps=k)
        assert sum(n for _, n in B.muon_profile_end(op.handle).values()) == op.launches_per_step(k)
    op.close()


def test_half_is_nearer_than_fast():
    """The reason for the mode: on the same bf16 inputs the error is at least four times smaller (an eighth expected)."""
    shape = (512, 768)
    x = [random(shape, torch.bfloat16, 3, "plain")]
    err = {}
    for mode in ("fast", "half"):
        op = MuonStep([shape], dtype=torch.float32 if mode == "fast" else torch.bfloat16, mode=mode)
        o = [torch.empty(shape, dtype=torch.float32, device="cuda")]
        op.orthogonalize([x[0].float()], o)
        err[mode] = rel_fro(to_f64(o[0]), iterate(to_f64(x[0]), [QUINTIC] * 5))
        op.close()
    assert err["half"] * 4 <= err["fast"]


@pytest.mark.parametrize("shapes", [[(331, 503), (7, 300, 300), (64, 128)], [(768, 512), (2, 512, 1024)], [(130, 2000)]], ids=str)
def test_schedules_agree(shapes):
    """One launch for every iteration, or one per stage: the same tiles and roundings, so the same bits."""
    abc = [QUINTIC] * 2 + [SETTLE, (1.5, -0.5, 0.0)]
    X = [random(s, torch.bfloat16, i) for i, s in enumerate(shapes)]
    outs = []
    for schedule in ("staged", "fused", "split", "auto"):
        op = MuonStep(shapes, mode="half", schedule=schedule)
        Os = [torch.empty_like(x) for x in X]
        for _ in range(2):
            op.orthogonalize(X, Os, abc=abc)
        check(shapes, X, Os, abc, op, schedule)
        outs.append(Os)
        op.close()
    for Os in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(Os, outs[0]))


def test_captured_and_on_another_stream():
    shapes = [(12, 64, 96), (300, 256)]
    op = MuonStep(shapes, mode="half")
    X = [random(s, torch.bfloat16, i) for i, s in enumerate(shapes)]
    eager = [torch.empty_like(x) for x in X]
    op.orthogonalize(X, eager)
    out = [torch.empty_like(x) for x in X]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    op.orthogonalize(X, out, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, eager))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        op.orthogonalize(X, out)
    for o in out:
        o.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, eager))
    op.close()


def test_refusals():
    shape = (64, 96)
    x = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
    fast, half = MuonStep([shape]), MuonStep([shape], mode="half")
    with pytest.raises(ValueError):
        fast.orthogonalize([x], [x], abc=[QUINTIC] * 5)
    with pytest.raises(ValueError):
        half.orthogonalize([x], [x], abc=[QUINTIC] * 5, ns_steps=4)
    with pytest.raises(ValueError):
        half.orthogonalize([torch.zeros(128, 192, dtype=torch.bfloat16, device="cuda")[::2, ::2]], [x])
    with pytest.raises(ValueError):
        half.orthogonalize([x.double()], [x])
    with pytest.raises(ValueError):
        half.orthogonalize([x, x], [x, x])
    with pytest.raises(B.MuonError) as e:
        half.orthogonalize([x], [x[:1].expand(64, 96)])         # rows of the output overlap
    assert e.value.code == B.MUON_ERR_INVALID_ARG
    with pytest.raises(B.MuonError):
        half.orthogonalize([x], [x], eps=-1.0)
    with pytest.raises(B.MuonError):
        half.orthogonalize([x], [x], ns_steps=65)
    with pytest.raises(B.MuonError) as e:
        half.set_schedule("fused")
    assert e.value.code == B.MUON_ERR_UNSUPPORTED
    v = B.views([(x.data_ptr(), 1, 0, 96, 1, B.MUON_BF16)])
    with pytest.raises(B.MuonError) as e:
        B.muon_orthogonalize_views(fast.handle, v, v, 1, B.make_hparams(), 0)
    assert e.value.code == B.MUON_ERR_UNSUPPORTED
    with pytest.raises(B.MuonError) as e:
        B.muon_set_coefficients(half.handle, [(float("nan"), 0, 0)])
    assert e.value.code == B.MUON_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        MuonStep([(1, 2, 3, 4)])
    half.orthogonalize([x[:1].expand(64, 96)], [x.clone()])      # an input may repeat its rows
    fast.close()
    half.close()
