"""Argument handling of MuonStep without a device: what reaches the library, and what is refused before it.

The C entry points are replaced by recorders, so nothing here runs a kernel.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from muon_newton_schulz_07_b200 import binding as B
from muon_newton_schulz_07_b200.optimizer import QUINTIC, MuonStep

TRIPLE = (3.0, -3.25, 1.125)


def step(mode, n=3):
    op = object.__new__(MuonStep)
    op.mode, op.handle, op.device, op._n, op._streams = mode, None, torch.device("cpu"), n, {0}
    return op


@pytest.fixture
def coefficients(monkeypatch):
    sent = []
    monkeypatch.setattr(B, "muon_set_coefficients",
                        lambda handle, abc: sent.append([tuple(float(x) for x in t) for t in abc]))
    return sent


@pytest.mark.parametrize("mode", ["fast", "half", "fp32_ref"])
@pytest.mark.parametrize("kind", [tuple, list, np.array, torch.tensor,
                                  lambda t: [np.float32(x) for x in t], lambda t: [torch.tensor(x) for x in t]],
                         ids=["tuple", "list", "array", "tensor", "scalars", "scalar tensors"])
def test_one_triple_in_any_form(coefficients, mode, kind):
    abc, k = step(mode)._coefficients(kind(TRIPLE), None)
    hp = B.make_hparams(abc=abc, ns_steps=k)
    assert (hp.a, hp.b, hp.c) == TRIPLE and hp.ns_steps == 5
    assert coefficients == ([[]] if mode == "half" else [])
    assert step(mode)._coefficients(kind(TRIPLE), 7)[1] == 7


@pytest.mark.parametrize("kind", [list, np.array, torch.tensor, lambda t: [torch.tensor(x) for x in t]],
                         ids=["list", "array", "tensor", "tensors"])
@pytest.mark.parametrize("k", [1, 2, 3, 5])
def test_a_triple_for_each_iteration_in_any_form(coefficients, kind, k):
    abc = [TRIPLE if t % 2 else (1.5, -0.5, 0.0) for t in range(k)]
    assert step("half")._coefficients(kind(abc), None) == (QUINTIC, k)
    assert coefficients == [abc]
    with pytest.raises(ValueError):
        step("half")._coefficients(kind(abc), k + 1)
    with pytest.raises(ValueError):
        step("fast")._coefficients(kind(abc), None)


def test_coefficients_that_are_neither(coefficients):
    for abc in ((1.0, 2.0), (1.0, 2.0, 3.0, 4.0), [(1.0, 2.0)] * 3, [TRIPLE, 1.0, 2.0]):
        with pytest.raises(ValueError):
            step("half")._coefficients(abc, None)
    assert coefficients == []


def test_a_buffer_that_does_not_hold_the_norms_is_refused(monkeypatch):
    """The copy goes to its address: one that is too short, of another type or strided would be written past its end."""
    sent = []
    monkeypatch.setattr(B, "muon_get_norms", lambda handle, dst, stream: sent.append(dst))
    monkeypatch.setattr("muon_newton_schulz_07_b200.optimizer._stream", lambda device, stream: 0)
    op = step("half", n=3)
    for bad in (torch.zeros(2), torch.zeros(3, dtype=torch.float64), torch.zeros(3, dtype=torch.bfloat16),
                torch.zeros(6)[::2], torch.zeros(3, device="meta")):
        with pytest.raises(ValueError):
            op.norms(bad)
    assert sent == []
    for good in (torch.zeros(3), torch.zeros(1, 3), torch.zeros(7)[1:]):
        assert op.norms(good) is good
    assert len(sent) == 3


def test_momentum_refuses_before_it_updates_anything(monkeypatch):
    """A call that is refused leaves the state as it was: the buffer for the norms is looked at first."""
    monkeypatch.setattr(B, "muon_momentum_state", lambda *a: pytest.fail("called"))
    monkeypatch.setattr("muon_newton_schulz_07_b200.optimizer._stream", lambda device, stream: 0)
    op = step("half", n=1)
    op._entries, op.shapes, op.dtype = [(1, 4, 4, (4, 4))], [(4, 4)], torch.float32
    state = type("S", (), {"shapes": [(4, 4)], "device": op.device, "_fmt": 0, "_states": lambda self: b""})()
    g = [torch.zeros(4, 4)]
    with pytest.raises(ValueError):
        op.momentum(g, state, [torch.zeros(4, 4)], norms=torch.zeros(0))
