"""The gradient written over the logits ends the forward's saved state."""

import contextlib

import pytest
import torch

from orthogonal_reparameterized_cnp_amd import binding as B
from orthogonal_reparameterized_cnp_amd import layer as L


@pytest.fixture
def on_cpu(monkeypatch):
    monkeypatch.setattr(L, "_on", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(L, "_check_device", lambda device, **tensors: None)
    monkeypatch.setattr(B, "_current_stream", lambda: 1)
    for name in ("poetx_logp_fwd", "poetx_logp_bwd"):
        monkeypatch.setattr(B, name, lambda *a, **k: None)


def test_second_backward_after_one_in_place(on_cpu):
    p = L.PoetxLogProb(9, "f32", device="cpu")
    X, t, a = torch.randn(4, 9), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    p.forward(X, t)
    p.backward(a, dX=torch.empty(4, 9))
    p.backward(a)  # the logits are still there
    p.backward(a, dX=X)
    with pytest.raises(ValueError, match="before a forward"):
        p.backward(a)  # here X holds the gradient
    p.forward(X, t)
    p.backward(a, dX=X.view(4, 9))
    assert p.saved is None


def test_a_refused_call_keeps_the_state(on_cpu, monkeypatch):
    p = L.PoetxLogProb(9, "f32", device="cpu")
    X, t, a = torch.randn(4, 9), torch.zeros(4, dtype=torch.int32), torch.zeros(4)
    p.forward(X, t)

    def refuse(*args):
        raise B.PoetxError(B.POETX_E_SHAPE, "no")

    with monkeypatch.context() as m:
        m.setattr(B, "poetx_logp_bwd", refuse)
        with pytest.raises(B.PoetxError):
            p.backward(a, dX=X)
    p.backward(a)
