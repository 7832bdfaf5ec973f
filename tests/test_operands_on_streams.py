"""Operands of a forward that runs on a given stream belong to the caller's stream.  The layer may be the last to hold
them: their memory is not given out again before the given stream's work is done (as tests/test_attention_on_streams.py
holds the saved state to it)."""

import contextlib

import pytest
import torch

from orthogonal_reparameterized_cnp_amd import binding as B
from orthogonal_reparameterized_cnp_amd import layer as L


@pytest.fixture
def kept(monkeypatch):
    """The classes on the CPU: the caller's stream has the handle 1, a given stream is its handle, no launch is made, and
    what is recorded comes as (handle, data pointer)."""
    now, kept = [1], set()

    @contextlib.contextmanager
    def on(device, stream):
        now[0] = stream or 1
        yield
        now[0] = 1

    monkeypatch.setattr(L, "_on", on)
    monkeypatch.setattr(L, "_made_on", lambda device: now[0])
    monkeypatch.setattr(L, "_check_device", lambda device, **tensors: None)
    monkeypatch.setattr(B, "_current_stream", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[0])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.add((s, t.data_ptr())))
    for name in ("poetx_attn_fwd", "poetx_attn_bwd", "poetx_logp_fwd", "poetx_logp_bwd", "poetx_norm_fwd", "poetx_norm_bwd"):
        monkeypatch.setattr(B, name, lambda *a, **k: None)
    return kept


@pytest.mark.parametrize("packed", [False, True])
def test_attention(kept, packed):
    at = L.PoetxAttention(2, 1, 8, "f32", device="cpu")
    Q, K, V, O = torch.randn(6, 16), torch.randn(6, 8), torch.randn(6, 8), torch.randn(6, 16)
    cu = torch.tensor([0, 2, 6], dtype=torch.int32) if packed else None
    at.forward(Q, K, V, cu)
    assert not kept
    at.forward(Q, K, V, cu, O=O, stream=2)
    given = [Q, K, V, O, *([cu] if packed else [])]
    assert kept == {(2, t.data_ptr()) for t in given}
    kept.clear()
    at.backward(Q, stream=2)  # nothing that the recordings of the forward do not cover
    at.forward(Q, K, V, cu, stream=2)
    assert kept == {(2, t.data_ptr()) for t in given if t is not O}


def test_log_probabilities(kept):
    p = L.PoetxLogProb(9, "f32", device="cpu")
    X, t = torch.randn(4, 9), torch.zeros(4, dtype=torch.int32)
    p.forward(X, t)
    assert not kept
    p.forward(X, t, stream=2)
    assert kept == {(2, X.data_ptr()), (2, t.data_ptr())}
    kept.clear()
    p.forward(X, stream=2)
    assert kept == {(2, X.data_ptr())}


@pytest.mark.parametrize("res", [False, True])
def test_norm(kept, res):
    norm = L.PoetxNorm(16, "layer", "f32", device="cpu")
    X, R, S = torch.randn(4, 16), torch.randn(4, 16), torch.randn(4, 16)
    norm.forward(X, R if res else None)
    assert not kept
    norm.forward(X, R if res else None, S=S if res else None, stream=2)
    assert kept == {(2, (S if res else X).data_ptr())}  # what the norm keeps


needs_gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def _late(stream):
    """Work of some milliseconds in front of what `stream` gets next, which starts after what is queued here."""
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)


@pytest.mark.parametrize("act", [pytest.param(c, marks=needs_gpu) for c in ("f32", "bf16")])
def test_operands_dropped_while_their_stream_waits(act):
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[act]
    at, lp, norm = L.PoetxAttention(4, 2, 64, act), L.PoetxLogProb(1000, act), L.PoetxNorm(256, "rms", act)
    new = lambda *s: torch.randn(*s, device="cuda").to(dt)
    Q, K, V, dO, X = new(500, 256), new(500, 128), new(500, 128), new(500, 256), new(300, 1000)
    cu = torch.tensor([0, 100, 500], dtype=torch.int32, device="cuda")
    t, a = torch.arange(300, dtype=torch.int32, device="cuda"), torch.randn(300, device="cuda")

    def step(stream=None):
        copies = [x.clone() for x in (Q, K, V, cu, X, t)]
        if stream is not None:
            _late(stream)
        out = [at.forward(*copies[:4], stream=stream), *lp.forward(*copies[4:], stream=stream)[:3],
               norm.forward(copies[0], stream=stream)]
        return out + [*at.backward(dO, stream=stream), lp.backward(a, a, stream=stream), norm.backward(dO, stream=stream)[0]]

    want = step()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        got = step(s)  # its copies of the operands are held by the layers alone, until the next line
        at.saved, lp.saved, norm.S = None, None, None
        junk = [torch.full_like(x, 7) for x in (Q, K, V, cu, X, t) for _ in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and len(junk) == 12
