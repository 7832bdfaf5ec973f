"""What the attention, the log probabilities and the rotary positions allocate or keep on one stream and use on another
stays theirs until the work there is done (as tests/test_saved_on_streams.py holds the norm to)."""

import contextlib

import pytest
import torch

from orthogonal_reparameterized_cnp_amd import binding as B
from orthogonal_reparameterized_cnp_amd import layer as L


@pytest.fixture
def streams(monkeypatch):
    """The classes on the CPU: no launch is made, `now[0]` is the current stream's handle, and `kept` collects what is
    recorded on it as (handle, data pointer)."""
    now, kept = [1], set()
    monkeypatch.setattr(L, "_on", lambda device, stream: contextlib.nullcontext())
    monkeypatch.setattr(L, "_check_device", lambda device, **tensors: None)
    monkeypatch.setattr(B, "_current_stream", lambda: now[0])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: now[0])
    monkeypatch.setattr(torch.Tensor, "record_stream", lambda t, s: kept.add((s, t.data_ptr())))
    for name in ("poetx_attn_fwd", "poetx_attn_bwd", "poetx_logp_fwd", "poetx_logp_bwd", "poetx_rope"):
        monkeypatch.setattr(B, name, lambda *a, **k: None)
    return now, kept


@pytest.mark.parametrize("packed", [False, True])
def test_attention_backward_on_another_stream(streams, packed):
    now, kept = streams
    at = L.PoetxAttention(2, 1, 8, "f32", device="cpu")
    Q, K, V = torch.randn(6, 16), torch.randn(6, 8), torch.randn(6, 8)
    cu = torch.tensor([0, 2, 6], dtype=torch.int32) if packed else None
    O = at.forward(Q, K, V, cu)
    at.backward(Q)
    assert not kept
    now[0] = 2
    at.backward(Q)
    assert kept == {(2, t.data_ptr()) for t in (Q, K, V, O, at.saved[4], *([cu] if packed else []))}


def test_log_probability_backward_on_another_stream(streams):
    now, kept = streams
    p = L.PoetxLogProb(9, "f32", device="cpu")
    X, t = torch.randn(4, 9), torch.zeros(4, dtype=torch.int32)
    out = p.forward(X, t)
    p.backward(torch.zeros(4))
    assert not kept
    now[0] = 2
    p.backward(torch.zeros(4))
    assert kept == {(2, x.data_ptr()) for x in (X, t, out.lse, out.entropy)}


def test_rope_frequencies_on_another_stream(streams):
    now, kept = streams
    r = L.PoetxRope(8, act="f32", device="cpu")
    r._made_on = 1  # as on a GPU whose current stream is 1
    r.forward([torch.randn(3, 16)])
    assert not kept
    now[0] = 2
    r.backward([torch.randn(3, 16)])
    assert kept == {(2, r.freqs.data_ptr())}


needs_gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def _late(stream):
    """Work of some milliseconds in front of what `stream` gets next, which starts after what is queued here."""
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)


@pytest.mark.parametrize("act", [pytest.param(c, marks=needs_gpu) for c in ("f32", "bf16")])
def test_next_forward_while_the_backward_waits(act):
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[act]
    at, lp = L.PoetxAttention(4, 2, 64, act), L.PoetxLogProb(1000, act)
    new = lambda *s: torch.randn(*s, device="cuda").to(dt)
    Q, K, V, dO, X = new(500, 256), new(500, 128), new(500, 128), new(500, 256), new(300, 1000)
    cu = torch.tensor([0, 100, 500], dtype=torch.int32, device="cuda")
    t, a = torch.arange(300, dtype=torch.int32, device="cuda"), torch.randn(300, device="cuda")

    def forwards():
        at.forward(Q.clone(), K.clone(), V.clone(), cu.clone())
        lp.forward(X.clone(), t.clone())

    forwards()
    want = [*at.backward(dO), lp.backward(a, a)]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        forwards()
        _late(s)
        got = [*at.backward(dO, stream=s), lp.backward(a, a, stream=s)]
        forwards()  # drops the saved state that the backward is still to read
        junk = [torch.full_like(x, 7.0) for x in (Q, K, V, X) for _ in range(2)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want)) and len(junk) == 8
