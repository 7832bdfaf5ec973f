"""What the norm and the orthogonalised updates allocate on one stream and use on another stays theirs until the work
there is done.  Dropped earlier, torch's allocator would hand its memory to the first stream's next allocation while
the second stream still reads it."""

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
    for name in ("poetx_norm_fwd", "poetx_norm_bwd", "poetx_muon_step_batch", "poetx_orthogonalize"):
        monkeypatch.setattr(B, name, lambda *a, **k: None)
    return now, kept


@pytest.mark.parametrize("res", [False, True])
def test_norm_backward_on_another_stream(streams, res):
    now, kept = streams
    norm = L.PoetxNorm(16, "layer", "f32", device="cpu")
    X = torch.randn(4, 16)
    norm.forward(X, X.clone() if res else None)
    S, stats = norm.S, norm.stats
    norm.backward(X)
    assert not kept
    now[0] = 2
    norm.backward(X)
    assert kept == {(2, S.data_ptr()), (2, stats.data_ptr())}


def test_workspaces_on_another_stream(streams):
    now, kept = streams
    op = L.PoetxOrthogonalizer(10, 20, device="cpu")
    opt = L.PoetxMuon([L.PoetxLinear(64, 48, 16, device="cpu")])
    for o in (op, opt):
        o._made_on = 1  # as on a GPU whose current stream is 1
    G, dq = torch.zeros(10, 20), [(opt.layers[0].q_R, opt.layers[0].q_P)]
    op(G)
    opt.step(dq)
    assert not kept
    now[0] = 2
    op(G)
    assert kept == {(2, op.ws.data_ptr())}
    opt.step(dq)
    assert {(2, t.data_ptr()) for t in [opt.ws, *opt.m]} <= kept


needs_gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


def _late(stream):
    """Work of some milliseconds in front of what `stream` gets next, which starts after what is queued here."""
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        torch.cuda._sleep(20_000_000)


@pytest.mark.parametrize("case", [pytest.param(c, marks=needs_gpu) for c in ("layer", "rms")])
def test_next_forward_while_the_backward_waits(case):
    T, d = 400, 512
    norm = L.PoetxNorm(d, case, "f32")
    X, other, R, dY = (torch.randn(T, d, device="cuda") for _ in range(4))
    norm.forward(X, R)
    want = norm.backward(dY)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        norm.forward(X, R)
        _late(s)
        got = norm.backward(dY, stream=s)
        norm.forward(other, R)  # drops the saved state that the backward is still to read
        norm.forward(other, R)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert (a is None and b is None) or torch.equal(a, b)


@pytest.mark.parametrize("case", [pytest.param(c, marks=needs_gpu) for c in ("f32", "bf16")])
def test_orthogonalizer_dropped_while_its_call_waits(case):
    dt = {"f32": torch.float32, "bf16": torch.bfloat16}[case]
    G = torch.randn(200, 300, device="cuda").to(dt)
    want = L.PoetxOrthogonalizer(200, 300, case)(G)
    need = L.PoetxOrthogonalizer(200, 300, case).ws.numel()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(3):
        _late(s)
        got = L.PoetxOrthogonalizer(200, 300, case)(G, stream=s)
        junk = [torch.full((need,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]
        torch.cuda.synchronize()
        assert torch.equal(got, want) and len(junk) == 3
