"""GPU parity of the rotary positions (poetx_rope, layer.PoetxRope) against the fp64 oracle.

Bounds, with u = 2^-24 and h half a step of the output type (0 extra for fp32, 2^-8 for bf16).  The angle is formed in
fp64 and reduced to at most half a turn, which rounds to fp32 within 2^-26 of a turn: pi 2^-25 < 2 u radians.  The sine
and cosine are off by at most 2 more units in the last place (4 u), and the amplitude's product by u: 7 u; the two
products and their sum by 2 u more each: amplitude (|x| + |y|) 11 u + h |Y|.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from orthogonal_reparameterized_cnp_amd.layer import PoetxRope

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

U = 2.0**-24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 0.0, "bf16": 2.0**-8}


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(T, cols, act, seed, pitch=None, offset=0):
    """[T, cols] of the given pitch, `offset` elements into a buffer whose other cells hold a mark."""
    g = torch.Generator().manual_seed(seed)
    pitch = pitch or cols
    buf = torch.full((offset + T * pitch + 8,), 77.0, dtype=DT[act], device="cuda")
    v = buf[offset:offset + T * pitch].view(T, pitch)[:, :cols]
    v.copy_(torch.randn(T, cols, generator=g).to(DT[act]))
    return v


def check(rope, X, Y, pos, inverse=False):
    x, p = f64(X), f64(pos) if pos is not None else np.arange(len(X), dtype=float)
    f = f64(rope.freqs)
    ref = O.rope(x, p, f, rope.head_dim, rope.layout, rope.amplitude, inverse)
    # |x| + |y| of every pair, at both of its elements; what is copied is exact
    half = len(f)
    mag = np.zeros_like(x).reshape(len(x), -1, rope.head_dim)
    a = np.abs(x).reshape(mag.shape)
    first = np.arange(half) if rope.layout == "half" else 2 * np.arange(half)
    second = first + (half if rope.layout == "half" else 1)
    mag[..., first] = mag[..., second] = a[..., first] + a[..., second]
    tol = abs(rope.amplitude) * 11 * U * mag.reshape(x.shape)
    tol = np.where(tol > 0, tol * (1 + HALF[rope.act]) + HALF[rope.act] * np.abs(ref) + 1e-38, 0.0)
    d = np.abs(f64(Y) - ref)
    print(f"  worst |d| / bound {np.max(d[tol > 0] / tol[tol > 0], initial=0):.3f}", flush=True)
    assert (d <= tol).all(), d.max()


@pytest.mark.parametrize("layout", ["half", "pairs"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T,heads,hd,rot", [(1, (32, 8), 128, 128), (7, (3,), 2, 2), (33, (9, 3), 75, 34), (5, (2, 1, 1), 64, 16),
                                            (2, (2,), 1024, 1024), (3, (1,), 1023, 2), (2500, (4, 2), 64, 64),
                                            (9000, (1,), 8, 6), (130, (8, 8), 80, 80), (1100, (2,), 96, 48)])
def test_rotation(T, heads, hd, rot, act, layout):
    rope = PoetxRope(hd, rot, layout, act, base=500000.0)
    g = torch.Generator().manual_seed(T)
    pos = torch.randint(0, 200000, (T,), generator=g, dtype=torch.int32).cuda()
    Xs = [rows(T, n * hd, act, i) for i, n in enumerate(heads)]
    Ys = rope.forward(Xs, pos)
    for x, y in zip(Xs, Ys):
        check(rope, x, y, pos)
    for x, y in zip(Xs, rope.backward(Xs, pos)):
        check(rope, x, y, pos, inverse=True)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_far_and_negative_positions(act):
    """Angles of up to 2^31 radians keep their digits."""
    rope = PoetxRope(64, act=act)
    pos = torch.tensor([2**31 - 1, -2**31, -1, 0, 1 << 24, (1 << 30) + 1], dtype=torch.int32, device="cuda")
    X = rows(6, 128, act, 3)
    # the oracle's own angle, pos f in fp64, is off by 2^31 2^-53 radians: 4 u, added to the bound's 7
    x, ref = f64(X), O.rope(f64(X), f64(pos), f64(rope.freqs), 64)
    Y = f64(rope.forward([X], pos)[0])
    mag = np.abs(x).max()
    assert np.abs(Y - ref).max() <= 2 * 15 * U * mag + HALF[act] * np.abs(ref).max()


def test_scaled_frequencies_and_amplitude():
    for scaling in ("linear", "base", "bands", "ramp"):
        rope = PoetxRope(128, 96, "half", "f32", scaling=scaling, factor=8.0, original=4096.0, low=1.0, high=32.0)
        pos = torch.arange(50, dtype=torch.int32, device="cuda") * 600
        X = rows(50, 256, "f32", 4)
        check(rope, X, rope.forward([X], pos)[0], pos)
        check(rope, X, rope.backward([X], pos)[0], pos, inverse=True)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("hd,rot", [(64, 64), (75, 34)])
def test_pitches_offsets_and_in_place(act, hd, rot):
    """Columns of one buffer at odd pitches and element offsets; the cells around them stay as they were."""
    rope = PoetxRope(hd, rot, "half", act)
    T, pitch = 37, 5 * hd + 3
    buf = torch.full((T * pitch + 8,), 77.0, dtype=DT[act], device="cuda")
    v = buf[1:1 + T * pitch].view(T, pitch)
    Q, K = v[:, :3 * hd], v[:, 3 * hd:5 * hd]
    Q.copy_(rows(T, 3 * hd, act, 1))
    K.copy_(rows(T, 2 * hd, act, 2))
    q0, k0 = Q.clone(), K.clone()
    pos = torch.arange(100, 100 + T, dtype=torch.int32, device="cuda")
    out = rows(T, 3 * hd, act, 5, pitch=3 * hd + 7, offset=3)
    rope.forward([Q, K], pos, [out, K])
    check(rope, q0, out, pos)
    check(rope, k0, K, pos)
    assert torch.equal(Q, q0) and (v[:, 5 * hd:] == 77).all() and (buf[0] == 77) and (buf[1 + T * pitch:] == 77).all()
    fresh = rope.forward([q0])[0]  # positions 0, 1, ...
    check(rope, q0, fresh, None)
    assert rope.forward([q0[:0]])[0].shape == (0, 3 * hd)


def test_backward_is_the_transpose():
    rope = PoetxRope(32, 20, "pairs", "f32", scaling="ramp", factor=4.0, original=64.0, low=1.0, high=8.0)
    pos = torch.arange(64, dtype=torch.int32, device="cuda")
    X, G = rows(64, 64, "f32", 1), rows(64, 64, "f32", 2)
    a, b = f64(rope.forward([X], pos)[0]) * f64(G), f64(X) * f64(rope.backward([G], pos)[0])
    assert abs(a.sum() - b.sum()) <= 11 * U * 2 * rope.amplitude * (np.abs(f64(X)).max() * np.abs(f64(G)).max()) * X.numel()


def test_graph_and_streams():
    rope = PoetxRope(64)
    pos = torch.arange(300, dtype=torch.int32, device="cuda")
    X = rows(300, 256, "bf16", 1)
    ref = rope.forward([X], pos)[0]
    out = torch.empty_like(X)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    rope.forward([X], pos, [out], stream=s)
    s.synchronize()
    assert torch.equal(out, ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rope.forward([X], pos, [out])
    for i in range(3):
        X.copy_(rows(300, 256, "bf16", 10 + i))
        ref = rope.forward([X], pos)[0]
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)
