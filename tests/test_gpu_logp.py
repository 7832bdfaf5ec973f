"""GPU parity of the log probabilities (poetx_logp_fwd / poetx_logp_bwd, layer.PoetxLogProb) against the fp64 oracle.

Bounds, with u = 2^-24, h half a step of the output type and y = scale (x - m).  An element's y is off by 3 u |y| (the
difference, scale log2 e, the product) and its exponential by that and 2 u.  A thread adds at most N = V / 256 + 8 terms
and is joined in at most 20 steps, each of which rescales the sums: n = N + 80 roundings.
  * s within s (n u + 3 u E|y|), so lse within that and 4 u (|lse| + |scale m|); logp adds 2 u |scale x|.
  * H = ln 2 (log2 s - w / s): w within n u E|y| + 3 u E y^2 + 3 u E|y| of s, the quotient by s's part times E|y|:
    u ((n + 4) (1 + 2 E|y|) + 3 E y^2 + 3 E|y| (1 + E|y|) + 4 H).
  * backward, at the saved lse and H: log p off by e = u (2 |scale x| + 2 |lse| + 2 |log p|), p by e + 3 u of itself:
    scale (|dlogp| p (e + 5 u) + |dH| p ((|log p + H|) (e + 6 u) + e + 2 u |log p|)) + 4 u |dX| + h |dX|.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from orthogonal_reparameterized_cnp_amd.layer import PoetxLogProb

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

U = 2.0**-24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 0.0, "bf16": 2.0**-8}
MARK = 77.0


def f64(t):
    return t.detach().double().cpu().numpy()


def logits(T, V, act, seed, pitch=None, offset=0, scale=2.0):
    g = torch.Generator().manual_seed(seed)
    pitch = pitch or V
    buf = torch.full((offset + T * pitch + 8,), MARK, dtype=DT[act], device="cuda")
    v = buf[offset:offset + T * pitch].view(T, pitch)[:, :V]
    v.copy_((scale * torch.randn(T, V, generator=g) + torch.randn(T, 1, generator=g)).to(DT[act]))
    return v


def targets(T, V, seed):
    g = torch.Generator().manual_seed(seed)
    t = torch.randint(0, V, (T,), generator=g, dtype=torch.int32)
    t[T // 3::5] = -1
    t[T // 2::7] = V
    return t.cuda()


def within(name, got, ref, tol):
    inf = np.isinf(ref)
    assert (got[inf] == ref[inf]).all(), name
    d = np.abs(got[~inf] - ref[~inf])
    tol = np.broadcast_to(tol, ref.shape)[~inf]
    print(f"  {name}: worst |d| / bound {np.max(d / np.maximum(tol, 1e-300), initial=0.0):.3f}", flush=True)
    assert np.isfinite(got[~inf]).all() and (d <= tol).all(), f"{name}: max |d| {d.max():.3e}"


def check_forward(op, X, t, out):
    x, sc, V = f64(X), float(np.float32(op.scale)), X.shape[1]
    tn = t.cpu().numpy()
    lp, lse, H, ids, tlp = O.token_logprobs(x, tn, sc, op.top)
    m = x.max(1, initial=-np.inf)
    m0 = np.where(np.isinf(m), 0.0, m)[:, None]
    y = np.where(np.isinf(x), 0.0, sc * (x - m0))
    with np.errstate(invalid="ignore"):
        p = np.where(np.isneginf(x), 0.0, np.exp(np.where(np.isneginf(x), 0.0, sc * x) - np.where(np.isinf(lse), 0.0, lse)[:, None]))
    Ey, Ey2 = (p * abs(y)).sum(1), (p * y * y).sum(1)
    n = V / 256 + 88
    l0 = np.where(np.isinf(lse), 0.0, lse)
    tl = U * (n + 3 * Ey + 4 * (abs(l0) + abs(sc * m0[:, 0])) + 4)
    within("lse", f64(out.lse), lse, tl)
    given = (tn >= 0) & (tn < V)
    at = np.where(given, x[np.arange(len(x)), np.where(given, tn, 0)], 0.0)
    at = np.where(np.isinf(at), 0.0, at)
    within("logp", f64(out.logp), lp, np.where(given, tl + U * (2 * abs(sc * at) + 2 * abs(np.where(np.isinf(lp), 0, lp))), 0))
    within("entropy", f64(out.entropy), H, U * ((n + 4) * (1 + 2 * Ey) + 3 * Ey2 + 3 * Ey * (1 + Ey) + 4 * H))
    if op.top:
        assert (out.top_ids.cpu().numpy() == ids).all()
        v = np.take_along_axis(np.where(np.isinf(x), 0.0, x), ids, 1)
        within("top", f64(out.top_logp), tlp, tl[:, None] + U * (2 * abs(sc * v) + 2 * abs(np.where(np.isinf(tlp), 0, tlp))))


def check_backward(op, X, t, saved, dlogp, dent, dX):
    x, sc = f64(X), float(np.float32(op.scale))
    tn = t.cpu().numpy()
    lse, H = f64(saved[2]), f64(saved[3])
    a = f64(dlogp) if dlogp is not None else np.zeros(len(x))
    b = f64(dent) if dent is not None else np.zeros(len(x))
    ref = O.token_logprobs_backward(x, tn, lse, H, a, b, sc)
    off = np.isneginf(x) | np.isneginf(lse)[:, None]
    l0 = np.where(np.isneginf(lse), 0.0, lse)[:, None]
    lx = np.where(off, 0.0, np.where(off, 0.0, x) * sc - l0)
    p = np.where(off, 0.0, np.exp(lx))
    e = U * (2 * abs(np.where(off, 0, sc * x)) + 2 * abs(l0) + 2 * abs(lx))
    tol = abs(a)[:, None] * p * (e + 5 * U) + abs(b)[:, None] * p * (abs(lx + H[:, None]) * (e + 6 * U) + e + 2 * U * abs(lx))
    h = HALF[op.act]
    within("dX", f64(dX), ref, (sc * tol + 4 * U * abs(ref)) * (1 + h) + h * abs(ref) + 1e-38)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("top", [0, 1, 5, 64])
@pytest.mark.parametrize("T,V", [(1, 64), (3, 65), (1, 131072), (2, 50001), (7, 2049), (70, 1000), (1030, 257), (1100, 2500),
                                 (40, 32000), (5, 8191), (1, 1 << 20)])
def test_forward_backward(T, V, act, top):
    print(f"logp T={T} V={V} {act} top={top}", flush=True)
    op = PoetxLogProb(V, act, top, scale=0.8)
    X, t = logits(T, V, act, T + V), targets(T, V, 1)
    out = op.forward(X, t)
    check_forward(op, X, t, out)
    if top not in (0, 5):
        return
    g = torch.Generator().manual_seed(2)
    a, b = torch.randn(T, generator=g).cuda(), torch.randn(T, generator=g).cuda()
    for da, db in ((a, b), (a, None), (None, b)):
        check_backward(op, X, t, op.saved, da, db, op.backward(da, db))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 7])
def test_small_vocabularies(act, V):
    op = PoetxLogProb(V, act, top=min(V, 3))
    X = logits(9, V, act, 3)
    t = (torch.arange(9, dtype=torch.int32) % V).cuda()
    check_forward(op, X, t, op.forward(X, t))
    a = torch.ones(9, device="cuda")
    check_backward(op, X, t, op.saved, a, a, op.backward(a, a))


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 20000])
def test_masked_and_equal_logits(act, V):
    """-infinity and the type's lowest value in masked places, whole rows of either, and ties, which go to the lowest
    index in every order of the columns."""
    low = torch.finfo(DT[act]).min
    op = PoetxLogProb(V, act, top=20)
    X = logits(8, V, act, 5)
    X[0, V // 4:] = float("-inf")
    X[1, ::2] = low
    X[2] = float("-inf")
    X[3] = low
    X[4] = 1.5
    X[5] = torch.round(X[5])  # few values, many of each
    X[6, 7:] = float("-inf")
    X[7, :-1] = float("-inf")
    t = torch.tensor([V - 1, 1, 5, 5, V - 1, 3, 0, V - 1], dtype=torch.int32, device="cuda")
    out = op.forward(X, t)
    check_forward(op, X, t, out)
    assert out.top_ids[4].tolist() == list(range(20)) and out.top_ids[2].tolist() == list(range(20))
    assert float(out.entropy[2]) == 0 and float(out.logp[7]) == 0
    a, b = torch.full((8,), 0.5, device="cuda"), torch.full((8,), -0.25, device="cuda")
    dX = op.backward(a, b)
    check_backward(op, X, t, op.saved, a, b, dX)
    assert not dX[2].any() and torch.isfinite(dX).all()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_nan_and_infinity_stay_in_their_rows(act):
    V = 5000
    op = PoetxLogProb(V, act, top=4)
    X = logits(6, V, act, 6)
    t = torch.zeros(6, dtype=torch.int32, device="cuda")
    ref = op.forward(X, t)
    dref = op.backward(torch.ones(6, device="cuda"))
    Y = X.clone()
    Y[1, 2500], Y[4, 17], Y[4, 4000] = float("nan"), float("inf"), float("nan")
    out = op.forward(Y, t)
    dX = op.backward(torch.ones(6, device="cuda"))
    keep = [0, 2, 3, 5]
    for a, b in zip([*out, dX], [*ref, dref]):
        assert torch.equal(a[keep], b[keep])
    for a in (out.lse, out.entropy, out.logp):
        assert torch.isnan(a[[1, 4]]).all()
    assert out.top_ids[1, 0] == 2500 and out.top_ids[4, :2].tolist() == [4000, 17]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("V,pitch,offset", [(1000, 1003, 1), (5001, 5001, 3), (2048, 2064, 0)])
def test_pitches_offsets_and_in_place(act, V, pitch, offset):
    T = 21
    op = PoetxLogProb(V, act, top=3)
    X, t = logits(T, V, act, 7, pitch, offset), targets(T, V, 2)
    out = op.forward(X, t)
    check_forward(op, X, t, out)
    a, b = torch.randn(T, device="cuda"), torch.randn(T, device="cuda")
    x0, saved = X.clone(), op.saved
    dX = logits(T, V, act, 8, pitch + 5, offset + 1)
    op.backward(a, b, dX)
    check_backward(op, x0, t, saved, a, b, dX)
    whole = dX._base if dX._base is not None else dX
    assert (whole[:offset + 1] == MARK).all() and (whole[offset + 1:offset + 1 + T * (pitch + 5)].view(T, -1)[:, V:] == MARK).all()
    op.backward(a, b, X)
    assert torch.equal(X, dX)


def test_without_targets_or_entropy():
    op = PoetxLogProb(700, "bf16", top=2)
    X = logits(5, 700, "bf16", 1)
    full = op.forward(X, targets(5, 700, 1))
    out = op.forward(X)
    assert out.logp is None and torch.equal(out.lse, full.lse) and torch.equal(out.top_ids, full.top_ids)
    assert op.forward(X[:0], targets(5, 700, 1)[:0]).lse.shape == (0,)
    assert op.backward(None, torch.zeros(0, device="cuda")).shape == (0, 700)


def test_rows_do_not_depend_on_their_number():
    """A row's results with a few rows (cut into parts) are within the bounds of those among many, and a call's are the
    same to the bit when it is repeated."""
    op = PoetxLogProb(9000, "f32", top=6)
    X, t = logits(2000, 9000, "f32", 9), targets(2000, 9000, 3)
    many, again = op.forward(X, t), op.forward(X, t)
    assert all(torch.equal(a, b) for a, b in zip(many, again))
    few = op.forward(X[:3], t[:3])
    assert torch.equal(few.top_ids, many.top_ids[:3])
    check_forward(op, X[:3], t[:3], few)


def test_gradients_by_differences():
    """fp32, along random directions: with a step of 2^-5 of unit length the cubic term is under 1e-3 of the gradient's
    norm, and a forward's rounding of 2^-20 is 2^-15 of the step."""
    op = PoetxLogProb(40, "f32", scale=1.3)
    X = logits(3, 40, "f32", 1, scale=1.0).clone()
    t = torch.tensor([3, -1, 39], dtype=torch.int32, device="cuda")
    a, b = torch.tensor([1.0, 2.0, -0.5], device="cuda"), torch.tensor([0.3, -1.0, 0.7], device="cuda")
    op.forward(X, t)
    g = op.backward(a, b)
    for s in range(4):
        d = logits(3, 40, "f32", 30 + s)
        d = d / d.norm()
        f = []
        for e in (2.0**-5, -(2.0**-5)):
            o = op.forward(X + e * d, t)
            f.append(float((a * o.logp).double().sum() + (b * o.entropy).double().sum()))
        num, ref = (f[0] - f[1]) * 16, float((g.double() * d.double()).sum())
        assert abs(num - ref) <= 2e-3 * float(g.double().norm()), (num, ref)


def test_graph_and_streams():
    op, other = PoetxLogProb(30000, "bf16", top=4), PoetxLogProb(30000, "bf16", top=4)
    X, t = logits(6, 30000, "bf16", 1), targets(6, 30000, 4)
    a = torch.randn(6, device="cuda")
    op.forward(X, t)
    op.backward(a, a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = op.forward(X, t)
        dX = op.backward(a, a)
    s = torch.cuda.Stream()
    for i in range(3):
        X.copy_(logits(6, 30000, "bf16", 10 + i))
        s.wait_stream(torch.cuda.current_stream())
        ref = other.forward(X, t, stream=s)
        torch.cuda.current_stream().wait_stream(s)
        dref = other.backward(a, a)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip([*out, dX], [*ref, dref]))
