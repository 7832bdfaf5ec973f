"""GPU parity of the norm (poetx_norm_fwd / poetx_norm_bwd, layer.PoetxNorm) against the fp64 oracle.

Bounds, with u = 2^-24 and h half a step of the output type (0 extra for fp32, 2^-8 for bf16).  A row sum adds each
thread's at most 32 elements one after another, then 6 shuffle steps and at most 16 waves: n = 54 additions, each
off by at most u times the running sum of magnitudes.
  * mean: n u mean|S| and one rounding; it moves every S - mu by as much.
  * rs: the variance is off by (n + 3) u of itself (the mean's error enters squared, which stays under the bound's
    slack), halved by the root, plus 3 roundings: 32 u.
  * Y = (S - mu) rs w + b: 4 more roundings: u (40 |xh w| + 56 rs |w| mean|S| + |Y|) + h |Y|.
  * backward, at the saved statistics: xh off by 2 u; the row means of g and g xh by (n + 5) u of their mean
    magnitudes; the sum by 4 more roundings: u rs (8 (|g| + |xh| |m0|) + 62 mean|g| + 62 |xh| mean|g xh|)
    + u (2 |dS| + |dX|) + h |dX|.
  * dw, db: N additions with N at most the rows of one workgroup's thread + 4 + parts / 16 + 16 <= T / 256 + 64 here,
    or T where there are fewer rows: u (N + 4) sum|dY xh|.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from orthogonal_reparameterized_cnp_amd import binding as B
from orthogonal_reparameterized_cnp_amd.layer import PoetxNorm

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

U = 2.0**-24
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 0.0, "bf16": 2.0**-8}


def _rows(T, d, act, seed, pitch=None, offset=0, scale=1.0):
    """A [T, d] matrix of the given row pitch whose first element is `offset` elements into its storage; the cells
    between the rows hold a mark."""
    g = torch.Generator().manual_seed(seed)
    pitch = pitch or d
    buf = torch.full((offset + T * pitch + 8,), 77.0, dtype=DT[act], device="cuda")
    v = buf[offset:offset + T * pitch].view(T, pitch)[:, :d]
    if T:
        v.copy_((torch.randn(T, d, generator=g) * scale * (0.3 + 2 * torch.rand(T, 1, generator=g)) + 0.4).to(DT[act]))
    return v


def f64(t):
    return t.detach().double().cpu().numpy()


def _within(name, got, ref, tol):
    d = np.abs(got - ref)
    worst = float(np.max(d / np.maximum(tol, 1e-300), initial=0.0))
    print(f"  {name}: worst |d| / bound {worst:.3f}", flush=True)
    assert np.isfinite(got).all() and (d <= tol).all(), f"{name}: max |d| {d.max():.3e}"


def check_forward(norm, S, Y, act):
    w = f64(norm.weight)
    b = None if norm.bias is None else f64(norm.bias)
    Sd = f64(S)
    ref, mean, rs = O.norm_forward(Sd, w, b, norm.kind, float(np.float32(norm.eps)))
    mag = np.abs(Sd).mean(1, keepdims=True) if norm.kind == "layer" else np.zeros((len(Sd), 1))
    xw = np.abs((Sd - mean[:, None]) * rs[:, None] * w)
    tol = U * (40 * xw + 56 * rs[:, None] * np.abs(w) * mag + np.abs(ref))
    _within("Y", f64(Y), ref, tol * (1 + HALF[act]) + HALF[act] * np.abs(ref) + 1e-38)
    st = f64(norm.stats)
    if norm.kind == "layer":
        _within("mean", st[0], mean, U * 56 * mag[:, 0] + 1e-38)
    # the mean's own error d moves the variance by d^2, and the deviation by rs^2 d^2 / 2 of itself
    off = (56 * U * mag[:, 0] * rs) ** 2
    _within("rs", st[-1], rs, (32 * U + off) * rs)


def check_backward(norm, S, dY, dS, dX, dw, db, act):
    w, st, Sd, dYd = f64(norm.weight), f64(norm.stats), f64(S), f64(dY)
    mean, rs = (st[0], st[1]) if norm.kind == "layer" else (np.zeros(len(Sd)), st[0])
    ref, rdw, rdb = O.norm_backward(Sd, dYd, w, mean, rs, norm.kind)
    xh, g = (Sd - mean[:, None]) * rs[:, None], dYd * w
    dSd = 0.0 if dS is None else f64(dS)
    ref = ref + dSd
    m0 = np.abs((g * xh).mean(1, keepdims=True))
    tol = U * rs[:, None] * (8 * (np.abs(g) + np.abs(xh) * m0) + 62 * np.abs(g).mean(1, keepdims=True)
                             + 62 * np.abs(xh) * np.abs(g * xh).mean(1, keepdims=True))
    tol = tol + U * (2 * np.abs(dSd) + np.abs(ref))
    _within("dX", f64(dX), ref, tol * (1 + HALF[act]) + HALF[act] * np.abs(ref) + 1e-38)
    N = min(len(Sd), len(Sd) // 256 + 64) + 4
    _within("dw", f64(dw), rdw, U * N * np.abs(dYd * xh).sum(0) + 1e-38)
    if db is not None:
        _within("db", f64(db), rdb, U * N * np.abs(dYd).sum(0) + 1e-38)


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("T,d", [(1, 1), (3, 2), (1, 4096), (5, 7), (64, 256), (130, 513), (37, 1376), (600, 1025),
                                 (9, 2049), (17, 5461), (4, 14336), (2, 20000), (2, 32768), (2600, 40), (1100, 5461),
                                 (600, 7001), (300, 10001), (300, 12289), (1300, 513), (700, 3)])
def test_forward_backward(T, d, act, kind, res):
    print(f"norm T={T} d={d} {act} {kind} res={res}", flush=True)
    norm = PoetxNorm(d, kind, act)
    g = torch.Generator().manual_seed(d)
    norm.weight.copy_(1 + 0.3 * torch.randn(d, generator=g))
    if norm.bias is not None:
        norm.bias.copy_(0.2 * torch.randn(d, generator=g))
    X, R = _rows(T, d, act, 1), _rows(T, d, act, 2) if res else None
    out = norm.forward(X, R)
    Y, S = out if res else (out, X)
    if res:
        assert torch.equal(S, (X.float() + R.float()).to(DT[act]))
    dY, dS = _rows(T, d, act, 3, scale=0.1), _rows(T, d, act, 4, scale=0.1) if res else None
    dX, dw, db = norm.backward(dY, dS)
    torch.cuda.synchronize()
    check_forward(norm, S, Y, act)
    check_backward(norm, S, dY, dS, dX, dw, db, act)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("d,pitch,offset", [(256, 300, 0), (100, 103, 1), (1376, 1377, 3), (4096, 4099, 5)])
def test_pitches_and_unaligned_rows(act, d, pitch, offset):
    """Rows of any pitch and alignment; the cells between them are neither read into a result nor written."""
    print(f"norm pitch d={d} pitch={pitch} offset={offset} {act}", flush=True)
    T = 33
    norm = PoetxNorm(d, "layer", act)
    norm.weight.copy_(torch.linspace(0.5, 1.5, d))
    X, R = (_rows(T, d, act, s, pitch + s, offset) for s in (1, 2))
    S, Y = (_rows(T, d, act, s, pitch + s, offset + s) for s in (3, 4))
    norm.forward(X, R, Y=Y, S=S)
    dY, dS, dX = (_rows(T, d, act, s, pitch + s, offset) for s in (5, 6, 7))
    _, dw, db = norm.backward(dY, dS, dX=dX)
    torch.cuda.synchronize()
    check_forward(norm, S, Y, act)
    check_backward(norm, S, dY, dS, dX, dw, db, act)
    for t in (S, Y, dX):
        gap = t.as_strided((T, t.stride(0) - d), (t.stride(0), 1), t.storage_offset() + d)
        assert (gap == 77.0).all()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T,d", [(50, 1376), (1100, 5461), (3000, 1377), (600, 513), (5000, 63)])
def test_in_place(act, T, d):
    """S in place of the residual, dX in place of dS or dY: the results of separate buffers, bit for bit."""
    norm = PoetxNorm(d, "layer", act)
    X, R = _rows(T, d, act, 1), _rows(T, d, act, 2)
    Y, S = norm.forward(X, R)
    dY, dS = _rows(T, d, act, 3), _rows(T, d, act, 4)
    dX, dw, db = norm.backward(dY, dS)
    R2 = R.clone()
    Y2, S2 = norm.forward(X, R2, S=R2)
    assert S2 is R2 and torch.equal(S2, S) and torch.equal(Y2, Y)
    for which in (0, 1):
        a, b = dY.clone(), dS.clone()
        got, dw2, db2 = norm.backward(a, b, dX=(a, b)[which])
        assert torch.equal(got, dX) and torch.equal(dw2, dw) and torch.equal(db2, db)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_operands_in_each_others_gaps(act):
    """Y beside X, and dX beside dY, as columns of one array: the results of separate arrays, bit for bit."""
    T, d = 70, 513
    norm = PoetxNorm(d, "layer", act)
    X, dY = _rows(T, d, act, 1), _rows(T, d, act, 2)
    Y = norm.forward(X)
    dX, dw, db = norm.backward(dY)
    both = torch.cat([X, torch.zeros_like(X)], 1)
    assert torch.equal(norm.forward(both[:, :d], Y=both[:, d:]), Y) and torch.equal(both[:, :d], X)
    both = torch.cat([torch.zeros_like(dY), dY], 1)
    norm.forward(X)
    got = norm.backward(both[:, d:], dX=both[:, :d])
    assert all(torch.equal(a, b) for a, b in zip(got, (dX, dw, db))) and torch.equal(both[:, d:], dY)
    with pytest.raises(B.PoetxError):
        norm.forward(both[:, :d], Y=both[:, 1:d + 1])


def test_rows_that_degenerate():
    """A constant row and a zero row have variance 0; a NaN or an infinity stays in its own row and in the column sums."""
    d = 300
    norm = PoetxNorm(d, "layer", "f32", eps=1e-4)
    X = _rows(6, d, "f32", 1)
    X[1], X[2] = 3.25, 0.0
    Y = norm.forward(X)
    torch.cuda.synchronize()
    assert torch.equal(Y[1], torch.zeros(d, device="cuda")) and torch.equal(Y[2], torch.zeros(d, device="cuda"))
    check_forward(norm, X, Y, "f32")
    clean = Y.clone()
    X[3, 7], X[4, 0] = float("nan"), float("inf")
    Y = norm.forward(X)
    dX, dw, _ = norm.backward(torch.ones_like(X))
    torch.cuda.synchronize()
    for t in (0, 1, 2, 5):
        assert torch.equal(Y[t], clean[t]) and torch.isfinite(dX[t]).all()
    assert torch.isnan(Y[3]).all() and torch.isnan(Y[4]).any() and torch.isnan(dw).any()


def test_no_rows():
    norm = PoetxNorm(64, "layer", "bf16")
    assert norm.forward(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")).shape == (0, 64)
    dw, db = torch.ones(64, device="cuda"), torch.ones(64, device="cuda")
    norm.backward(torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), dw=dw, db=db)
    assert not dw.any() and not db.any()


def test_no_parameters_and_partial_gradients():
    """NULL weight and bias are ones and zeros; dw and dbias may each be left out."""
    T, d = 20, 96
    X, dY = _rows(T, d, "f32", 1), _rows(T, d, "f32", 2)
    norm = PoetxNorm(d, "layer", "f32")
    Y = norm.forward(X)
    dX, dw, db = norm.backward(dY)
    dsc = norm.desc
    Y2, st, dX2, dw2, db2 = torch.empty_like(Y), torch.empty(2, T, device="cuda"), *(torch.empty_like(t) for t in (dX, dw, db))
    ws = torch.empty(B.poetx_norm_workspace_size(dsc, T), dtype=torch.uint8, device="cuda")
    B.poetx_norm_fwd(dsc, T, X, d, None, d, None, None, None, d, Y2, d, st)
    assert torch.equal(Y2, Y) and torch.equal(st, norm.stats)
    B.poetx_norm_bwd(dsc, T, dY, d, X, d, None, st, None, d, dX2, d, dw2, None, ws, ws.numel())
    assert torch.equal(dX2, dX) and torch.equal(dw2, dw)
    dX2.zero_()
    B.poetx_norm_bwd(dsc, T, dY, d, X, d, None, st, None, d, dX2, d, None, db2, ws, ws.numel())
    assert torch.equal(dX2, dX) and torch.equal(db2, db)
    dX2.zero_()
    B.poetx_norm_bwd(dsc, T, dY, d, X, d, None, st, None, d, dX2, d, None, None, ws, ws.numel())
    assert torch.equal(dX2, dX)


def test_gradients_match_differences_of_the_kernel():
    """Central differences of the fp32 forward's loss along random directions: the loss is summed in float64, its
    terms are off by at most 100 u |Y| each, so the quotient by 2 e is off by 100 u sum|Y dY| / e, and by e^2 times
    the third derivative."""
    T, d = 4, 48
    norm = PoetxNorm(d, "layer", "f32", eps=1e-2)
    norm.weight.copy_(torch.linspace(0.5, 1.5, d))
    X, dY = _rows(T, d, "f32", 1), _rows(T, d, "f32", 2)
    Y = norm.forward(X)
    dX, dw, db = norm.backward(dY)
    e = 2.0**-7
    noise = 100 * U * float((Y.double() * dY.double()).abs().sum()) / e
    for k in range(4):
        V = _rows(T, d, "f32", 10 + k)
        lo, hi = (float((norm.forward(X + s * e * V).double() * dY.double()).sum()) for s in (-1, 1))
        lo2, hi2 = (float((norm.forward(X + s * 2 * e * V).double() * dY.double()).sum()) for s in (-1, 1))
        # Richardson's combination of steps e and 2 e drops the e^2 term; what is left is of order e^4
        d1, d2 = (hi - lo) / (2 * e), (hi2 - lo2) / (4 * e)
        want = float((dX.double() * V.double()).sum())
        assert abs((4 * d1 - d2) / 3 - want) <= 2 * noise + 0.1 * abs(d1 - d2) + 1e-9, (k, d1, d2, want)


@pytest.mark.parametrize("kind,res", [("layer", False), ("rms", True)])
def test_replays_in_a_graph(kind, res):
    T, d = 700, 1376
    norm = PoetxNorm(d, kind, "bf16")
    X, R = _rows(T, d, "bf16", 1), _rows(T, d, "bf16", 2) if res else None
    dY, dS = _rows(T, d, "bf16", 3), _rows(T, d, "bf16", 4) if res else None
    outs = [torch.empty(T, d, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    dw = torch.empty(d, device="cuda")

    def step():
        norm.forward(X, R, Y=outs[0], S=outs[1] if res else None)
        norm.backward(dY, dS, dX=outs[2], dw=dw)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    ref = [t.clone() for t in outs + [dw]]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(3):
        X.mul_(1.0)  # eager work between the replays
        for t in (outs if res else [outs[0], outs[2]]) + [dw]:
            t.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(outs + [dw], ref)):
            if res or i != 1:
                assert torch.equal(a, b), f"replay {k}"


def test_on_another_stream():
    """A call on a stream of its own, and two at once on two streams: each allocates its own workspace."""
    T, d = 900, 2048
    norms = [PoetxNorm(d, "layer", "bf16") for _ in range(2)]
    Xs, dYs = [_rows(T, d, "bf16", k) for k in (1, 2)], [_rows(T, d, "bf16", k) for k in (3, 4)]
    ref = []
    for n, X, dY in zip(norms, Xs, dYs):
        Y = n.forward(X)
        ref.append((Y, *n.backward(dY)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [None, None]
    for _ in range(3):
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.current_stream())
            Y = norms[i].forward(Xs[i], stream=s)
            got[i] = (Y, *norms[i].backward(dYs[i], stream=s))
    torch.cuda.synchronize()
    for a, b in zip(got, ref):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
    with pytest.raises(TypeError):
        norms[0].forward(Xs[0], stream=streams[0].cuda_stream)
