"""GPU parity of the attention (poetx_attn_fwd / poetx_attn_bwd, layer.PoetxAttention) against the fp64 oracle.

Bounds, with u = 2^-24 and h half a step of the operand type (0 for fp32, 2^-8 for bf16; bf16 products are exact in fp32).
  * a score: hd terms summed in fp32, the scale, the difference to the maximum or lse and its product with log2 e:
    dx = u ((hd + 4) scale sum|q||k| + 4 |x - lse| + 2 |lse|), by which exp is off relatively, plus 2 u of its own.
  * forward: e = max over the row of dx + (tiles + 4) u, for the running rescalings, with at most nk / 32 + 2 tiles.
    The sum of p is off by e + nk u of itself, sum p v by (e + h + nk u) sum p |v|; the quotient and its rounding:
    O within (2 e + h + (2 nk + 4) u) sum p|v| + h |O|;  lse within e + nk u + 4 u |lse| + 4 u.
  * backward, at the saved lse and O: ep = dx + 4 u.  dO . v off by (hd + 1) u sum|dO||v|, D by (hd + 1) u sum|dO||O|;
    g = p (dO v - D) off by dg = p ((hd + 1) u (sum|dO||v| + sum|dO||O|) + 2 u |dO v - D|) + (ep + h) |g|.
    (The exponential gives 0 for what is under 2^-126, so p is off by up to t = 2^-126 besides, and so are its products:
    dg has t |dO v - D| more and dV's terms t |dO|, times the number of terms.)
    dQ within scale (sum dg|k| + (nk + 4) u sum|g||k|) + h |dQ|, dK likewise over the queries and heads (n of them),
    dV within sum p (ep + h + (n + 4) u) |dO| + h |dV|.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from orthogonal_reparameterized_cnp_amd import binding as B
from orthogonal_reparameterized_cnp_amd.layer import PoetxAttention

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

U = 2.0**-24
TINY = 2.0**-126
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 0.0, "bf16": 2.0**-8}
MARK = 77.0


def f64(t):
    return t.detach().double().cpu().numpy()


def rows(T, cols, act, seed, pitch=None, offset=0, scale=1.0):
    """[T, cols] of the given pitch, `offset` elements into a buffer whose other cells hold a mark."""
    g = torch.Generator().manual_seed(seed)
    pitch = pitch or cols
    buf = torch.full((offset + T * pitch + 8,), MARK, dtype=DT[act], device="cuda")
    v = buf[offset:offset + T * pitch].view(T, pitch)[:, :cols]
    v.copy_((scale * torch.randn(T, cols, generator=g)).to(DT[act]))
    return v


def cu_of(lens, first=0):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int64) + first


def dev(cu):
    return torch.tensor(cu, dtype=torch.int32, device="cuda")


def within(name, got, ref, tol):
    d = np.abs(got - ref)
    print(f"  {name}: worst |d| / bound {np.max(d / np.maximum(tol, 1e-300), initial=0.0):.3f}", flush=True)
    assert np.isfinite(got).all() and (d <= tol).all(), f"{name}: max |d| {d.max():.3e}"


def check(at, c, act, mats, dO, out, lse, grads, cu_q, cu_k):
    """Forward and backward of every sequence within the bounds above."""
    h, hd = HALF[act], c.head_dim
    Q, K, V = [f64(m) for m in mats]
    Od, ls, G = f64(out), f64(lse), f64(dO)
    refO, refl = O.attention(c, Q, K, V, cu_q, cu_k)
    ref = O.attention_backward(c, G, Q, K, V, Od, ls, cu_q, cu_k)
    tol = {n: np.zeros_like(r) for n, r in zip(("O", "dQ", "dK", "dV"), (refO, *ref))}
    tl = np.zeros_like(refl)
    fold = lambda x: c.join(x.reshape(c.kv_heads, -1, *x.shape[1:]).sum(1))
    for (q, k, x), v, g, o, a, b, e, f in zip(c.scores(Q, K, cu_q, cu_k), c.split(V, cu_k, c.kv_heads),
                                              c.split(G, cu_q, c.heads), c.split(Od, cu_q, c.heads),
                                              cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:]):
        nq, nk = b - a, f - e
        if nq == 0 or nk == 0:
            continue
        l = ls[:, a:b, None]
        l0 = np.where(np.isneginf(l), 0.0, l)
        p = np.exp(x - l0)
        dist = np.where(np.isneginf(x), 0.0, np.abs(x - l0))
        t = lambda y: y.transpose(0, 2, 1)
        dx = U * ((hd + 4) * c.scale * (abs(q) @ t(abs(k))) + 4 * dist + 2 * abs(l0))
        dx = np.where(p > 0, dx, 0.0)
        er = dx.max(2, keepdims=True) + (nk / 32 + 6) * U
        pv = p @ abs(v)
        tol["O"][a:b] = c.join((2 * er + h + (2 * nk + 4) * U) * pv + TINY * abs(v).sum(1, keepdims=True))
        tl[:, a:b] = (er + nk * U)[..., 0] + 4 * U * abs(l0[..., 0]) + 4 * U
        ep = dx + 4 * U
        dp = g @ t(v) - (g * o).sum(2, keepdims=True)
        gr = p * dp
        dg = p * ((hd + 1) * U * (abs(g) @ t(abs(v)) + (abs(g) * abs(o)).sum(2, keepdims=True)) + 2 * U * abs(dp))
        dg = dg + (ep + h) * abs(gr) + TINY * abs(dp)
        n = nq * c.heads // c.kv_heads
        tol["dQ"][a:b] = c.join(c.scale * ((dg + (nk + 4) * U * abs(gr)) @ abs(k)))
        tol["dK"][e:f] = fold(c.scale * (t(dg + (n + 4) * U * abs(gr)) @ abs(q)))
        tol["dV"][e:f] = fold(t(p * (ep + h + (n + 4) * U) + TINY) @ abs(g))
    for name, got, r in (("O", out, refO), *zip(("dQ", "dK", "dV"), grads, ref)):
        inside = np.zeros(len(r), bool)
        for cu in (cu_q if name in ("O", "dQ") else cu_k,):
            inside[cu[0]:cu[-1]] = True
        within(name, f64(got)[inside], r[inside], (tol[name] * (1 + h) + h * abs(r) + 1e-38)[inside])
    l, r = f64(lse)[:, cu_q[0]:cu_q[-1]], refl[:, cu_q[0]:cu_q[-1]]
    assert (np.isneginf(l) == np.isneginf(r)).all()
    fin = ~np.isneginf(r)
    within("lse", l[fin], r[fin], tl[:, cu_q[0]:cu_q[-1]][fin])


def run(heads, kv, hd, act, lq, lk, causal=True, window=0, seed=0, first=0, behind=0, scale=None, qk=1.0):
    """Forward and backward on rows with `first` unused ones before the sequences and `behind` after them."""
    at = PoetxAttention(heads, kv, hd, act, causal, window, scale)
    c = O.Attn(heads, kv, hd, float(np.float32(at.desc.scale)), causal, window)
    cu_q, cu_k = cu_of(lq, first), cu_of(lk, first)
    Tq, Tk = cu_q[-1] + behind, cu_k[-1] + behind
    mats = (rows(Tq, heads * hd, act, seed + 1, scale=qk), rows(Tk, kv * hd, act, seed + 2, scale=qk),
            rows(Tk, kv * hd, act, seed + 3))
    dO = rows(Tq, heads * hd, act, seed + 4)
    print(f"attention {heads}/{kv} x {hd} {act} q {lq} k {lk} causal={causal} window={window}", flush=True)
    out = at.forward(*mats, dev(cu_q), dev(cu_k))
    grads = at.backward(dO)
    torch.cuda.synchronize()
    check(at, c, act, mats, dO, out, at.saved[4], grads, cu_q, cu_k)
    return at, mats, dO, out, grads, cu_q, cu_k


LENS = [
    ([1], [1]),
    ([5], [5]),
    ([128, 64, 32], [128, 64, 32]),
    ([129, 0, 1, 63, 33], [129, 0, 1, 63, 33]),
    ([1, 1, 1], [300, 64, 1]),
    ([7, 40, 0, 3], [100, 33, 5, 0]),
    ([200], [77]),
]


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 20), (False, 9)])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("lq,lk", LENS)
@pytest.mark.parametrize("heads,kv,hd", [(2, 1, 64), (2, 2, 128)])
def test_masks_and_lengths(heads, kv, hd, act, lq, lk, causal, window):
    run(heads, kv, hd, act, lq, lk, causal, window)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,hd", [(1, 1, 1), (3, 1, 3), (6, 3, 75), (8, 2, 80), (4, 4, 96), (5, 5, 127), (4, 1, 8),
                                         (2, 2, 33), (9, 3, 64), (12, 2, 128)])
def test_heads(heads, kv, hd, act):
    run(heads, kv, hd, act, [70, 1, 150], [70, 1, 150])
    run(heads, kv, hd, act, [3, 140], [260, 141], causal=False, window=50, seed=9)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 100)])
def test_longer(act, causal, window):
    run(4, 2, 64, act, [700, 513], [700, 513], causal, window)
    run(2, 1, 128, act, [400, 1], [1000, 900], causal, window, seed=5)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_single_tokens_over_long_keys(act):
    run(8, 2, 128, act, [1, 1, 1, 1], [4000, 3, 1024, 2049])
    run(4, 4, 64, act, [2, 1], [3000, 2500], window=700)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("scale,qk", [(1e-3, 1.0), (4.0, 2.0)])
def test_flat_and_sharp_rows(act, scale, qk):
    """Probabilities all alike, and rows whose largest one is nearly 1."""
    run(2, 1, 64, act, [150], [150], scale=scale, qk=qk)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_rows_outside_the_sequences(act):
    """Rows before the first sequence and behind the last are neither read (they may hold anything) nor written."""
    heads, kv, hd, cu_q, cu_k = 4, 2, 64, cu_of([40, 90], 5), cu_of([60, 90], 3)
    at = PoetxAttention(heads, kv, hd, act)
    Tq, Tk = 5 + 130 + 11, 3 + 150 + 9
    mats = [rows(Tq, heads * hd, act, 1), rows(Tk, kv * hd, act, 2), rows(Tk, kv * hd, act, 3)]
    dO = rows(Tq, heads * hd, act, 4)
    out = torch.full_like(mats[0], MARK)
    grads = [torch.full_like(m, MARK) for m in mats]
    plain = at.forward(*mats, dev(cu_q), dev(cu_k)).clone()
    plain_grads = [g.clone() for g in at.backward(dO)]
    assert not plain[:5].any() and not plain_grads[1][-9:].any()
    for m, cu in zip([*mats, dO], (cu_q, cu_k, cu_k, cu_q)):
        m[:cu[0]] = float("nan")
        m[cu[-1]:] = float("inf")
    at.forward(*mats, dev(cu_q), dev(cu_k), O=out)
    at.backward(dO, *grads)
    for got, ref, cu in ((out, plain, cu_q), *zip(grads, plain_grads, (cu_q, cu_k, cu_k))):
        assert torch.equal(got[cu[0]:cu[-1]], ref[cu[0]:cu[-1]])
        assert (got[:cu[0]] == MARK).all() and (got[cu[-1]:] == MARK).all()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_nan_stays_in_its_sequence(act):
    lens = [30, 50, 64, 7]
    cu = cu_of(lens)
    at = PoetxAttention(2, 1, 64, act)
    mats = [rows(151, n * 64, act, s) for n, s in ((2, 1), (1, 2), (1, 3))]
    dO = rows(151, 128, act, 4)
    ref = [at.forward(*mats, dev(cu)).clone(), *[g.clone() for g in at.backward(dO)]]
    for m in (*mats, dO):
        m[cu[1]:cu[2]] = float("nan")
        m[cu[1] + 3] = float("inf")
    got = [at.forward(*mats, dev(cu)), *at.backward(dO)]
    for g, r in zip(got, ref):
        assert torch.equal(g[:cu[1]], r[:cu[1]]) and torch.equal(g[cu[2]:], r[cu[2]:])
        assert torch.isnan(g[cu[1]:cu[2]].float()).any()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,hd,offset,gap", [(4, 2, 64, 0, 0), (4, 2, 64, 1, 3), (2, 2, 128, 8, 8), (3, 1, 75, 1, 0)])
def test_columns_of_one_buffer(act, heads, kv, hd, offset, gap):
    """Q, K and V as columns of one buffer, their gradients as columns of another, at any pitch and element offset: within
    the bounds, and the cells around them as they were."""
    T, n = 200, (heads + 2 * kv) * hd
    pitch = n + gap
    at = PoetxAttention(heads, kv, hd, act)
    lens = cu_of([64, 136])
    cu = dev(lens)
    buf = rows(T, n, act, 1, pitch, offset)
    cut = lambda m: (m[:, :heads * hd], m[:, heads * hd:(heads + kv) * hd], m[:, (heads + kv) * hd:])
    whole = torch.full((offset + T * pitch + 8,), MARK, dtype=DT[act], device="cuda")
    grads = whole[offset:offset + T * pitch].view(T, pitch)
    out = rows(T, heads * hd, act, 3, heads * hd + gap, offset)
    at.forward(*cut(buf), cu, O=out)
    dO = rows(T, heads * hd, act, 2, heads * hd + gap, offset)
    at.backward(dO, *cut(grads[:, :n]))
    c = O.Attn(heads, kv, hd, float(np.float32(at.desc.scale)))
    check(at, c, act, cut(buf), dO, out, at.saved[4], cut(grads[:, :n]), lens, lens)
    assert (grads[:, n:] == MARK).all() and (whole[:offset] == MARK).all() and (whole[offset + T * pitch:] == MARK).all()


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_equal_sequences_without_offsets(act):
    at = PoetxAttention(4, 2, 64, act)
    mats = [rows(3 * 70, 256, act, 1), rows(3 * 70, 128, act, 2), rows(3 * 70, 128, act, 3)]
    dO = rows(210, 256, act, 4)
    cu = dev(cu_of([70, 70, 70]))
    ref = [at.forward(*mats, cu).clone(), *at.backward(dO)]
    got = [at.forward(*mats, batch=3).clone(), *at.backward(dO)]
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_many_sequences():
    """More sequences than rows, most of them empty, and a run of single tokens."""
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 2, 3000)
    lens[1234] = 150
    run(1, 1, 16, "bf16", list(lens), list(lens), seed=3)
    run(2, 1, 64, "f32", [1] * 300, [1] * 300)


def test_no_rows():
    at = PoetxAttention(2, 1, 64, "bf16")
    e = lambda n, c: torch.zeros(n, c, dtype=torch.bfloat16, device="cuda")
    z = dev([0, 0, 0])
    assert at.forward(e(0, 128), e(5, 64), e(5, 64), z, dev([0, 2, 5])).shape == (0, 128)
    dK = torch.full((5, 64), MARK, dtype=torch.bfloat16, device="cuda")
    _, dK, dV = at.backward(e(0, 128), dK=dK)
    assert not dK.any() and not dV.any()
    out = at.forward(rows(4, 128, "bf16", 1), e(0, 64), e(0, 64), dev([0, 1, 4]), z)
    assert not out.any() and torch.isneginf(at.saved[4]).all()
    dQ, dK, dV = at.backward(rows(4, 128, "bf16", 2))
    assert not dQ.any() and dK.shape == (0, 64)


def test_runs_alike():
    """No atomics: two runs are the same to the bit, and a sequence's results do not depend on its neighbours."""
    at = PoetxAttention(8, 2, 128)
    mats = [rows(600, 1024, "bf16", 1), rows(600, 256, "bf16", 2), rows(600, 256, "bf16", 3)]
    dO, cu = rows(600, 1024, "bf16", 4), dev(cu_of([100, 300, 200]))
    one = [at.forward(*mats, cu).clone(), *at.backward(dO)]
    two = [at.forward(*mats, cu).clone(), *at.backward(dO)]
    assert all(torch.equal(a, b) for a, b in zip(one, two))
    alone = [at.forward(*[m[100:400] for m in mats], dev([0, 300])).clone(), *at.backward(dO[100:400])]
    assert all(torch.equal(a[100:400], b) for a, b in zip(one, alone))


def test_gradients_by_differences():
    """fp32, along random directions: (f(x + s d) - f(x - s d)) / 2 s against the gradients.  With s = 2^-6 the cubic term
    of these rows of 24 keys stays under 1e-4 of the derivative's scale, and a forward's rounding of 2^-22 is 2^-16 of it."""
    at = PoetxAttention(4, 2, 32, "f32", True, 9)
    cu = dev(cu_of([24, 10]))
    mats = [rows(34, 128, "f32", 1).clone(), rows(34, 64, "f32", 2).clone(), rows(34, 64, "f32", 3).clone()]
    dO = rows(34, 128, "f32", 4)
    at.forward(*mats, cu)
    grads = [g.clone() for g in at.backward(dO)]
    for i in range(3):
        d = rows(34, mats[i].shape[1], "f32", 20 + i)
        d = d / d.double().norm().float()
        f = []
        for s in (2.0**-6, -(2.0**-6)):
            m = [x.clone() for x in mats]
            m[i] += s * d
            f.append(float((at.forward(*m, cu).double() * dO.double()).sum()))
        num, ref = (f[0] - f[1]) / 2.0**-5, float((grads[i].double() * d.double()).sum())
        assert abs(num - ref) <= 1e-3 * float(grads[i].double().norm()), (i, num, ref)


def test_graph_replays():
    """Forward and backward in one graph, replayed on new data between eager calls of the same object."""
    at, other = PoetxAttention(4, 2, 64), PoetxAttention(4, 2, 64)
    mats = [rows(300, 256, "bf16", 1), rows(300, 128, "bf16", 2), rows(300, 128, "bf16", 3)]
    dO, cu = rows(300, 256, "bf16", 4), dev(cu_of([1, 199, 100]))
    at.forward(*mats, cu)
    at.backward(dO)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = at.forward(*mats, cu)
        grads = at.backward(dO)
    for i in range(3):
        for k, m in enumerate([*mats, dO]):
            m.copy_(rows(300, m.shape[1], "bf16", 50 + 4 * i + k))
        ref = [other.forward(*mats, cu).clone(), *other.backward(dO)]
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([out, *grads], ref))


def test_two_streams_at_once():
    """Two objects on two streams, and a backward on another stream than its forward."""
    ats = [PoetxAttention(4, 2, 64), PoetxAttention(4, 2, 64)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    cu = dev(cu_of([500, 268]))
    data = [[rows(768, 256, "bf16", 10 * s + 1), rows(768, 128, "bf16", 10 * s + 2), rows(768, 128, "bf16", 10 * s + 3),
             rows(768, 256, "bf16", 10 * s + 4)] for s in range(2)]
    ref = []
    for at, (q, k, v, g) in zip(ats, data):
        ref.append([at.forward(q, k, v, cu).clone(), *at.backward(g)])
    torch.cuda.synchronize()
    got = []
    for at, (q, k, v, g), s in zip(ats, data, streams):
        got.append([at.forward(q, k, v, cu, stream=s)])
    for i, (at, (q, k, v, g)) in enumerate(zip(ats, data)):
        streams[1 - i].wait_stream(streams[i])
        got[i] += at.backward(g, stream=streams[1 - i])
    torch.cuda.synchronize()
    for a, b in zip(got, ref):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_of_no_use_stay_in_bounds():
    """Offsets that decrease or leave the rows (which the documentation forbids) are held within them: nothing outside the
    operands is touched, and sequences that are in order are right."""
    at = PoetxAttention(2, 1, 64)
    mats = [rows(100, 128, "bf16", 1), rows(100, 64, "bf16", 2), rows(100, 64, "bf16", 3)]
    ref = at.forward(*[m[:40] for m in mats], dev([0, 40])).clone()
    big = torch.full((300, 128), MARK, dtype=torch.bfloat16, device="cuda")
    out = big[100:200]
    at.forward(*mats, dev([0, 40, 1 << 30, -5, 200]), O=out)
    at.backward(rows(100, 128, "bf16", 4))
    torch.cuda.synchronize()
    assert torch.equal(out[:40], ref) and (big[:100] == MARK).all() and (big[200:] == MARK).all()
