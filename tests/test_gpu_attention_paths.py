"""GPU parity of the attention where its calls take other ways than at small sizes: more workgroups than the card holds at
once (their order, and key heads whose query heads one workgroup sums alone), the forward of few rows (rows of several
heads in a tile, many parts, sequences of more than a tile), and offsets past 32 bits.  Bounds as in
tests/test_gpu_attention.py."""

import numpy as np
import pytest
import torch

import oracle as O
from orthogonal_reparameterized_cnp_amd import binding as B
from orthogonal_reparameterized_cnp_amd.layer import PoetxAttention, PoetxLogProb, PoetxRope

from . import test_gpu_attention as A
from . import test_gpu_logp as LP
from . import test_gpu_rope as R

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]


def _lens(n, most, seed):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, most, n)
    lens[n // 2] = most
    lens[n // 3] = 0
    return [int(x) for x in lens]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("causal", [True, False])
def test_more_workgroups_than_the_card_holds(act, causal):
    lens = _lens(20, 300, 1)
    A.run(64, 16, 16, act, lens, lens, causal)
    A.run(64, 16, 64, act, [256] * 9, [256] * 9, causal, seed=5)
    # more sequences than a wave has lanes
    lens = _lens(100, 60, 2)
    A.run(16, 8, 64, act, lens, lens, causal, seed=9)


@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_queries_and_keys_of_other_lengths_in_order(act):
    lq, lk = _lens(30, 200, 3), _lens(30, 400, 4)
    A.run(32, 32, 32, act, lq, lk, True)
    A.run(32, 32, 128, act, lq[:12], lk[:12], False, window=70, seed=7)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("heads,kv,hd,lq,lk", [
    (2, 1, 64, [1], [20000]),  # 79 parts
    (32, 1, 128, [1, 1, 1], [3000, 600, 1]),  # a full tile of rows
    (32, 1, 64, [2, 0, 0, 0], [2000, 5, 0, 700]),  # more rows than a tile: tiles shared, not keys
    (24, 8, 128, [1, 0, 2, 3, 1], [1500, 9, 1300, 2, 0]),
    (5, 5, 75, [1] * 70, list(range(0, 350, 5))),  # more sequences than a wave has lanes
    (8, 2, 96, [1, 2], [4000, 900]),
])
def test_few_rows(act, heads, kv, hd, lq, lk):
    A.run(heads, kv, hd, act, lq, lk)
    A.run(heads, kv, hd, act, lq, lk, window=500, seed=3)  # parts that no row sees
    A.run(heads, kv, hd, act, lq, lk, causal=False, seed=6, first=3, behind=2)


def test_few_rows_leave_others_alone():
    """Single tokens with rows between the last sequence and the end, an O of another pitch."""
    at = PoetxAttention(8, 2, 64)
    cu_q, cu_k = A.cu_of([1, 1, 1], 2), A.cu_of([900, 0, 1200], 1)
    mats = [A.rows(9, 512, "bf16", 1), A.rows(2110, 128, "bf16", 2), A.rows(2110, 128, "bf16", 3)]
    out = torch.full((9, 520), A.MARK, dtype=torch.bfloat16, device="cuda")
    at.forward(*mats, A.dev(cu_q), A.dev(cu_k), O=out[:, :512])
    assert (out[:2] == A.MARK).all() and (out[5:] == A.MARK).all() and (out[:, 512:] == A.MARK).all()
    assert not out[3, :512].any() and torch.isneginf(at.saved[4][:, 3]).all() and out[2, :512].any()


def test_few_rows_in_a_graph():
    at, other = PoetxAttention(8, 2, 64), PoetxAttention(8, 2, 64)
    mats = [A.rows(3, 512, "bf16", 1), A.rows(4000, 128, "bf16", 2), A.rows(4000, 128, "bf16", 3)]
    cu_q, cu_k = A.dev(A.cu_of([1, 1, 1])), A.dev(A.cu_of([100, 3000, 900]))
    at.forward(*mats, cu_q, cu_k)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = at.forward(*mats, cu_q, cu_k)
    for i in range(3):
        for k, m in enumerate(mats):
            m.copy_(A.rows(len(m), m.shape[1], "bf16", 20 + 3 * i + k))
        # other lengths at replay: the offsets are read on the device
        cu_k.copy_(A.dev(A.cu_of([100 + 500 * i, 3000 - 700 * i, 900 - 50 * i])))
        ref = other.forward(*mats, cu_q, cu_k).clone()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


@pytest.mark.parametrize("pitch,T", [(1 << 20, 2200), ((1 << 24) + 8, 140)])
def test_offsets_past_32_bits(pitch, T):
    """Q, K and V as columns of one buffer of more than 2^31 elements, by direct copies and (the wider pitch) without."""
    heads, kv, hd = 2, 1, 64
    lens = [T - 100, 100]
    cu = A.cu_of(lens)
    buf = A.rows(T, 256, "bf16", 1, pitch)
    mats = (buf[:, :128], buf[:, 128:192], buf[:, 192:])
    at = PoetxAttention(heads, kv, hd)
    c = O.Attn(heads, kv, hd, float(np.float32(at.desc.scale)))
    dO = A.rows(T, 128, "bf16", 2, pitch)
    out = at.forward(*mats, A.dev(cu))
    grads = at.backward(dO)
    A.check(at, c, "bf16", mats, dO, out, at.saved[4], grads, cu, cu)
    # single tokens over the same keys
    q = A.rows(2, 128, "bf16", 3)
    cu1 = A.cu_of([1, 1])
    out = at.forward(q, mats[1], mats[2], A.dev(cu1), A.dev(cu))
    g1 = A.rows(2, 128, "bf16", 4)
    grads = at.backward(g1)
    A.check(at, c, "bf16", (q, *mats[1:]), g1, out, at.saved[4], grads, cu1, cu)


def test_offsets_past_32_bits_of_the_others():
    T, pitch = 2200, 1 << 20
    X = R.rows(T, 256, "bf16", 1, pitch)
    rope = PoetxRope(64)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    R.check(rope, X, rope.forward([X], pos, [X.new_empty(T, 256)])[0], pos)
    op = PoetxLogProb(256, "bf16", top=3)
    t = LP.targets(T, 256, 1)
    LP.check_forward(op, X, t, op.forward(X, t))
    a = torch.randn(T, device="cuda")
    LP.check_backward(op, X, t, op.saved, a, a, op.backward(a, a))


def test_workspaces_hold_what_the_calls_write():
    """A call with exactly the bytes that were asked for leaves the bytes behind them alone."""
    for lq, lk, heads, kv, hd in (([1, 1], [3000, 700], 8, 2, 64), ([130, 70], [130, 70], 8, 2, 128), ([1], [2000], 3, 1, 75)):
        cu_q, cu_k = A.cu_of(lq), A.cu_of(lk)
        Tq, Tk = int(cu_q[-1]), int(cu_k[-1])
        d = B.attn_desc(heads, kv, hd, "bf16")
        nq, nk = heads * hd, kv * hd
        q, k, v, g = (A.rows(T, n, "bf16", s) for T, n, s in ((Tq, nq, 1), (Tk, nk, 2), (Tk, nk, 3), (Tq, nq, 4)))
        o, lse = torch.empty_like(q), torch.empty(heads, Tq, device="cuda")
        args = (len(lq), Tq, Tk, A.dev(cu_q), A.dev(cu_k))
        for op in (B.POETX_OP_FWD, B.POETX_OP_BWD):
            n = B.poetx_attn_workspace_size(d, len(lq), Tq, Tk, op)
            ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
            if op == B.POETX_OP_FWD:
                B.poetx_attn_fwd(d, *args, q, nq, k, nk, v, nk, o, nq, lse, ws, n)
            else:
                dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
                B.poetx_attn_bwd(d, *args, g, nq, q, nq, k, nk, v, nk, o, nq, lse, dq, nq, dk, nk, dv, nk, ws, n)
            torch.cuda.synchronize()
            assert (ws[n:] == 0x5A).all()
    for T, V, top in ((1, 131072, 64), (3, 50001, 5), (600, 9000, 0)):
        d = B.logp_desc(V, "bf16", top)
        n = B.poetx_logp_workspace_size(d, T)
        ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        X, t = LP.logits(T, V, "bf16", 1), LP.targets(T, V, 1)
        new = lambda *s, dt=torch.float32: torch.empty(*s, dtype=dt, device="cuda")
        B.poetx_logp_fwd(d, T, X, V, t, new(T), new(T), new(T), new(T, top, dt=torch.int32) if top else None,
                         new(T, top) if top else None, ws, n)
        torch.cuda.synchronize()
        assert (ws[n:] == 0x5A).all()


@pytest.mark.parametrize("hd", [8, 24, 32, 40, 56, 72, 88, 96, 104, 120])
def test_heads_of_a_multiple_of_eight(hd):
    """Copied straight to LDS without the columns behind the head, which hold zeros whatever was there before."""
    nan = torch.full((300, 8 * 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    other = PoetxAttention(8, 8, 128)
    for lq, lk, causal, window in (([1, 130, 300], [1, 130, 300], True, 0), ([5, 260], [300, 100], False, 70),
                                   ([1, 1], [700, 40], True, 0)):
        other.backward(torch.zeros_like(other.forward(nan, nan, nan)))  # not-a-numbers in LDS
        A.run(6, 2, hd, "bf16", lq, lk, causal, window, seed=hd)
    A.run(16, 1, hd, "bf16", [200, 33], [200, 33], seed=1)  # query heads shared among workgroups


def test_heads_of_a_multiple_of_eight_elsewhere():
    """The same heads in rows that are no multiple of 16 bytes, or begin at none: through registers."""
    q, k, v, dO = (A.rows(150, 4 * 40, "bf16", s, 4 * 40 + gap, offset)
                   for s, gap, offset in ((1, 3, 0), (2, 8, 1), (3, 0, 4), (4, 1, 1)))
    at = PoetxAttention(4, 4, 40)
    out = at.forward(q, k, v)
    A.check(at, O.Attn(4, 4, 40, float(np.float32(at.desc.scale)), True), "bf16", (q, k, v), dO, out, at.saved[4],
            at.backward(dO), A.cu_of([150]), A.cu_of([150]))


def test_more_rows_than_a_launch_holds():
    """Rows whose workgroups of one launch would have 2^32 threads and more: every 1024 rows give the same bits."""
    T, n = 2**24 + 1024, 1024
    op, few = PoetxLogProb(3, top=2), PoetxLogProb(3, top=2)
    X, t = LP.logits(n, 3, "bf16", 1), LP.targets(n, 3, 2)
    g, h = (torch.randn(n, device="cuda", generator=torch.Generator("cuda").manual_seed(s)) for s in (3, 4))
    many = lambda x: x.repeat(T // n, *[1] * (x.dim() - 1))
    for a, b in zip(op.forward(many(X), many(t)), few.forward(X, t)):
        assert torch.equal(a.view(T // n, *b.shape), b.expand(T // n, *b.shape))
    dX = few.backward(g, h)
    assert torch.equal(op.backward(many(g), many(h)).view(T // n, n, 3), dX.expand(T // n, n, 3))


def test_more_tokens_than_a_launch_holds():
    rope = PoetxRope(512)  # a workgroup a token
    T, at = 2**22 + 2, [0, 2**22 - 1, 2**22, 2**22 + 1]
    x = A.rows(1, 512, "bf16", 1)
    X = x.expand(T, 512).contiguous()
    rope.forward([X], Ys=[X])
    want = rope.forward([x.expand(4, 512).contiguous()], torch.tensor(at, dtype=torch.int32, device="cuda"))[0]
    assert torch.equal(X[at], want)


@pytest.mark.parametrize("heads,kv,hd,lq,lk,causal,window", [
    (64, 64, 32, [1000], [1000], True, 20),
    (64, 64, 128, [1000], [1000], True, 20),
    (64, 64, 64, [130, 900], [700, 900], True, 0),
    (32, 32, 96, [130, 900], [700, 900], False, 33),
])
def test_waves_with_no_part_in_a_tile(heads, kv, hd, lq, lk, causal, window):
    """Waves that skip the tiles which their rows do not see have copied a share of them all the same."""
    at, mats, dO, out, grads, cu_q, cu_k = A.run(heads, kv, hd, "bf16", lq, lk, causal, window)
    out, grads = out.clone(), [g.clone() for g in grads]
    for _ in range(10):
        assert torch.equal(at.forward(*mats, A.dev(cu_q), A.dev(cu_k)), out)
        assert all(torch.equal(a, b) for a, b in zip(at.backward(dO), grads))


def test_more_joined_rows_than_a_launch_holds():
    """Many short sequences and a long one behind them, whose parts are joined by a second launch."""
    heads, n = 512, 15000
    at = PoetxAttention(heads, heads, 1, causal=False)
    lq, lk = [3] * n + [3], [2] * n + [600]
    q, k, v = (A.rows(sum(x), heads, "bf16", s) for x, s in ((lq, 1), (lk, 2), (lk, 3)))
    dO = A.rows(sum(lq), heads, "bf16", 4)
    out = at.forward(q, k, v, A.dev(A.cu_of(lq)), A.dev(A.cu_of(lk)))
    dQ, dK, dV = at.backward(dO)
    c, lse = O.Attn(heads, heads, 1, float(np.float32(at.desc.scale)), False), at.saved[4]
    for a, b, x, y in ((0, 3, 0, 2), (-3, None, -600, None)):
        A.check(at, c, "bf16", (q[a:b], k[x:y], v[x:y]), dO[a:b], out[a:b], lse[:, a:b], (dQ[a:b], dK[x:y], dV[x:y]),
                A.cu_of([3]), A.cu_of([2 if b else 600]))


@pytest.mark.parametrize("hd", [1, 37, 75, 127])
def test_heads_that_are_laid_out_first(hd):
    """bf16 heads of no multiple of 8 columns over longer sequences: rows outside all sequences (not-a-numbers) stay out of
    it, and a workspace of exactly the bytes asked for holds what the calls write."""
    A.run(6, 2, hd, "bf16", [1, 130, 300], [150, 130, 300], True, 0, seed=hd, first=3, behind=2)
    A.run(4, 4, hd, "bf16", [260, 5], [300, 100], False, 70)
    A.run(16, 1, hd, "bf16", [200, 133], [200, 133], seed=1)  # query heads shared among workgroups
    heads, kv, lens = 6, 2, [130, 300]
    cu = A.dev(A.cu_of(lens, 3))
    T, nq, nk = 435, heads * hd, kv * hd
    q, k, v, g = (A.rows(T, n, "bf16", s) for n, s in ((nq, 1), (nk, 2), (nk, 3), (nq, 4)))
    at = PoetxAttention(heads, kv, hd)
    want = [at.forward(q, k, v, cu)[3:433].clone(), *(x[3:433].clone() for x in at.backward(g))]
    for x in (q, k, v, g):
        x[:3] = x[433:] = float("nan")
    o, lse = torch.zeros_like(q), torch.empty(heads, T, device="cuda")
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    for op in (B.POETX_OP_FWD, B.POETX_OP_BWD):
        n = B.poetx_attn_workspace_size(at.desc, 2, T, T, op)
        ws = torch.full((n + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
        if op == B.POETX_OP_FWD:
            B.poetx_attn_fwd(at.desc, 2, T, T, cu, cu, q, nq, k, nk, v, nk, o, nq, lse, ws, n)
        else:
            B.poetx_attn_bwd(at.desc, 2, T, T, cu, cu, g, nq, q, nq, k, nk, v, nk, o, nq, lse, dq, nq, dk, nk, dv, nk, ws, n)
        torch.cuda.synchronize()
        assert (ws[n:] == 0x5A).all()
    assert all(torch.equal(x[3:433], y) for x, y in zip((o, dq, dk, dv), want))
    assert not any(x[:3].any() or x[433:].any() for x in (o, dq, dk, dv))


def test_heads_that_are_laid_out_first_in_a_graph():
    at = PoetxAttention(6, 2, 37)
    q, k, v, g = (A.rows(430, n * 37, "bf16", s) for n, s in ((6, 1), (2, 2), (2, 3), (6, 4)))
    cu = A.dev(A.cu_of([130, 300]))
    want = [at.forward(q, k, v, cu), *at.backward(g)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [at.forward(q, k, v, cu), *at.backward(g)]
    for _ in range(3):
        for x in got:
            x.fill_(A.MARK)
        got[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
        assert torch.equal(at.forward(q, k, v, cu), want[0])
        at.forward(q, k, v, cu)
