"""GPU parity of the orthogonalised updates (poetx_muon_step_batch, poetx_orthogonalize and their layer classes)
against the fp64 oracle.

Bounds, in Frobenius norms.  One step X -> p(X) passes an error on by at most L = max |p'| on [0, |X|_2] (the largest
divided difference of the odd function p on the singular values), and adds the rounding of its own operands and sums:
each of a X, b A X and c A^2 X is off by at most w times |X|_F times the number of rounded factors in it, w the
relative error of a factor with its products and sums: (|a| + 3 |b| s^2 + 5 |c| s^4) w |X|_F with s = |X|_2.
ns_bound() adds these over the oracle's iterates.
  * fp32 and packed parameters: factors of two fp16 planes are off by 2^-22 (11 + 11 bits), the dropped low-by-low
    product by 2^-22, and the fp32 sums of up to 1024 products by less than 2^-22 on the average of their signs:
    w = 3 * 2^-22.
  * bf16: w would be 2^-11, and the worst case says nothing; the same computation is made in float64 with the X, A
    and B factors rounded to fp16 where the kernel rounds them, and the kernel may be 3 times as far from the
    definition as that is, and 2^-8 (half a step) for the final rounding.
Entries are held to the same bound as the norm.  The fp32 bound takes every rounding at its worst; what the calls
promise, products as exact as fp32 products, is checked besides: dense fp32 results are at most 4 times as far from the
definition as the definition computed in numpy float32, or 16 * 2^-22 where that is by chance exact (the 5 steps round
X, A and B once each).
The step of q adds three fp32 roundings of q and of the step: 4 u (|q| + lr |O| + lr wd |q|).
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from orthogonal_reparameterized_cnp_amd import binding as B
from orthogonal_reparameterized_cnp_amd.layer import (PoetxAdam, PoetxGroup, PoetxMuon, PoetxNorm, PoetxOrthogonalizer)
from tests.poetx_cases import TOL, assert_close, dev, errs, host, make_layer, oracle_w
from workloads.gen import custom_linear_inputs

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

U = 2.0**-24
f32 = lambda x: float(np.float32(x))


def ns32(**kw):
    h = O.NsHP(**kw)
    return O.NsHP(h.steps, f32(h.a), f32(h.b), f32(h.c), f32(h.eps), f32(h.rms))


def ns_bound(M, hp, w):
    """Frobenius bound of the error of the last iterate for M (short side first)."""
    err = w * 1.0  # X_0, of norm at most 1
    for X in O.ns_iterates(M, hp)[:-1]:
        s = np.linalg.norm(X, 2) if min(X.shape) > 0 and X.any() else 0.0
        x = np.linspace(0, s, 200)
        L = np.abs(hp.a + 3 * hp.b * x**2 + 5 * hp.c * x**4).max()
        err = L * err + w * (abs(hp.a) + 3 * abs(hp.b) * s**2 + 5 * abs(hp.c) * s**4) * np.linalg.norm(X)
    return err


def emulate_bf16(M, hp):
    """The last iterate with fp16 factors: X in two planes of which the products read the first, A and B in one."""
    h16 = lambda x: x.astype(np.float16).astype(np.float64)
    sx, sa = 8 * 2.0 ** np.round(np.log2(np.sqrt(max(M.shape)))), 256.0
    X = M / (np.linalg.norm(M) + hp.eps) * sx
    X = h16(X) + h16(X - h16(X))
    for _ in range(hp.steps):
        A = h16(h16(X) @ h16(X).T * (sa / sx**2))
        Bm = h16(hp.b * A + hp.c / sa * (A @ A))
        X = hp.a * X + Bm @ h16(X) / sa
        X = h16(X) + h16(X - h16(X))
    return X / sx


def plain32(M, hp):
    """The last iterate computed in float32 throughout, but for the norm."""
    X = (M / (np.linalg.norm(M) + hp.eps)).astype(np.float32)
    a, b, c = (np.float32(x) for x in (hp.a, hp.b, hp.c))
    for _ in range(hp.steps):
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.astype(np.float64)


def packed_skew(rng, nb, b, rank=3):
    """Packed gradients with a few strong directions over noise, as training gives them."""
    i, j = np.triu_indices(b, 1)
    D = rng.standard_normal((nb, b, rank)) @ rng.standard_normal((nb, rank, b)) + 0.5 * rng.standard_normal((nb, b, b))
    return np.ascontiguousarray((D[:, i, j] - D[:, j, i]).astype(np.float32))


class Side:
    def __init__(self, rng, d, b, q_std=0.01):
        self.d, self.b, self.nb, self.L = d, b, -(-d // b), b * (b - 1) // 2
        self.q = (q_std * rng.standard_normal((self.nb, self.L))).astype(np.float32)
        self.g, self.m = packed_skew(rng, self.nb, b), 0.5 * packed_skew(rng, self.nb, b)
        self.dead = np.triu_indices(b, 1)[1] >= d - (self.nb - 1) * b
        for a in (self.q, self.g, self.m):  # marks that no kernel may read or write
            a[-1][self.dead] = np.nan

    def upload(self):
        self.Q, self.G, self.M = (torch.from_numpy(a).cuda() for a in (self.q, self.g, self.m))
        return self


def run_step(sides, b, hp, steps=1, stream=None):
    d = [s.d for s in sides]
    ws = torch.empty(max(256, B.poetx_muon_workspace_size(d, b)), dtype=torch.uint8, device="cuda")
    p = B.muon_params(lr=hp.lr, beta=hp.beta, weight_decay=hp.weight_decay, nesterov=hp.nesterov, steps=hp.ns.steps,
                      a=hp.ns.a, b=hp.ns.b, c=hp.ns.c, eps=hp.ns.eps, rms=hp.ns.rms)
    for _ in range(steps):
        B.poetx_muon_step_batch([s.Q for s in sides], [s.G for s in sides], [s.M for s in sides], d, b, p, ws, ws.numel(),
                                stream)


def check_step(side, hp):
    q, g, m = (a.astype(np.float64) for a in (side.q, side.g, side.m))
    rq, rm = O.muon_step(q, g, m, side.d, side.b, hp)
    got_q, got_m = side.Q.cpu().numpy().astype(np.float64), side.M.cpu().numpy().astype(np.float64)
    i, j = np.triu_indices(side.b, 1)
    worst = 0.0
    for k in range(side.nb):
        live = ~side.dead if k == side.nb - 1 else np.ones(side.L, bool)
        assert np.isnan(got_q[k][~live]).all() and np.isnan(got_m[k][~live]).all(), "an unused slot was written"
        if not live.any():
            continue
        # the momentum: two products and a sum
        tol = 3 * U * (np.abs(hp.beta * m[k]) + np.abs((1 - hp.beta) * g[k]))
        assert (np.abs(got_m[k] - rm[k]) <= tol)[live].all()
        r = min(side.b, side.d - k * side.b)
        _, u = O.muon_update(g[k], m[k], hp)
        Mx = np.zeros((r, r))
        Mx[i[live], j[live]] = u[live]
        Mx -= Mx.T
        scale = O.ns_scale(r, r, hp.ns)
        # u's own roundings are relative to its terms: their norm against |M|
        cond = np.sqrt(2) * np.linalg.norm((np.abs(m[k]) + np.abs(g[k]))[live]) / max(np.linalg.norm(Mx), 1e-300)
        e = ns_bound(Mx, hp.ns, 3 * 2.0**-22 + (6 * U * cond if Mx.any() else 0.0))
        step = np.abs(rq[k] - q[k])
        tol = hp.lr * scale * e + 4 * U * (np.abs(q[k]) + step + hp.lr * abs(hp.weight_decay) * np.abs(q[k]))
        d = np.abs(got_q[k] - rq[k])
        assert np.isfinite(got_q[k][live]).all()
        worst = max(worst, float((d / tol)[live].max()))
        fro = np.linalg.norm(d[live])
        assert fro <= hp.lr * scale * e + np.linalg.norm(tol[live] - hp.lr * scale * e), f"block {k}: {fro:.3e}"
        assert (d <= tol)[live].all(), f"block {k}"
    print(f"  d={side.d} b={side.b}: worst |d| / bound {worst:.3f}", flush=True)


def muon_hp(lr=0.02, beta=0.95, weight_decay=0.1, nesterov=True, **ns):
    return O.MuonHP(f32(lr), f32(beta), f32(weight_decay), nesterov, ns32(**ns))


@pytest.mark.parametrize("dims,b", [
    ([1], 2), ([2, 5, 3], 2), ([7], 5), ([256, 256], 32), ([100, 70, 33], 33), ([64, 1], 64), ([40], 100), ([200, 130], 100),
    ([128], 128), ([300, 129], 129), ([1000, 96], 256), ([1376, 512], 256), ([257], 256), ([700, 1100], 512), ([600], 600),
    ([1024], 1024), ([60], 1024),
])
def test_step_matches_oracle(dims, b):
    print(f"muon dims={dims} b={b}", flush=True)
    rng = np.random.default_rng(b)
    sides = [Side(rng, d, b, q_std=0.0 if k == 1 else 0.01).upload() for k, d in enumerate(dims)]
    hp = muon_hp()
    run_step(sides, b, hp)
    torch.cuda.synchronize()
    for s in sides:
        check_step(s, hp)


@pytest.mark.parametrize("b", [30, 150])
@pytest.mark.parametrize("kw", [dict(nesterov=False), dict(rms=0.0, lr=0.3), dict(steps=1), dict(steps=9), dict(beta=0.0),
                                dict(a=1.875, b=-1.25, c=0.375, steps=12), dict(a=1.5, b=-0.5, c=0.0), dict(lr=0.0)])
def test_parameters(b, kw):
    print(f"muon b={b} {kw}", flush=True)
    side = Side(np.random.default_rng(1), b + 20, b).upload()
    hp = muon_hp(**kw)
    run_step([side], b, hp)
    torch.cuda.synchronize()
    check_step(side, hp)


@pytest.mark.parametrize("b", [32, 96, 256])
def test_blocks_are_independent(b):
    """A zero update leaves O = 0 (decay alone), a NaN stays in its block, extreme scales do not matter, and the
    blocks of a batch get what calls of their own give, bit for bit."""
    rng = np.random.default_rng(2)
    side = Side(rng, 5 * b, b)
    side.g[0] = side.m[0] = 0.0
    side.g[1, 3] = np.nan
    side.g[2] *= np.float32(1e30)
    side.m[2] *= np.float32(1e30)
    side.g[3] *= np.float32(1e-30)
    side.m[3] *= np.float32(1e-30)
    hp = muon_hp(eps=1e-38)
    side.upload()
    run_step([side], b, hp)
    torch.cuda.synchronize()
    q = side.Q.cpu().numpy()
    # O = 0: q - lr (wd q) in at most three roundings (fewer where the compiler fuses a product with its sum), the
    # first two of quantities below lr wd |q|, the last of the result
    q0 = side.q[0].astype(np.float64)
    decay = hp.lr * hp.weight_decay * q0
    assert (np.abs(q[0] - (q0 - decay)) <= U * (2 * np.abs(decay) + np.abs(q0))).all()
    assert np.isnan(q[1]).any() and np.isfinite(q[[0, 2, 3, 4]]).all()
    for k in (2, 3, 4):
        one = Side(rng, b, b)
        one.q, one.g, one.m = (a[k:k + 1].copy() for a in (side.q, side.g, side.m))
        one.upload()
        run_step([one], b, hp)
        torch.cuda.synchronize()
        check_step(one, hp)
        assert np.array_equal(one.Q.cpu().numpy()[0], q[k])


@pytest.mark.parametrize("b", [64, 256])
def test_many_sides_and_repeats(b):
    """64 sides in one call; the same call on the same state gives the same bits."""
    rng = np.random.default_rng(3)
    sides = [Side(rng, 20 + (37 * k) % (2 * b), b) for k in range(64)]
    hp = muon_hp()
    got = []
    for _ in range(2):
        for s in sides:
            s.upload()
        run_step(sides, b, hp, steps=3)
        torch.cuda.synchronize()
        got.append([s.Q.cpu().numpy() for s in sides])
    assert all(np.array_equal(x, y, equal_nan=True) for x, y in zip(*got))
    for s in sides[::9]:
        s.upload()
    run_step(sides[::9], b, hp)
    torch.cuda.synchronize()
    for s in sides[::9]:
        check_step(s, hp)


def test_more_blocks_than_one_chunk():
    """1400 blocks of 129 take two passes through the workspace (1 GiB holds 1365), most of them on the wide tiles;
    blocks on either side of the seam equal calls of their own, and the last one, of 100, its own call and the oracle."""
    b, nb, last = 129, 1400, 100
    d, L = b * (nb - 1) + last, b * (b - 1) // 2
    g = torch.Generator(device="cuda").manual_seed(4)
    Q, G, M = (torch.randn(nb, L, device="cuda", generator=g) for _ in range(3))
    q0, g0, m0 = (t[[0, 700, 1364, 1365, 1398, 1399]].clone() for t in (Q, G, M))
    assert B.poetx_muon_workspace_size([d], b) < 1200 << 20
    hp = muon_hp()
    whole = Side.__new__(Side)
    whole.d, whole.b, whole.Q, whole.G, whole.M = d, b, Q, G, M
    run_step([whole], b, hp)
    for i, k in enumerate([0, 700, 1364, 1365, 1398, 1399]):
        one = Side(np.random.default_rng(0), b if k < nb - 1 else last, b)
        one.q, one.g, one.m = (t[i:i + 1].cpu().numpy().copy() for t in (q0, g0, m0))
        one.upload()
        run_step([one], b, hp)
        torch.cuda.synchronize()
        live = torch.from_numpy(~one.dead).cuda() if k == nb - 1 else slice(None)
        assert torch.equal(one.Q[0], Q[k]) and torch.equal(one.M[0], M[k]), k
        if k == nb - 1:
            assert torch.equal(Q[k][~live], q0[i][~live]) and torch.equal(M[k][~live], m0[i][~live])
            for a in (one.q, one.m):
                a[-1][one.dead] = np.nan
            for t in (one.Q, one.M):
                t[-1][~live] = float("nan")
        check_step(one, hp) if k in (0, nb - 1) else None


def _matrices(rng, count, rows, cols, dtype, pitch=None):
    r = max(1, min(rows, cols) // 8)
    M = rng.standard_normal((count, rows, r)) @ rng.standard_normal((count, r, cols)) / np.sqrt(r)
    M = 1e-3 * (M + 0.7 * rng.standard_normal((count, rows, cols)))
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    buf = torch.full((count, rows + 1, (pitch or cols)), 55.0, dtype=dt, device="cuda")
    buf[:, :rows, :cols].copy_(torch.from_numpy(M))
    return buf[:, :rows, :cols]


def check_orth(G64, got, hp, dtype, name=""):
    ref = O.orthogonalize(G64, hp)
    W = G64 if G64.shape[0] <= G64.shape[1] else G64.T
    scale = O.ns_scale(*G64.shape, hp)
    if dtype == "f32" or W.shape[0] <= 128:
        tol = ns_bound(W, hp, 3 * 2.0**-22) * scale
        if dtype == "f32":
            X = O.ns_iterates(W, hp)[-1]
            off32 = np.linalg.norm(plain32(W, hp) - X)
            tol = min(tol, (4 * off32 + 16 * 2.0**-22 * np.linalg.norm(X)) * scale)
    else:
        X = O.ns_iterates(W, hp)[-1]
        tol = 3 * np.linalg.norm(emulate_bf16(W, hp) - X) * scale
    d, half = np.linalg.norm(got - ref), {"f32": U, "bf16": 2.0**-8}[dtype]
    n = np.linalg.norm(ref)
    print(f"  {name} {G64.shape} {dtype}: off by {d / n if n else d:.2e} of the norm, bound {(tol / n if n else 0) + half:.2e}", flush=True)
    assert np.isfinite(got).all() and d <= tol + half * n
    assert (np.abs(got - ref) <= tol + half * np.abs(ref)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("count,rows,cols", [(1, 1, 1), (1, 1, 1000), (2, 2, 7), (1, 16, 16), (3, 100, 130), (1, 130, 100),
                                             (1, 129, 129), (1, 257, 513), (1, 512, 1376), (2, 1376, 300), (1, 150, 9000)])
def test_orthogonalize_matches_oracle(count, rows, cols, dtype):
    print(f"orth {count}x{rows}x{cols} {dtype}", flush=True)
    G = _matrices(np.random.default_rng(rows + cols), count, rows, cols, dtype)
    hp = ns32()
    before = G.clone()
    out = PoetxOrthogonalizer(rows, cols, dtype, count)(G)
    torch.cuda.synchronize()
    assert torch.equal(G, before) and out.is_contiguous()
    for k in range(count):
        check_orth(G[k].double().cpu().numpy(), out[k].double().cpu().numpy(), hp, dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("count,rows,cols", [(7, 700, 2300), (16, 1024, 1024), (8, 2300, 700), (4, 1950, 2100),
                                             (6, 1000, 1100), (3, 1300, 1250)])
def test_orthogonalize_large_tiles(count, rows, cols, dtype):
    """Enough tiles of 256 x 256 or 128 x 128 for the wide kernels; the first and the last matrix against the oracle."""
    print(f"orth {count}x{rows}x{cols} {dtype}", flush=True)
    G = _matrices(np.random.default_rng(9), count, rows, cols, dtype)
    out = PoetxOrthogonalizer(rows, cols, dtype, count)(G)
    torch.cuda.synchronize()
    for k in (0, count - 1):
        check_orth(G[k].double().cpu().numpy(), out[k].double().cpu().numpy(), ns32(), dtype)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows,cols,pitch", [(90, 200, 207), (200, 90, 91), (300, 400, 401)])
def test_orthogonalize_pitches_and_in_place(rows, cols, pitch, dtype):
    rng = np.random.default_rng(7)
    G = _matrices(rng, 2, rows, cols, dtype, pitch)
    out = _matrices(rng, 2, rows, cols, dtype, pitch + 2)
    o = PoetxOrthogonalizer(rows, cols, dtype, 2)
    ref = o(G.contiguous())
    o(G, out)
    torch.cuda.synchronize()
    assert torch.equal(out, ref)
    gap = out.as_strided((2, rows, pitch + 2 - cols), out.stride(), out.storage_offset() + cols)
    assert (gap == 55.0).all() and (out.as_strided((2, pitch + 2), (out.stride(0), 1), out.storage_offset() + rows * out.stride(1)) == 55.0).all()
    assert o(G, G) is G
    torch.cuda.synchronize()
    assert torch.equal(G, ref)


def test_orthogonalize_degenerate():
    """A zero matrix gives zeros, a NaN stays in its matrix, and no scale overflows."""
    G = _matrices(np.random.default_rng(8), 4, 150, 170, "f32")
    G[0] = 0.0
    G[1, 5, 5] = float("nan")
    G[2] *= 1e36
    G[3] *= 1e-30
    o = PoetxOrthogonalizer(150, 170, "f32", 4)
    o.hp.eps = 1e-38
    out = o(G)
    torch.cuda.synchronize()
    assert not out[0].any() and torch.isnan(out[1]).any() and torch.isfinite(out[2:]).all()
    for k in (2, 3):
        check_orth(G[k].double().cpu().numpy(), out[k].double().cpu().numpy(), ns32(eps=1e-38), "f32")


def _replays(step, outs, before):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    ref = [t.clone() for t in outs]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for k in range(3):
        before()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, ref):
            assert torch.equal(a, b), f"replay {k}"


@pytest.mark.parametrize("b", [32, 256])
def test_step_replays_in_a_graph(b):
    lays = [make_layer(custom_linear_inputs(2 * b, b + b // 2, b, 16, "bf16", "bf16", 0.02, seed=5))]
    opt = PoetxMuon(lays, lr=0.01)
    g = torch.Generator(device="cuda").manual_seed(1)
    dqs = [tuple(torch.randn(q.shape, generator=g, device="cuda") for q in (lays[0].q_R, lays[0].q_P))]
    outs = opt.params() + opt.m
    init = [t.clone() for t in outs]

    def before():
        for t, i in zip(outs, init):
            t.copy_(i)

    _replays(lambda: opt.step(dqs), outs, before)


def test_orthogonalize_replays_in_a_graph_and_on_streams():
    G = _matrices(np.random.default_rng(10), 1, 300, 900, "bf16")[0]
    outs = [torch.empty_like(G) for _ in range(2)]
    os_ = [PoetxOrthogonalizer(300, 900, "bf16") for _ in range(2)]
    _replays(lambda: os_[0](G, outs[0]), [outs[0]], lambda: outs[0].zero_())
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):  # two at once, each with its workspace
        for o, out, s in zip(os_, outs, streams):
            s.wait_stream(torch.cuda.current_stream())
            o(G, out, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1])


def test_merge_cadence():
    """As PoetxAdam: every second step merges, restarts q and the momentum, and leaves the layer usable."""
    lay = make_layer(custom_linear_inputs(96, 80, 32, 64, "bf16", "bf16", 0.02, seed=23))
    opt = PoetxMuon([lay], lr=0.01, merge_every=2)
    X = dev(custom_linear_inputs(96, 80, 32, 64, "bf16", "bf16", 0.02, seed=24).X, "bf16")
    dqs = [(torch.randn_like(lay.q_R), torch.randn_like(lay.q_P))]
    perm = lay.perm_R.clone()
    assert not opt.step(dqs) and opt.m[0].any()
    lay.build()
    Y0 = lay.forward(X).clone()
    q = lay.q_R.clone()
    assert opt.step(dqs)
    torch.cuda.synchronize()
    assert q.any() and not lay.q_R.any() and not any(m.any() for m in opt.m) and not torch.equal(perm, lay.perm_R)
    # the merged layer is the layer after the second step: near the one before it (lr 0.01)
    Y1 = lay.forward(X)
    assert errs(host(Y1, "bf16"), host(Y0, "bf16"))[1] < 0.2


def test_training_step_end_to_end():
    """Norm -> a group of two linears -> their gradients -> the norm's gradient -> Muon on the packed parameters and
    Adam on the norm's weight, against the oracle's chain; the residual's gradient passes the norm."""
    T, d, n, b = 96, 160, (96, 200), 64
    rng = np.random.default_rng(11)
    inps = [custom_linear_inputs(d, k, b, T, "bf16", "bf16", 0.02, seed=30 + i) for i, k in enumerate(n)]
    lays = [make_layer(i) for i in inps]
    group = PoetxGroup(lays, batch_grads=True)
    norm = PoetxNorm(d, "rms", "bf16", eps=1e-5)
    w0 = (1 + 0.2 * rng.standard_normal(d)).astype(np.float32)
    norm.weight.copy_(torch.from_numpy(w0))
    bf = lambda a: torch.from_numpy(a.astype(np.float32)).cuda().bfloat16()
    f64 = lambda t: t.double().cpu().numpy()
    X, R, dS = (bf(rng.standard_normal((T, d))) for _ in range(3))
    opt = PoetxMuon(lays, lr=0.01, weight_decay=0.1)
    m1, m2 = torch.zeros_like(norm.weight), torch.zeros_like(norm.weight)
    q0 = [q.clone() for q in opt.params()]

    group.build()
    Y, S = norm.forward(X, R)
    Zs = group.forward([0, 1], [Y, Y])
    dZs = [dev(i.dZ, "bf16") for i in inps]
    dY = torch.empty_like(Y)
    group.backward_dx_many([0, 1], dZs, [dY, dY])
    dqs = group.backward_q()
    dX, dw, _ = norm.backward(dY, dS)
    assert not opt.step(dqs)
    B.poetx_adam_step_batch([norm.weight], [dw], [m1], [m2], 1e-3, 0.9, 0.99, 1e-3, 0.0, 1)
    torch.cuda.synchronize()

    S64 = f64(S)
    Y64, mean, rs = O.norm_forward(S64, w0.astype(np.float64), None, "rms", f32(1e-5))
    assert_close("Y", f64(Y), Y64, "bf16")
    dY64 = np.zeros((T, d))
    for k, inp in enumerate(inps):
        g = O.backward(f64(Y), O.to_f64(inp.dZ, "bf16"), oracle_w(inp), inp.perm_R, inp.perm_P, inp.q_R.astype(np.float64),
                       inp.q_P.astype(np.float64), b)
        dY64 += g.dX
        assert_close(f"dq_R {k}", f64(dqs[k][0]), g.dq_R, "bf16")
        assert_close(f"dq_P {k}", f64(dqs[k][1]), g.dq_P, "bf16")
    assert_close("dY", f64(dY), dY64, "bf16")
    dS64, dw64, _ = O.norm_backward(S64, f64(dY), w0.astype(np.float64), mean, rs, "rms")
    assert_close("dX", f64(dX), dS64 + f64(dS), "bf16")
    assert_close("dw", f64(dw), dw64, "f32")
    # the optimiser on the kernel's own gradients: the bounds of the single step
    hp = muon_hp(lr=0.01, weight_decay=0.1)
    for i, (q, dq, dd) in enumerate(zip(q0, [x for p in dqs for x in p], opt.d)):
        s = Side(rng, dd, b)
        s.q, s.g, s.m = (a.cpu().numpy().copy() for a in (q, dq, torch.zeros_like(q)))
        s.Q, s.M = opt.params()[i].clone(), opt.m[i].clone()
        for a in (s.q, s.m):
            a[-1][s.dead] = np.nan
        for t in (s.Q, s.M):
            t[-1][torch.from_numpy(s.dead)] = float("nan")
        check_step(s, hp)
    w1, _, _ = O.adam_step(w0.astype(np.float64), f64(dw), 0.0, 0.0, 1, O.AdamHP(*(f32(x) for x in (1e-3, 0.9, 0.99, 1e-3, 0.0))))
    np.testing.assert_allclose(f64(norm.weight), w1, rtol=2e-6)


def test_orthogonalize_between_its_operands():
    """G and O as the halves of one array, matrix by matrix: the results of separate arrays, bit for bit."""
    count, rows, cols = 3, 100, 130
    G = _matrices(np.random.default_rng(5), count, rows, cols, "f32")
    op = PoetxOrthogonalizer(rows, cols, "f32", count)
    want = op(G)
    both = torch.stack([G, torch.zeros_like(G)], 1)
    assert torch.equal(op(both[:, 0], out=both[:, 1]), want) and torch.equal(both[:, 0], G)
    wide = torch.cat([G, torch.zeros_like(G)], 2)
    assert torch.equal(op(wide[:, :, :cols], out=wide[:, :, cols:]), want) and torch.equal(wide[:, :, :cols], G)
