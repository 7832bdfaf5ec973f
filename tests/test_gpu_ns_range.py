"""The orthogonalised updates over operands of differing scale: rows far below or above the others, and matrices whose
norm is far below eps.  Against the definition in 64 bits, rows of each scale judged by their own norm.

Bound.  Values are kept as hi + lo / 2^11, both fp16: to 2^-23 of themselves down to 2^-14 of the scale they are held
at, and to 2^-36 of it (half the smallest step of lo) below.  So a set of rows is off by at most
  * 4 times what the same computation in numpy float32 is off by there, or 16 * 2^-22 of those rows' norm (X, A and B
    rounded once each in 5 steps), and
  * what steps of 2^-36 / SX, SX = 8 sqrt(K) to the nearest power of two, do to X: of n entries 2^-36 / SX sqrt(n), in
    every step, each passed on with at most a = 3.4445 (the slope of p is largest at 0): a geometric sum, 684 for 5.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from orthogonal_reparameterized_cnp_amd import binding as B
from orthogonal_reparameterized_cnp_amd.layer import PoetxOrthogonalizer
from tests.test_gpu_muon import ns32, plain32

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]


def strong_and_noise(rng, n, m):
    r = max(1, min(n, m) // 16)
    return rng.standard_normal((n, r)) @ rng.standard_normal((r, m)) / np.sqrt(r) + 0.7 * rng.standard_normal((n, m))


def check_rows(got, M, hp, sets):
    """Iterates `got` of M (short side first) on the given sets of rows."""
    X = O.ns_iterates(M, hp)[-1]
    p32 = plain32(M, hp)
    sx = 8 * 2.0 ** np.round(np.log2(np.sqrt(max(M.shape))))
    steps = sum(abs(hp.a) ** (k + 1) for k in range(hp.steps))
    for name, rows in sets.items():
        n = np.linalg.norm(X[rows])
        d, off32 = np.linalg.norm((got - X)[rows]), np.linalg.norm((p32 - X)[rows])
        tol = 4 * off32 + 16 * 2.0**-22 * n + steps * 2.0**-36 / sx * np.sqrt(X[rows].size)
        print(f"  {name}: off by {d / n:.2e}, float32 {off32 / n:.2e}, bound {tol / n:.2e}", flush=True)
        assert d <= tol, name


def dense(M):
    hp = ns32()
    G = torch.from_numpy(M).cuda().float()
    out = PoetxOrthogonalizer(*M.shape, "f32")(G)
    torch.cuda.synchronize()
    G64 = G.double().cpu().numpy()
    return out.double().cpu().numpy() / O.ns_scale(*M.shape, hp), G64, hp


def skew(M, eps=1e-7):
    """The orthogonalised skew blocks [count, b, b], from a step that leaves q = -O: lr 1, no momentum, no decay."""
    nb, b, _ = M.shape
    i, j = np.triu_indices(b, 1)
    hp = ns32(eps=eps, rms=0.0)
    g = torch.from_numpy(np.ascontiguousarray(M[:, i, j])).cuda().float()
    q, m = torch.zeros_like(g), torch.zeros_like(g)
    ws = torch.empty(max(256, B.poetx_muon_workspace_size([nb * b], b)), dtype=torch.uint8, device="cuda")
    p = B.muon_params(lr=1.0, beta=0.0, weight_decay=0.0, nesterov=False, rms=0.0, eps=hp.eps)
    B.poetx_muon_step_batch([q], [g], [m], [nb * b], b, p, ws, ws.numel())
    torch.cuda.synchronize()
    out = []
    for a in (-q, g):
        a = a.double().cpu().numpy()
        F = np.zeros(M.shape)
        F[:, i, j], F[:, j, i] = a, -a
        out.append(F)
    return out[0], out[1], hp


@pytest.mark.parametrize("scale", [1e-3, 1e-4, 1e-5, 1e3, 1e4, 1e5])
@pytest.mark.parametrize("rows,cols,n", [(256, 256, 1), (512, 1376, 2), (512, 1376, 64), (100, 300, 5), (2100, 1950, 9)])
def test_rows_of_differing_scale(rows, cols, n, scale):
    print(f"orth {rows}x{cols}, {n} rows at {scale}", flush=True)
    M = strong_and_noise(np.random.default_rng(rows + n), rows, cols)
    sel = np.arange(n) * 3 + 2
    M[sel] *= scale
    got, G, hp = dense(M)
    if rows > cols:  # the scaled rows are columns of the short-side-first matrix: both sets by the whole
        return check_rows(got.T, G.T, hp, {"all": slice(None)})
    rest = np.setdiff1d(np.arange(rows), sel)
    check_rows(got, G, hp, {"all": slice(None), "scaled": sel, "others": rest})


@pytest.mark.parametrize("scale", [1e-3, 1e-5, 1e3, 1e4, 1e5])
@pytest.mark.parametrize("b", [32, 64, 128, 256, 512])
def test_skew_rows_of_differing_scale(b, scale):
    """One row, with its column, of another scale, in one of three blocks."""
    print(f"muon b={b}, a row and its column at {scale}", flush=True)
    rng = np.random.default_rng(b)
    M = np.stack([strong_and_noise(rng, b, b) for _ in range(3)])
    M = M - M.transpose(0, 2, 1)
    M[1, 3] *= scale
    M[1, :, 3] *= scale
    got, G, hp = skew(M)
    rest = np.setdiff1d(np.arange(b), [3])
    for k in range(3):
        check_rows(got[k], G[k], hp, {"all": slice(None), "row": [3], "others": rest})


@pytest.mark.parametrize("norm", [1e-8, 1e-10, 1e-12])
@pytest.mark.parametrize("b", [32, 128, 512])
def test_norms_far_below_eps(b, norm):
    """X_0 = M / (|M|_F + eps) is then far below 1, and so is the update."""
    print(f"muon b={b}, |M| = {norm}", flush=True)
    M = strong_and_noise(np.random.default_rng(b), b, b)
    M = (M - M.T)[None]
    got, G, hp = skew(M * (norm / np.linalg.norm(M)))
    check_rows(got[0], G[0], hp, {"all": slice(None)})
    if b > 32:
        got, G, hp = dense(M[0, : b // 2] * (norm / np.linalg.norm(M)))
        check_rows(got, G, hp, {"all": slice(None)})
