"""Accuracy of the orthogonalised updates on matrices that do not average roundings out: sparse, identity-like, of few
rows.  Against the definition in 64 bits.

Bound.  The products are to be as exact as fp32 products: off by at most 4 times what the same computation in numpy
float32 is off by, or by 16 * 2^-22 of the result's norm where that is by chance exact (5 steps round X, A and B once
each to 22 bits or more).  A bf16 result is rounded once, to nearest: rounding is monotone, so that a result within t of
the definition lies between the definition's value - t and + t, both rounded to bf16, and is further from it than the
definition's own rounding by at most 2 t, entry by entry and so in the norm.  No other allowance is made.
"""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O
from orthogonal_reparameterized_cnp_amd.layer import PoetxOrthogonalizer
from tests.test_gpu_muon import ns32, plain32

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]


def tolerance(W, hp):
    """Frobenius bound of the last iterate's error for W, short side first."""
    X = O.ns_iterates(W, hp)[-1]
    return 4 * np.linalg.norm(plain32(W, hp) - X) + 16 * 2.0**-22 * np.linalg.norm(X)


def sparse(shape, places, values):
    M = np.zeros(shape)
    for (i, j), v in zip(places, values):
        M[i, j] = v
    return M


def structured():
    rng = np.random.default_rng(0)
    few = np.zeros((300, 400))
    few[[3, 150, 299]] = rng.standard_normal((3, 400))
    low = rng.standard_normal((1300, 80)) @ rng.standard_normal((80, 1250)) / 9 + 0.7 * rng.standard_normal((1300, 1250))
    return {
        "four entries of 160 x 200": sparse((160, 200), [(3, 4), (9, 50), (77, 99), (150, 180)], [1, 2, -1, 0.5]),
        "three entries of 256 x 256": sparse((256, 256), [(0, 0), (100, 7), (255, 255)], [1.0, 1.25, 0.75]),
        "identity of 129": np.eye(129),
        "a permutation of 200, signed": np.eye(200)[::-1] * np.where(np.arange(200) % 3, 1.0, -1.0),
        "three rows of 300 x 400": few,
        "their transpose": few.T.copy(),
        "low rank and noise 257 x 513": rng.standard_normal((257, 16)) @ rng.standard_normal((16, 513)) / 4
        + 0.7 * rng.standard_normal((257, 513)),
        "low rank and noise 1300 x 1250": low,
    }


@pytest.mark.parametrize("name", list(structured()))
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_structured_matrices(name, dtype):
    print(f"orth {name} {dtype}", flush=True)
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    G = torch.from_numpy(structured()[name]).cuda().to(dt)
    out = PoetxOrthogonalizer(*G.shape, dtype)(G)
    torch.cuda.synchronize()
    G64, got = G.double().cpu().numpy(), out.double().cpu().numpy()
    hp = ns32()
    ref = O.orthogonalize(G64, hp)
    W = G64 if G64.shape[0] <= G64.shape[1] else G64.T
    tol = tolerance(W, hp) * O.ns_scale(*G64.shape, hp)
    rounded = lambda x: torch.from_numpy(x).to(dt).double().numpy()
    n = np.linalg.norm(ref)
    print(f"  off by {np.linalg.norm(got - ref) / n:.2e} of the norm, bound {tol / n:.2e} before the rounding", flush=True)
    assert (rounded(ref - tol) <= got).all() and (got <= rounded(ref + tol)).all()
    # for y within t of x, |RN(y) - y| <= |RN(x) - y| <= |RN(x) - x| + t, so |RN(y) - x| <= |RN(x) - x| + 2 t
    off = np.maximum(np.abs(got - ref) - np.abs(rounded(ref) - ref), 0.0)
    assert np.linalg.norm(off) <= 2 * tol


@pytest.mark.parametrize("count,rows,cols", [(1, 16, 131072), (1, 131072, 5), (1024, 20, 24)])
def test_largest_sizes(count, rows, cols):
    """The longest rows and the largest batch that the call takes; of the batch the first and the last matrix."""
    print(f"orth {count}x{rows}x{cols}", flush=True)
    rng = np.random.default_rng(rows)
    G = torch.from_numpy(rng.standard_normal((count, rows, cols))).cuda().float()
    out = PoetxOrthogonalizer(rows, cols, "f32", count)(G)
    torch.cuda.synchronize()
    hp = ns32()
    for k in sorted({0, count - 1}):
        G64, got = G[k].double().cpu().numpy(), out[k].double().cpu().numpy()
        ref = O.orthogonalize(G64, hp)
        W = G64 if rows <= cols else G64.T
        tol = tolerance(W, hp) * O.ns_scale(rows, cols, hp) + 2.0**-24 * np.linalg.norm(ref)
        d = np.linalg.norm(got - ref)
        print(f"  off by {d / np.linalg.norm(ref):.2e}, bound {tol / np.linalg.norm(ref):.2e}", flush=True)
        assert d <= tol
