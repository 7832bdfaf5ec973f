"""The norm with more rows than its grid holds at once, for every thread count of a row: each workgroup then walks
several rows with the next one's loads under way, its sums in alternating buffers, and the column sums over all of them.
The forward holds 8192 rows of up to 512 columns, 2048 of up to 2048, 1024 of up to 4096 (layer norm: of 6145 to 8192
too), 512 of more; the backward 4096, 2048, 1024 and 512 rows of up to 512, 1024, 2048 and 4096 columns, 256 of more.
Every T below leaves a ragged last pass.  Bounds as in test_gpu_norm."""

from __future__ import annotations

import pytest
import torch

from orthogonal_reparameterized_cnp_amd.layer import PoetxNorm
from tests.test_gpu_norm import DT, _rows, check_backward, check_forward

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("T,d", [(8200, 40), (17000, 512), (2500, 1000), (5000, 1376), (2100, 4096), (1100, 5999), (1100, 8000),
                                 (1300, 9000), (700, 13001), (600, 17000)])
def test_more_rows_than_the_grid(T, d, act, kind, res):
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
