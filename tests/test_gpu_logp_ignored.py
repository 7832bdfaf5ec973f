"""The gradient of rows whose target asks for nothing, whatever the row holds (the padding of a batch)."""

from __future__ import annotations

import pytest
import torch

from orthogonal_reparameterized_cnp_amd.layer import PoetxLogProb

from . import test_gpu_logp as LP

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(6, 5001), (1200, 300)])
def test_ignored_rows_have_no_gradient(act, T, V):
    op = PoetxLogProb(V, act)
    X = LP.logits(T, V, act, 1)
    X[0], X[1, 17], X[2, 4], X[3, 9] = float("nan"), float("inf"), float("nan"), float("nan")
    t = torch.zeros(T, dtype=torch.int32)
    t[0], t[1], t[2] = -1, V, -100
    t = t.cuda()
    a = torch.full((T,), 0.5, device="cuda")
    a[0] = float("nan")  # not asked for either
    out = op.forward(X, t)
    assert out.logp[:3].tolist() == [0, 0, 0] and torch.isnan(out.logp[3])
    dX = op.backward(a)
    assert not dX[:3].any() and torch.isnan(dX[3]).all() and torch.isfinite(dX[4:]).all() and dX[4:].any()
    # the entropy of these rows is asked for where its gradient is given
    dX = op.backward(a, torch.ones(T, device="cuda"))
    assert torch.isnan(dX[:4]).all() and torch.isfinite(dX[4:]).all()
    # no targets at all
    op.forward(X)
    assert not op.backward().any()


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("T,V", [(6, 5001), (1200, 300)])
def test_rows_of_no_upstream_gradient_have_none(act, T, V):
    """Padding that is masked in the loss: upstream gradients of 0, with targets like any others."""
    op = PoetxLogProb(V, act)
    X, t = LP.logits(T, V, act, 2), torch.zeros(T, dtype=torch.int32, device="cuda")
    a, b = torch.full((T,), 0.5, device="cuda"), torch.full((T,), 0.25, device="cuda")
    a[:3], b[:3] = 0, 0
    a[1], t[2] = -0.0, -1
    op.forward(X, t)
    want, only = op.backward(a, b), op.backward(None, b)
    Y = X.clone()
    Y[0], Y[1, 5], Y[2, 7] = float("nan"), float("inf"), float("nan")
    op.forward(Y, t)
    for dX, ref in ((op.backward(a, b), want), (op.backward(None, b), only)):
        assert not dX[:3].any() and torch.equal(dX[3:], ref[3:]) and ref[3:].any() and torch.isfinite(ref).all()
