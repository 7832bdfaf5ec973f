"""Log probabilities at the ends of the range: rows whose scaled logits pass it."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from orthogonal_reparameterized_cnp_amd.layer import PoetxLogProb

from . import test_gpu_logp as LP

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]

MOST = float(np.finfo(np.float32).max)


@pytest.mark.parametrize("act", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 20000])
@pytest.mark.parametrize("T", [4, 1100])
def test_rows_whose_scaled_logits_leave_the_range(act, V, T):
    """With a scale of 1.25 rows of the type's lowest value, or with a largest logit near the highest, have a scaled
    maximum outside fp32.  Their lse stays at the end of the range, their log probabilities and entropy are those of the
    differences (within the bounds of test_gpu_logp.py: the exponentials are exact, V / 256 + 88 additions, a logarithm of
    at most log V), and the target's gradient is not lost."""
    op = PoetxLogProb(V, act, top=3, scale=1.25)
    X = LP.logits(T, V, act, 4)
    low, high = torch.finfo(LP.DT[act]).min, 3.0e38
    X[0] = low
    X[1] = float("-inf")
    X[1, 10:90] = low
    X[2, 7], X[2, 200] = high, high
    X[3] = float("-inf")
    t = torch.full((T,), 20, dtype=torch.int32)
    t[2] = 7
    t = t.cuda()
    out = op.forward(X, t)
    assert out.lse[:4].tolist() == [-MOST, -MOST, MOST, float("-inf")]
    n = np.log([V, 80, 2])
    tol = LP.U * (V / 256 + 88 + 8 * n)
    assert (abs(LP.f64(out.logp)[:3] + n) <= tol).all() and (abs(LP.f64(out.entropy)[:3] - n) <= tol * (1 + n)).all()
    assert out.logp[3] == float("-inf") and out.entropy[3] == 0
    assert out.top_ids[[0, 1, 3]].tolist() == [[0, 1, 2], [10, 11, 12], [0, 1, 2]] and out.top_ids[2, :2].tolist() == [7, 200]
    a, b = torch.full((T,), 0.5, device="cuda"), torch.full((T,), -0.25, device="cuda")
    for dent in (None, b):
        dX = op.backward(a, dent)
        assert torch.isfinite(dX).all()
        # p = exp(x - lse) is 0 for a scaled logit under the range: the target's share of 1 / V is lost, its 1 is not
        assert dX[0, 20] == 0.625 and dX[1, 20] == 0.625 and int((dX[:2] != 0).sum()) == 2
        assert not dX[3].any() and not dX[2, :7].any() and not dX[2, 8:200].any() and not dX[2, 201:].any()
    # the same rows with a scale of 1 stay as they are: the lse of row 0 is the logit, in whose digits log V is lost
    one = PoetxLogProb(V, act)
    assert one.forward(X[:1], t[:1]).lse[0] == low
