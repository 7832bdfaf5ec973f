"""Offsets that break their contract (they decrease, or lie outside the rows): the results of their sequences are no
one's, but every access stays within the rows and the workspace, other rows keep what they hold, and the next call is
right."""

import numpy as np
import pytest
import torch

from orthogonal_reparameterized_cnp_amd.layer import PoetxAttention

from . import test_gpu_attention as A

DECREASING = [0, 58, 1, 2, 60]


def _sequence_and_row(cu_q, rows, i):
    """What the join of the forward of few rows takes row i for: the sequence that it finds, and its row there.  (Up to 64
    sequences are counted at once: as many as begin at or before i.)"""
    first = np.clip(np.array(cu_q), 0, rows)
    s = max(int((first[:-1] <= i).sum()) - 1, 0)
    return s, i - int(first[s]), max(int(first[s + 1] - first[s]), 0)


def test_the_offsets_below_reach_it():
    """Some row of the decreasing offsets below is taken for one of a sequence that does not hold it."""
    found = [_sequence_and_row(DECREASING, 60, i) for i in range(60)]
    assert any(row < 0 or row >= n for _, row, n in found)
    assert min(row for _, row, _ in found) < -40


@pytest.mark.gpu
@pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")
@pytest.mark.parametrize("act", ["f32", "bf16"])
def test_decreasing_offsets_stay_within_their_buffers(act):
    heads, kv, hd = 2, 1, 64
    at = PoetxAttention(heads, kv, hd, act)
    mats = [A.rows(62, heads * hd, act, 1), A.rows(4000, kv * hd, act, 2), A.rows(4000, kv * hd, act, 3)]
    out = torch.full((62, heads * hd), A.MARK, dtype=A.DT[act], device="cuda")
    print(f"decreasing offsets {act}", flush=True)
    at.forward(*mats, A.dev(DECREASING), A.dev([0, 1500, 1500, 3000, 4000]), O=out)
    torch.cuda.synchronize()
    assert (out[60:] == A.MARK).all()
    print("offsets outside the rows", flush=True)
    at.forward(*mats, A.dev([-5, 1, 2, 3, 1 << 30]), A.dev([-(1 << 30), 1500, 1500, 3000, 1 << 30]), O=out)
    torch.cuda.synchronize()
    A.run(heads, kv, hd, act, [1, 1, 1, 1], [1500, 0, 1500, 1000])
