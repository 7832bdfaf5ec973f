"""A step whose blocks take several passes through the workspace."""

from __future__ import annotations

import numpy as np
import pytest
import torch

from orthogonal_reparameterized_cnp_amd import binding as B
from tests.test_gpu_muon import Side, check_step, muon_hp, run_step

pytestmark = [
    pytest.mark.gpu,
    pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU"),
]


def test_blocks_on_either_side_of_every_seam():
    """1400 blocks of 129 do not fit the workspace's 1 GiB and are spread evenly over passes, whose size the workspace
    tells: a block of a pass takes three buffers of 256 x 256 words of 4 bytes, and less than 1 KiB of sums.  Within a
    pass the blocks of the whole rounds of 512 workgroups, 3 tiles of 128 x 128 a block, run on those tiles and the
    others on 64 x 64 ones.  The blocks next to both kinds of seam equal calls of their own."""
    b, nb, last = 129, 1400, 100
    d, L = b * (nb - 1) + last, b * (b - 1) // 2
    size = B.poetx_muon_workspace_size([d], b)
    chunk = size // (3 * 256 * 256 * 4)
    while (chunk + 1) * 3 * 256 * 256 * 4 <= size:
        chunk += 1
    assert nb // 2 <= chunk < nb and size < chunk * (3 * 256 * 256 * 4 + 1024)
    wide = chunk * 3 // 512 * 512 // 3
    places = sorted({k for c in range(0, nb, chunk) for k in (c, c + wide - 1, c + wide, c + chunk - 1) if k < nb} | {nb - 2, nb - 1})
    print(f"passes of {chunk}, {wide} on the wide tiles; blocks {places}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    Q, G, M = (torch.randn(nb, L, device="cuda", generator=g) for _ in range(3))
    q0, g0, m0 = (t[places].clone() for t in (Q, G, M))
    hp = muon_hp()
    whole = Side.__new__(Side)
    whole.d, whole.b, whole.Q, whole.G, whole.M = d, b, Q, G, M
    run_step([whole], b, hp)
    for i, k in enumerate(places):
        one = Side(np.random.default_rng(0), b if k < nb - 1 else last, b)
        one.q, one.g, one.m = (t[i:i + 1].cpu().numpy().copy() for t in (q0, g0, m0))
        one.upload()
        run_step([one], b, hp)
        torch.cuda.synchronize()
        assert torch.equal(one.Q[0], Q[k]) and torch.equal(one.M[0], M[k]), k
        if k < nb - 1:
            check_step(one, hp)
