"""Refusals of the orthogonalised updates, on the CPU: the C ABI rejects before any device work (the pointers are
never dereferenced), and the layer classes reject malformed tensors before any library call."""

import ctypes

import pytest
import torch

from orthogonal_reparameterized_cnp_amd import binding as B
from orthogonal_reparameterized_cnp_amd import layer as L

FAKE = 1 << 20


def _pp(*ptrs):
    return (ctypes.c_void_p * len(ptrs))(*ptrs)


def _ii(*xs):
    return (ctypes.c_int32 * len(xs))(*xs)


def _hp(lr=1e-3, **kw):
    return B.muon_params(lr=lr, **kw)


MB = 1 << 20  # more than one of these arrays holds


def _step(n=2, q=_pp(FAKE, 2 * MB), dq=_pp(3 * MB, 3 * MB), m=_pp(5 * MB, 6 * MB), d=_ii(300, 200), b=256, hp=None, ws=FAKE, size=1 << 40):
    hp = _hp() if hp is None else hp
    return B.lib().poetx_muon_step_batch(n, q, dq, m, d, b, ctypes.byref(hp) if hp else None, ws, size, None)


def _orth(count=1, rows=100, cols=200, dt=B.POETX_F32, G=FAKE, ldg=200, sg=20000, O=2 * FAKE, ldo=200, so=20000, hp=None, ws=FAKE,
          size=1 << 40):
    hp = B.ns_params() if hp is None else hp
    return B.lib().poetx_orthogonalize(count, rows, cols, dt, G, ldg, sg, O, ldo, so, ctypes.byref(hp) if hp else None, ws, size,
                                       None)


BAD_NS = [dict(steps=0), dict(steps=21), dict(a=float("nan")), dict(b=float("inf")), dict(c=float("nan")), dict(eps=0.0),
          dict(eps=float("nan")), dict(rms=-0.1), dict(rms=float("inf")),
          dict(a=5.0, b=0.0, c=0.0),  # 5 x: leaves the range in the first step
          dict(a=3.0, b=0.0, c=0.0, steps=2),  # 3, then 9
          dict(a=1.0, b=-300.0, c=300.0),  # terms beyond fp16 even where they cancel
          dict(a=3.4445, b=-4.775, c=8.0)]


def test_workspace_sizes():
    assert B.poetx_muon_workspace_size([256, 256], 128) == 0 == B.poetx_muon_workspace_size([256], 1)
    assert B.poetx_muon_workspace_size([256], 2000) == 0 and B.poetx_muon_workspace_size([0], 256) == 0
    one, two = B.poetx_muon_workspace_size([256], 256), B.poetx_muon_workspace_size([256, 200], 256)
    assert two > one >= 3 * 2 * 256 * 256 * 2
    assert B.poetx_muon_workspace_size([129], 129) == one  # padded to whole tiles
    assert B.poetx_orthogonalize_workspace_size(1, 100, 200, B.POETX_F32) == B.poetx_orthogonalize_workspace_size(1, 200, 100, B.POETX_F32) > 0
    assert B.poetx_orthogonalize_workspace_size(1, 1024, 2048, B.POETX_F32) > B.poetx_orthogonalize_workspace_size(1, 1024, 2048, B.POETX_BF16)
    for bad in ((0, 10, 10, 0), (1025, 10, 10, 0), (1, 0, 10, 0), (1, 10, (1 << 17) + 1, 0), (1, 10, 10, B.POETX_I8), (1024, 1 << 17, 1 << 17, 0)):
        assert B.poetx_orthogonalize_workspace_size(*bad) == 0, bad


def test_step_refusals():
    for kw in (dict(q=None), dict(dq=None), dict(m=None), dict(hp=False), dict(d=None), dict(q=_pp(FAKE, None)),
               dict(dq=_pp(None, FAKE)), dict(m=_pp(5 * MB, None)), dict(ws=None)):
        assert _step(**kw) == B.POETX_E_NULL, kw
    for kw in (dict(n=0), dict(n=65), dict(b=1), dict(b=1025), dict(d=_ii(0, 5)), dict(d=_ii(5, (1 << 20) + 1)),
               dict(hp=_hp(lr=-1.0)), dict(hp=_hp(lr=float("nan"))), dict(hp=_hp(beta=1.0)), dict(hp=_hp(beta=-0.1)),
               dict(hp=_hp(weight_decay=float("inf")))):
        assert _step(**kw) == B.POETX_E_SHAPE, kw
    bad = _hp()
    bad.nesterov = 2
    assert _step(hp=bad) == B.POETX_E_SHAPE
    for ns in BAD_NS:
        assert _step(hp=_hp(**ns)) == B.POETX_E_SHAPE, ns
    assert _step(size=16) == B.POETX_E_WORKSPACE and _step(ws=FAKE + 8) == B.POETX_E_WORKSPACE


def test_step_refuses_arrays_that_overlap():
    """b = 4: a side of 8 holds 2 blocks of 6 slots, 48 bytes."""
    hp = _hp(lr=-1.0)  # checked before the arrays: a call that passes the array check would end as this does
    A = FAKE
    call = lambda q, dq, m: _step(2, _pp(*q), _pp(*dq), _pp(*m), _ii(8, 8), 4)
    for q, dq, m in (((A, A), (A + 800, A + 900), (A + 1000, A + 1100)),  # one side twice
                     ((A, A + 44), (A + 800, A + 900), (A + 1000, A + 1100)),
                     ((A, A + 48), (A + 800, A + 900), (A + 95, A + 1100)),  # m into q
                     ((A, A + 48), (A + 40, A + 900), (A + 1000, A + 1100)),  # dq in q
                     ((A, A + 48), (A + 800, A + 1140), (A + 1000, A + 1100))):
        assert call(q, dq, m) == B.POETX_E_SHAPE and "overlap" in B.poetx_last_error()
    assert _step(hp=hp) == B.POETX_E_SHAPE and "lr" in B.poetx_last_error()
    # side by side, and one gradient for both: past the array check (the workspace is what is wrong)
    assert _step(2, _pp(A, A + 40 * MB), _pp(A + 10 * MB, A + 10 * MB), _pp(A + 20 * MB, A + 30 * MB), _ii(300, 300), 256,
                 size=16) == B.POETX_E_WORKSPACE


def test_orthogonalize_refusals():
    for kw in (dict(G=None), dict(O=None), dict(hp=False), dict(ws=None)):
        assert _orth(**kw) == B.POETX_E_NULL, kw
    for kw in (dict(count=0), dict(rows=0), dict(cols=0), dict(rows=(1 << 17) + 1), dict(ldg=199), dict(ldo=1),
               dict(count=2, sg=19999), dict(count=2, so=0), dict(O=FAKE, ldo=201), dict(count=2, O=FAKE, so=20001),
               dict(G=FAKE + 2), dict(count=1024, rows=1 << 17, cols=1 << 17, ldg=1 << 17, ldo=1 << 17)):
        assert _orth(**kw) == B.POETX_E_SHAPE, kw
    # arrays that share a cell: rows 100 x 200 fp32, in one piece, with gaps, and in a batch
    for O in (FAKE + 4, FAKE - 4, FAKE + 80000 - 4, FAKE - 80000 + 4):
        assert _orth(O=O) == B.POETX_E_SHAPE, O
    for off in (4, 796, 1200 * 4 - 796, 99 * 1200 * 4 + 796):
        assert _orth(O=FAKE + off, ldg=1200, ldo=1200) == B.POETX_E_SHAPE, off
    for off in (80000 - 4, 160000, 240000 - 4, 160000 + 80000 - 4, 320000 + 80000 - 4):
        assert _orth(count=3, O=FAKE + off, sg=40000, so=40000) == B.POETX_E_SHAPE, off
    assert _orth(dt=B.POETX_I8) == B.POETX_E_DTYPE
    for ns in BAD_NS:
        assert _orth(hp=B.ns_params(**ns)) == B.POETX_E_SHAPE, ns
    assert _orth(size=16) == B.POETX_E_WORKSPACE and _orth(ws=FAKE + 128) == B.POETX_E_WORKSPACE


@pytest.fixture
def no_launch(monkeypatch):
    def boom(*a, **k):
        raise AssertionError("a library call was made before the arguments were checked")

    for name in ("poetx_muon_step_batch", "poetx_orthogonalize"):
        monkeypatch.setattr(B, name, boom)


def test_classes_reject(no_launch):
    with pytest.raises(ValueError, match="no linears"):
        L.PoetxMuon([])
    lay = L.PoetxLinear(96, 80, 32, device="cpu")
    opt = L.PoetxMuon([lay])
    with pytest.raises(ValueError, match="pair"):
        opt.step([])
    with pytest.raises(ValueError, match="shape"):
        opt.step([(lay.q_R[:1], lay.q_P)])
    with pytest.raises(ValueError, match="dtype"):
        opt.step([(lay.q_R.double(), lay.q_P)])
    with pytest.raises(ValueError, match="GPU"):
        opt.step([(lay.q_R, lay.q_P)])
    with pytest.raises(ValueError, match="dtype"):
        L.PoetxOrthogonalizer(10, 20, "i8", device="cpu")
    with pytest.raises(ValueError, match="rows and cols"):
        L.PoetxOrthogonalizer(0, 20, device="cpu")
    o = L.PoetxOrthogonalizer(10, 20, device="cpu")
    for G, msg in ((torch.zeros(20, 10), "shape"), (torch.zeros(10, 20).double(), "dtype"), (torch.zeros(20, 10).t(), "contiguous rows"),
                   (torch.zeros(10, 20), "GPU"), (torch.zeros(2, 10, 20), "shape")):
        with pytest.raises(ValueError, match=msg):
            o(G)


def test_sides_are_grouped_by_block_size():
    lays = [L.PoetxLinear(64, 64, b, device="cpu") for b in (32, 16, 32)] + [L.PoetxLinear(8, 8, 8, device="cpu") for _ in range(40)]
    opt = L.PoetxMuon(lays)
    assert [(b, len(i)) for b, i in opt.calls] == [(8, 64), (8, 16), (16, 2), (32, 4)]
    assert sorted(i for _, idx in opt.calls for i in idx) == list(range(86))
    assert all(opt.layers[i // 2].b == b for b, idx in opt.calls for i in idx)
