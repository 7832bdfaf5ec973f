"""Refusals of the norm calls, on the CPU: the C ABI rejects before any device work (the pointers are never
dereferenced), and layer.PoetxNorm rejects malformed tensors before any library call."""

import ctypes

import pytest
import torch

from orthogonal_reparameterized_cnp_amd import binding as B
from orthogonal_reparameterized_cnp_amd import layer as L

FAKE = 1 << 20


def _d(d=64, kind="layer", act="bf16", eps=1e-5):
    return B.norm_desc(d, kind, act, eps)


def _fwd(dsc, T=4, X=FAKE, ldx=64, R=None, ldr=64, w=FAKE, b=None, S=None, lds=64, Y=2 * FAKE, ldy=64, stats=FAKE):
    return B.lib().poetx_norm_fwd(ctypes.byref(dsc) if dsc else None, T, X, ldx, R, ldr, w, b, S, lds, Y, ldy, stats, None)


def _bwd(dsc, T=4, dY=FAKE, lddy=64, S=2 * FAKE, lds=64, stats=FAKE, dS=None, ldds=64, dX=3 * FAKE, lddx=64, dw=FAKE, db=FAKE,
         ws=FAKE, n=1 << 30):
    return B.lib().poetx_norm_bwd(ctypes.byref(dsc) if dsc else None, T, dY, lddy, S, lds, FAKE, stats, dS, ldds, dX, lddx, dw,
                                  db, ws, n, None)


def test_sizes():
    assert B.poetx_norm_stats_bytes(_d(), 10) == 80 and B.poetx_norm_stats_bytes(_d(kind="rms"), 10) == 40
    assert B.poetx_norm_workspace_size(_d(), 0) == 0
    assert B.poetx_norm_workspace_size(_d(), 1) == 2 * 64 * 4 == 2 * B.poetx_norm_workspace_size(_d(kind="rms"), 1)
    assert B.poetx_norm_workspace_size(_d(d=40000), 5) == 0 and B.poetx_norm_stats_bytes(_d(eps=0.0), 5) == 0


def test_descriptor_refusals():
    for bad, st in ((_d(d=0), B.POETX_E_SHAPE), (_d(d=32769), B.POETX_E_SHAPE), (_d(eps=0.0), B.POETX_E_SHAPE),
                    (_d(eps=float("nan")), B.POETX_E_SHAPE), (_d(eps=float("inf")), B.POETX_E_SHAPE),
                    (B.NormDesc(64, 2, B.POETX_BF16, 1e-5), B.POETX_E_SHAPE),
                    (B.NormDesc(64, 0, B.POETX_I8, 1e-5), B.POETX_E_DTYPE), (None, B.POETX_E_NULL)):
        assert _fwd(bad) == st and _bwd(bad) == st
    for T in (-1, (1 << 30) + 1):
        assert _fwd(_d(), T=T) == B.POETX_E_SHAPE and _bwd(_d(), T=T) == B.POETX_E_SHAPE


def test_forward_refusals():
    assert _fwd(_d(), T=0) == B.POETX_OK
    for kw in (dict(X=None), dict(Y=None), dict(stats=None), dict(R=FAKE), dict(S=3 * FAKE)):
        assert _fwd(_d(), **kw) == B.POETX_E_NULL, kw
    for kw in (dict(ldx=63), dict(ldy=63), dict(R=3 * FAKE, S=4 * FAKE, ldr=1), dict(R=3 * FAKE, S=4 * FAKE, lds=0),
               dict(X=FAKE + 1), dict(Y=FAKE), dict(R=2 * FAKE, S=4 * FAKE), dict(R=3 * FAKE, S=2 * FAKE),
               dict(R=3 * FAKE, S=3 * FAKE, lds=65), dict(R=3 * FAKE, S=FAKE, lds=80)):
        assert _fwd(_d(), **kw) == B.POETX_E_SHAPE, kw
    assert _fwd(_d(kind="rms"), b=FAKE) == B.POETX_E_SHAPE


def test_overlap_refusals():
    """Operands that share a cell are refused unless they are one array; rows in each other's gaps share none."""
    apart, row = 16 * FAKE, 64 * 2
    for Y in (FAKE + 2, FAKE - 2, FAKE + 3 * row, FAKE + row * 4 - 2, FAKE - row * 4 + 2):
        assert _fwd(_d(), Y=Y) == B.POETX_E_SHAPE, Y
        assert _fwd(_d(), X=apart, R=FAKE, S=2 * apart, Y=Y) == B.POETX_E_SHAPE, Y
        assert _fwd(_d(), X=apart, R=3 * apart, S=FAKE, Y=Y) == B.POETX_E_SHAPE, Y
        assert _fwd(_d(), X=FAKE, R=apart, S=Y, Y=2 * apart) == B.POETX_E_SHAPE, Y
        assert _fwd(_d(), X=apart, R=FAKE, S=Y, Y=2 * apart) == B.POETX_E_SHAPE, Y
        assert _bwd(_d(), dX=Y) == B.POETX_E_SHAPE, Y
        assert _bwd(_d(), dY=apart, S=FAKE, dX=Y) == B.POETX_E_SHAPE, Y
        assert _bwd(_d(), dY=apart, dS=FAKE, dX=Y) == B.POETX_E_SHAPE, Y
    wide = dict(ldx=200, ldy=200)
    for off in (0, 2, row - 2, 2 * 200 - row + 2, 2 * 200, 3 * 2 * 200 + row - 2):
        assert _fwd(_d(), Y=FAKE + off, **wide) == B.POETX_E_SHAPE, off
    assert _fwd(_d(), Y=FAKE + row, ldx=200, ldy=201) == B.POETX_E_SHAPE


def test_backward_refusals():
    for kw in (dict(dY=None), dict(S=None), dict(stats=None), dict(dX=None), dict(ws=None)):
        assert _bwd(_d(), **kw) == B.POETX_E_NULL, kw
    for kw in (dict(lddy=63), dict(lds=63), dict(lddx=1), dict(dS=4 * FAKE, ldds=63), dict(dX=2 * FAKE),
               dict(dX=FAKE, lddx=65), dict(dS=3 * FAKE, ldds=70), dict(dY=FAKE + 1)):
        assert _bwd(_d(), **kw) == B.POETX_E_SHAPE, kw
    assert _bwd(_d(kind="rms")) == B.POETX_E_SHAPE
    assert _bwd(_d(), n=16) == B.POETX_E_WORKSPACE and _bwd(_d(), ws=FAKE + 8) == B.POETX_E_WORKSPACE


@pytest.fixture
def no_launch(monkeypatch):
    def boom(*a, **k):
        raise AssertionError("a library call was made before the arguments were checked")

    for name in ("poetx_norm_fwd", "poetx_norm_bwd"):
        monkeypatch.setattr(B, name, boom)


bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)


@pytest.mark.parametrize("X, msg", [
    (bf(4, 63), "shape"), (bf(4, 64).float(), "dtype"), (bf(64, 4).t(), "contiguous rows"), (bf(4, 64), "GPU"),
    (bf(64), "2-D"),
])
def test_layer_forward_rejects(no_launch, X, msg):
    with pytest.raises(ValueError, match=msg):
        L.PoetxNorm(64, device="cpu").forward(X)


def test_layer_rejects(no_launch):
    with pytest.raises(ValueError, match="kind"):
        L.PoetxNorm(64, kind="batch", device="cpu")
    with pytest.raises(ValueError, match="act"):
        L.PoetxNorm(64, act="i8", device="cpu")
    n = L.PoetxNorm(64, device="cpu")
    with pytest.raises(ValueError, match="before a forward"):
        n.backward(bf(4, 64))
    n.S, n.stats = bf(8, 64), torch.zeros(2, 8)
    with pytest.raises(ValueError, match="forward of 8"):
        n.backward(bf(4, 64))
    with pytest.raises(ValueError, match="2-D"):
        n.backward(bf(64))
    assert L.PoetxNorm(64, kind="rms", device="cpu").bias is None
