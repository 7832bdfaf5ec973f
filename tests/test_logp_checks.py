"""Refusals of the log probabilities, on the CPU: the C ABI rejects before any device work (the pointers are never
dereferenced), and layer.PoetxLogProb rejects malformed tensors before any library call."""

import ctypes

import pytest
import torch

from orthogonal_reparameterized_cnp_amd import binding as B
from orthogonal_reparameterized_cnp_amd import layer as L

F = 1 << 20


def _d(V=1000, act="bf16", top=0, scale=1.0):
    return B.logp_desc(V, act, top, scale)


def _fwd(dsc, T=4, X=F, ldx=1000, target=2 * F, logp=3 * F, lse=4 * F, ent=5 * F, ids=None, lps=None, ws=6 * F, n=1 << 40):
    return B.lib().poetx_logp_fwd(ctypes.byref(dsc) if dsc else None, T, X, ldx, target, logp, lse, ent, ids, lps, ws, n, None)


def _bwd(dsc, T=4, X=F, ldx=1000, target=2 * F, lse=4 * F, ent=5 * F, dlogp=7 * F, dent=8 * F, dX=9 * F, lddx=1000):
    return B.lib().poetx_logp_bwd(ctypes.byref(dsc) if dsc else None, T, X, ldx, target, lse, ent, dlogp, dent, dX, lddx, None)


def test_descriptor_refusals():
    E = B.POETX_E_SHAPE
    for bad, st in ((B.LogpDesc(0, 1, 0, 1.0), E), (B.LogpDesc((1 << 20) + 1, 1, 0, 1.0), E),
                    (B.LogpDesc(9, 2, 0, 1.0), B.POETX_E_DTYPE), (B.LogpDesc(9, 1, -1, 1.0), E),
                    (B.LogpDesc(9, 1, 10, 1.0), E), (B.LogpDesc(100, 1, 65, 1.0), E), (B.LogpDesc(9, 1, 0, 0.0), E),
                    (B.LogpDesc(9, 1, 0, -1.0), E), (B.LogpDesc(9, 1, 0, float("nan")), E),
                    (B.LogpDesc(9, 1, 0, float("inf")), E), (None, B.POETX_E_NULL)):
        assert _fwd(bad) == st and _bwd(bad) == st
        if bad is not None:
            assert B.poetx_logp_workspace_size(bad, 5) == 0
    for T in (-1, (1 << 30) + 1):
        assert _fwd(_d(), T=T) == E and _bwd(_d(), T=T) == E
    assert _fwd(_d(), T=0) == B.POETX_OK and _bwd(_d(), T=0) == B.POETX_OK


def test_operand_refusals():
    N, E = B.POETX_E_NULL, B.POETX_E_SHAPE
    for kw in (dict(X=None), dict(lse=None), dict(target=None), dict(logp=None), dict(ids=F)):
        assert _fwd(_d(), **kw) == N, kw
    for kw in (dict(), dict(ids=F), dict(lps=F)):
        assert _fwd(_d(top=3), **kw) == N, kw
    for kw in (dict(X=None), dict(lse=None), dict(target=None), dict(dlogp=None), dict(ent=None), dict(dX=None)):
        assert _bwd(_d(), **kw) == N, kw
    for kw in (dict(ldx=999), dict(X=F + 1), dict(ldx=(1 << 31) + 1)):
        assert _fwd(_d(), **kw) == E and _bwd(_d(), **kw) == E, kw
    for kw in (dict(lddx=999), dict(dX=9 * F + 1), dict(dX=F, lddx=1001), dict(dX=F + 2), dict(dX=F + 3 * 2000),
               dict(dX=F - 2000 * 4 + 2)):
        assert _bwd(_d(), **kw) == E, kw
    need = B.poetx_logp_workspace_size(_d(V=100000), 1)
    assert need > 0 and B.poetx_logp_workspace_size(_d(V=100000, top=5), 1) > need
    assert _fwd(_d(V=100000), T=1, ldx=100000, n=need - 1) == B.POETX_E_WORKSPACE
    assert _fwd(_d(V=100000), T=1, ldx=100000, ws=6 * F + 8) == B.POETX_E_WORKSPACE
    assert _fwd(_d(V=100000), T=1, ldx=100000, ws=None) == N
    assert B.poetx_logp_workspace_size(_d(), 0) == 0 == B.poetx_logp_workspace_size(_d(V=100), 5000)


bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)
i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)


def test_layer_rejects(monkeypatch):
    def boom(*a, **k):
        raise AssertionError("a library call was made before the arguments were checked")

    for name in ("poetx_logp_fwd", "poetx_logp_bwd"):
        monkeypatch.setattr(B, name, boom)
    for a, msg in (((9, "i8"), "act"), ((9, "bf16", 10), "top"), ((100, "bf16", 65), "top"), ((9, "bf16", -1), "top")):
        with pytest.raises(ValueError, match=msg):
            L.PoetxLogProb(*a, device="cpu")
    p = L.PoetxLogProb(9, device="cpu")
    with pytest.raises(ValueError, match="before a forward"):
        p.backward()
    with pytest.raises(ValueError, match="GPU"):
        p.forward(bf(4, 9))
    monkeypatch.setattr(L, "_check_device", lambda device, **tensors: None)
    for X, t, msg in ((bf(9), None, "2-D"), (bf(4, 8), None, "shape"), (bf(4, 9).float(), None, "dtype"),
                      (bf(9, 4).t(), None, "contiguous rows"), (bf(4, 9), i32(3), "shape"), (bf(4, 9), i32(4).long(), "dtype")):
        with pytest.raises(ValueError, match=msg):
            p.forward(X, t)
    p.saved = (bf(4, 9), None, torch.zeros(4), torch.zeros(4))
    with pytest.raises(ValueError, match="no targets"):
        p.backward(torch.zeros(4))
    for kw in (dict(dentropy=torch.zeros(3)), dict(dentropy=torch.zeros(4).double()), dict(dX=bf(4, 8))):
        with pytest.raises(ValueError):
            p.backward(**kw)
