"""Refusals of the attention, on the CPU: the C ABI rejects before any device work (the pointers are never
dereferenced), and layer.PoetxAttention rejects malformed tensors before any library call."""

import ctypes

import pytest
import torch

from orthogonal_reparameterized_cnp_amd import binding as B
from orthogonal_reparameterized_cnp_amd import layer as L

F = 1 << 20
NQ, NK = 4 * 64, 2 * 64


def _d(heads=4, kv=2, hd=64, act="bf16", causal=True, window=0, scale=0.125):
    return B.attn_desc(heads, kv, hd, act, causal, window, scale)


def _fwd(dsc, batch=2, Tq=8, Tk=6, cu_q=F, cu_k=F, Q=2 * F, ldq=NQ, K=3 * F, ldk=NK, V=4 * F, ldv=NK, O=5 * F, ldo=NQ,
         lse=6 * F, ws=7 * F, n=1 << 40):
    return B.lib().poetx_attn_fwd(ctypes.byref(dsc) if dsc else None, batch, Tq, Tk, cu_q, cu_k, Q, ldq, K, ldk, V, ldv, O,
                                  ldo, lse, ws, n, None)


def _bwd(dsc, batch=2, Tq=8, Tk=6, cu_q=F, cu_k=F, dO=8 * F, lddo=NQ, Q=2 * F, ldq=NQ, K=3 * F, ldk=NK, V=4 * F, ldv=NK,
         O=5 * F, ldo=NQ, lse=6 * F, dQ=9 * F, lddq=NQ, dK=10 * F, lddk=NK, dV=11 * F, lddv=NK, ws=7 * F, n=1 << 40):
    return B.lib().poetx_attn_bwd(ctypes.byref(dsc) if dsc else None, batch, Tq, Tk, cu_q, cu_k, dO, lddo, Q, ldq, K, ldk, V,
                                  ldv, O, ldo, lse, dQ, lddq, dK, lddk, dV, lddv, ws, n, None)


def test_descriptor_refusals():
    E, D = B.POETX_E_SHAPE, B.POETX_E_DTYPE
    raw = lambda *a: B.AttnDesc(*a)
    for bad, st in ((raw(0, 1, 64, 1, 1, 0, 1.0), E), (raw(1025, 1, 64, 1, 1, 0, 1.0), E), (raw(4, 0, 64, 1, 1, 0, 1.0), E),
                    (raw(4, 3, 64, 1, 1, 0, 1.0), E), (raw(4, 8, 64, 1, 1, 0, 1.0), E), (raw(4, 2, 0, 1, 1, 0, 1.0), E),
                    (raw(4, 2, 129, 1, 1, 0, 1.0), E), (raw(4, 2, 64, 2, 1, 0, 1.0), D), (raw(4, 2, 64, 1, 2, 0, 1.0), E),
                    (raw(4, 2, 64, 1, 1, -1, 1.0), E), (raw(4, 2, 64, 1, 1, (1 << 30) + 1, 1.0), E),
                    (raw(4, 2, 64, 1, 1, 0, 0.0), E), (raw(4, 2, 64, 1, 1, 0, -1.0), E),
                    (raw(4, 2, 64, 1, 1, 0, float("nan")), E), (raw(4, 2, 64, 1, 1, 0, float("inf")), E),
                    (None, B.POETX_E_NULL)):
        assert _fwd(bad) == st and _bwd(bad) == st
        if bad is not None:
            assert B.poetx_attn_workspace_size(bad, 2, 8, 6, B.POETX_OP_BWD) == 0


def test_size_refusals():
    E = B.POETX_E_SHAPE
    for kw in (dict(batch=0), dict(batch=65537), dict(Tq=-1), dict(Tk=-1), dict(Tq=(1 << 30) + 1), dict(Tk=(1 << 30) + 1),
               dict(cu_q=None, Tq=7), dict(cu_k=None, Tk=5)):
        assert _fwd(_d(), **kw) == E and _bwd(_d(), **kw) == E, kw
    # workgroups beyond a grid's 2^31 - 1
    assert _fwd(_d(1024, 1024, 1), Tq=1 << 30, ldq=1024, ldk=1024, ldv=1024, ldo=1024) == E
    # 64 heads: tiles of 128 rows and one a sequence, below 2^23 in all
    size = lambda Tq, Tk: B.poetx_attn_workspace_size(_d(64, 64, 8), 2, Tq, Tk, B.POETX_OP_BWD)
    most = (2**23 // 64 - 2) * 128 - 128
    assert size(most, most) > 0 and size(most + 256, 8) == 0 and size(8, most + 256) == 0
    assert _fwd(_d(), Tq=0) == B.POETX_OK
    assert _fwd(_d(), Tq=0, cu_q=None, Q=None, O=None, lse=None) == B.POETX_OK
    assert _bwd(_d(), Tq=0, Tk=0) == B.POETX_OK
    assert B.poetx_attn_workspace_size(_d(), 2, 8, 6, B.POETX_OP_MERGE) == 0
    assert B.poetx_attn_workspace_size(_d(), 2, -8, 6, B.POETX_OP_BWD) == 0


def test_operand_refusals():
    for name in ("Q", "K", "V", "O", "lse"):
        assert _fwd(_d(), **{name: None}) == B.POETX_E_NULL, name
    for name in ("dO", "Q", "K", "V", "O", "lse", "dQ", "dK", "dV", "ws"):
        assert _bwd(_d(), **{name: None}) == B.POETX_E_NULL, name
    for kw in (dict(ldq=NQ - 1), dict(ldk=NK - 1), dict(ldv=0), dict(ldo=NQ - 1), dict(Q=2 * F + 1), dict(K=3 * F + 1),
               dict(V=4 * F + 1), dict(O=5 * F + 1), dict(ldq=(1 << 31) + 1)):
        assert _fwd(_d(), **kw) == B.POETX_E_SHAPE and _bwd(_d(), **kw) == B.POETX_E_SHAPE, kw
    for kw in (dict(lddo=1), dict(lddq=NQ - 1), dict(lddk=NK - 1), dict(lddv=-NK), dict(dO=8 * F + 1), dict(dQ=9 * F + 1),
               dict(dK=10 * F + 1), dict(dV=11 * F + 1)):
        assert _bwd(_d(), **kw) == B.POETX_E_SHAPE, kw
    assert _bwd(_d(), n=16) == B.POETX_E_WORKSPACE and _bwd(_d(), ws=7 * F + 8) == B.POETX_E_WORKSPACE


def test_overlap_refusals():
    """Results share no cell with an operand or one another; columns of one buffer share none."""
    row = 2 * NQ
    for O in (2 * F, 2 * F + 2, 3 * F, 4 * F + 2 * NK, 2 * F + 8 * row - 2, 2 * F - 8 * row + 2):
        assert _fwd(_d(), O=O) == B.POETX_E_SHAPE, O
    for name in ("dQ", "dK", "dV"):
        for at in (2 * F, 3 * F, 4 * F, 5 * F, 8 * F):
            assert _bwd(_d(), **{name: at}) == B.POETX_E_SHAPE, (name, at)
    assert _bwd(_d(), dK=9 * F) == B.POETX_E_SHAPE and _bwd(_d(), dV=9 * F + 2) == B.POETX_E_SHAPE
    assert _bwd(_d(), dV=10 * F + 6 * 2 * NK - 2) == B.POETX_E_SHAPE
    # one buffer of rows [dQ | dK | dV], and the same with the columns a cell too near
    fused = NQ + 2 * NK
    kw = dict(lddq=fused, lddk=fused, lddv=fused, dQ=9 * F)
    assert _bwd(_d(), dK=9 * F + 2 * NQ - 2, dV=9 * F + 2 * (NQ + NK), **kw) == B.POETX_E_SHAPE
    assert _bwd(_d(), dK=9 * F + 2 * NQ, dV=9 * F + 2 * (NQ + NK) - 2, **kw) == B.POETX_E_SHAPE
    assert _bwd(_d(), dK=9 * F + 2 * NQ, dV=9 * F + 2 * (NQ + NK) + 2, **kw) == B.POETX_E_SHAPE  # into the next dQ row


bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)


@pytest.fixture
def no_launch(monkeypatch):
    def boom(*a, **k):
        raise AssertionError("a library call was made before the arguments were checked")

    for name in ("poetx_attn_fwd", "poetx_attn_bwd"):
        monkeypatch.setattr(B, name, boom)


def test_layer_rejects(no_launch, monkeypatch):
    for a, msg in (((4, 3, 64), "divide"), ((4, 0, 64), "divide"), ((4, 2, 0), "head_dim"), ((4, 2, 129), "head_dim"),
                   ((4, 2, 64, "i8"), "act")):
        with pytest.raises(ValueError, match=msg):
            L.PoetxAttention(*a, device="cpu")
    at = L.PoetxAttention(4, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="before a forward"):
        at.backward(bf(8, NQ))
    with pytest.raises(ValueError, match="GPU"):
        at.forward(bf(8, NQ), bf(6, NK), bf(6, NK))
    monkeypatch.setattr(L, "_check_device", lambda device, **tensors: None)
    cu = torch.tensor([0, 3, 8], dtype=torch.int32)
    good = (bf(8, NQ), bf(6, NK), bf(6, NK))
    for (Q, K, V), kw, msg in (((bf(8, 64), *good[1:]), {}, "shape"), ((bf(NQ), *good[1:]), {}, "2-D"),
                               ((good[0], bf(NK), good[2]), {}, "2-D"), ((good[0], good[1], bf(5, NK)), {}, "shape"),
                               ((good[0].float(), *good[1:]), {}, "dtype"), (good, dict(cu_k=cu), "without cu_q"),
                               (good, dict(cu_q=cu.long()), "dtype"), (good, dict(cu_q=cu[:1]), "1-D"),
                               (good, dict(cu_q=cu, cu_k=cu[:2]), "one entry"), (good, dict(cu_q=[0, 8]), "1-D"),
                               (good, dict(O=bf(8, 8)), "shape")):
        with pytest.raises(ValueError, match=msg):
            at.forward(Q, K, V, **kw)
    at.saved = (*good, bf(8, NQ), torch.zeros(4, 8), cu, cu, 2)
    for args, kw in (((bf(7, NQ),), {}), ((bf(8, NQ),), dict(dQ=bf(7, NQ))), ((bf(8, NQ),), dict(dK=bf(6, NQ))),
                     ((bf(8, NQ),), dict(dV=bf(6, NK).float()))):
        with pytest.raises(ValueError):
            at.backward(*args, **kw)
