"""Refusals of arrays beside the matrices (row sums, offsets, targets, upstream gradients) that share a cell with a result,
on the CPU: the C ABI rejects before any device work (the pointers are never dereferenced)."""

from orthogonal_reparameterized_cnp_amd import binding as B

from . import test_attn_checks as A
from . import test_logp_checks as P

F = 1 << 20


def test_attention_forward():
    rows, keys = 8 * 2 * A.NQ, 6 * 2 * A.NK  # bytes of Q and O, of K and V
    for at in (2 * F, 2 * F + rows - 4, 3 * F + keys - 4, 4 * F, 5 * F, 5 * F - 4 * 8 * 4 + 4, 5 * F + rows - 4, F):
        assert A._fwd(A._d(), lse=at) == B.POETX_E_SHAPE, at
    for kw in (dict(cu_q=5 * F + 4), dict(cu_k=5 * F), dict(cu_q=6 * F), dict(cu_k=6 * F + 4 * 8 * 4 - 4)):
        assert A._fwd(A._d(), **kw) == B.POETX_E_SHAPE, kw


def test_attention_backward():
    for name, at in (("dQ", 6 * F), ("dK", 6 * F), ("dV", 6 * F - 4), ("dQ", F), ("dK", F + 2 * 4), ("dV", F)):
        assert A._bwd(A._d(), **{name: at}) == B.POETX_E_SHAPE, (name, at)


def test_log_probabilities():
    E, T = B.POETX_E_SHAPE, 4
    for kw in (dict(lse=F), dict(logp=F + 4), dict(ent=F + 4 * 2000 - 4), dict(lse=3 * F), dict(ent=3 * F + 4), dict(logp=2 * F),
               dict(ent=4 * F + 12), dict(lse=2 * F - 12)):
        assert P._fwd(P._d(), **kw) == E, kw
    top = dict(ids=10 * F, lps=11 * F)
    for kw in (dict(ids=11 * F), dict(ids=11 * F + 4 * 3 * T - 4), dict(lps=3 * F), dict(ids=2 * F - 4), dict(lps=F + 100)):
        assert P._fwd(P._d(top=3), **{**top, **kw}) == E, kw
    for at in (2 * F, 4 * F, 5 * F, 7 * F, 8 * F, 8 * F + 4 * T - 2):
        assert P._bwd(P._d(), dX=at) == E, at


def test_an_array_in_a_gap_shares_nothing():
    """One row sum between the rows of dK, whose pitch leaves 16 bytes: the call goes on to its workspace."""
    kw = dict(batch=1, Tq=1, cu_q=None, cu_k=None, lddk=A.NK + 8, n=16)
    one = A._d(heads=1, kv=1)
    for off, st in ((2 * 64, B.POETX_E_WORKSPACE), (2 * 64 - 4, B.POETX_E_SHAPE), (2 * A.NK + 12, B.POETX_E_WORKSPACE),
                    (2 * A.NK + 16, B.POETX_E_SHAPE), (5 * (2 * A.NK + 16) + 2 * 64, B.POETX_E_WORKSPACE)):
        assert A._bwd(one, lse=10 * F + off, **kw) == st, off
