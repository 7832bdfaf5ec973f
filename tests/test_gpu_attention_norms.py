"""How far bf16 attention is off in the norm, sequence by sequence, against what its roundings are expected to cost.

The bounds of tests/test_gpu_attention.py hold for every element and grow with the number of terms: among many alike a
missing one stays inside.  Here every rounding counts with its expected square, half a step squared over three (a value
anywhere between two neighbours), and different ones as independent: they add up as squares.  Rounded are
  * the results themselves;
  * p as the operand of O and dV (in the forward relative to a maximum that is not the last one, so that the step is taken
    as 2^-7 of p, its largest; where the row sees one key p is 1 and exact, which only helps);
  * p (dO v - D) as the operand of dK, and of dQ in tiles of keys that no mask cuts.  (In the others dQ's product takes what
    the rounding left as well; here they count alike.)
fp32 sums are 2^-12 of that.  A norm of some 10^4 independent errors stays within 10% of its expectation by far; a missing
key or query of 700 is ten times as far away."""

from __future__ import annotations

import numpy as np
import pytest
import torch

import oracle as O

from . import test_gpu_attention as A

MARGIN = 1.1
gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
t = lambda x: x.transpose(0, 2, 1)


def step(x):
    """bf16's step at x."""
    return np.where(x == 0, 0.0, 2.0 ** (np.floor(np.log2(np.maximum(abs(x), 1e-300))) - 7))


def square(x):
    """The expected square of what rounding x to bf16 changes."""
    return step(x) ** 2 / 12


def bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16).double().numpy()


class Terms:
    """What one sequence's gradients are formed of, from its rows in fp64."""

    def __init__(self, c, Q, K, V, dO, out, lse):
        cu_q, cu_k = np.array([0, len(Q)]), np.array([0, len(K)])
        self.c = c
        ((self.q, self.k, self.x),) = c.scores(Q, K, cu_q, cu_k)
        (self.v,), (self.do,), (self.o,) = c.split(V, cu_k, c.kv_heads), c.split(dO, cu_q, c.heads), c.split(out, cu_q, c.heads)
        self.l = np.where(np.isneginf(lse), 0.0, lse)[..., None]
        self.p = np.exp(self.x - self.l)
        self.dp = self.do @ t(self.v) - (self.do * self.o).sum(2, keepdims=True)
        self.g = self.p * self.dp

    def fold(self, x):
        return self.c.join(x.reshape(self.c.kv_heads, -1, *x.shape[1:]).sum(1))

    def results(self, p=None, g=None):
        """O, dQ, dK, dV with the given p and g as operands."""
        p, g, s = self.p if p is None else p, self.g if g is None else g, self.c.scale
        return self.c.join(p @ self.v), self.c.join(s * (g @ self.k)), self.fold(s * (t(g) @ self.q)), self.fold(t(p) @ self.do)

    def expected(self):
        """The squares that the operands' roundings are expected to add to O, dQ, dK and dV."""
        s2 = self.c.scale**2
        return (self.c.join((self.p * 2.0**-7) ** 2 / 12 @ self.v**2), self.c.join(s2 * (square(self.g) @ self.k**2)),
                self.fold(s2 * (t(square(self.g)) @ self.q**2)), self.fold(t(square(self.p)) @ self.do**2))


def check_norms(terms, got):
    for name, y, ref, add in zip(("O", "dQ", "dK", "dV"), got, terms.results(), terms.expected()):
        off, bound = np.linalg.norm(y - ref), np.sqrt((add + square(ref)).sum())
        print(f"  {name}: {off / np.linalg.norm(ref):.2e} of the norm, {off / bound:.3f} of what is expected", flush=True)
        assert off <= MARGIN * bound, f"{name}: {off / np.linalg.norm(ref):.2e} of the norm off, expected {bound / np.linalg.norm(ref):.2e}"


def check_dq_of_cut_tiles(terms, dQ):
    """With the rest of the rounding multiplied too, dQ before its own rounding is off by e, at most that of the sums in
    tests/test_gpu_attention.py with a rounding of 2^-16.  It then rounds to another neighbour than the definition's for
    at most 2 e of a step's places."""
    u, c = A.U, terms.c
    dist = np.where(np.isneginf(terms.x), 0.0, abs(np.log(np.maximum(terms.p, 1e-300))))
    e = u * ((c.head_dim + 4) * c.scale * (abs(terms.q) @ t(abs(terms.k))) + 4 * dist + 2 * abs(terms.l) + 4) + 2.0**-16
    e = np.where(terms.p > 0, e, 0.0) * abs(terms.g)
    e += terms.p * (c.head_dim + 3) * u * (abs(terms.do) @ t(abs(terms.v)) + (abs(terms.do) * abs(terms.o)).sum(2, keepdims=True))
    ref = terms.results()[1]
    share = np.minimum(1.0, 2 * c.join(c.scale * (e @ abs(terms.k))) / np.maximum(step(ref), 1e-300)).mean()
    other = (dQ != bf16(ref)).mean()
    print(f"  dQ: {other:.4f} of the elements are another neighbour, at most {share:.4f} expected", flush=True)
    assert other <= share + 5 * np.sqrt(share / ref.size), (other, share)


def _sequence(c, nq, nk, seed):
    rng = np.random.default_rng(seed)
    Q, K, V, dO = (bf16(rng.standard_normal((n, h * c.head_dim))) for n, h in
                   ((nq, c.heads), (nk, c.kv_heads), (nk, c.kv_heads), (nq, c.heads)))
    out, lse = O.attention(c, Q, K, V, np.array([0, nq]), np.array([0, nk]))
    return Terms(c, Q, K, V, dO, bf16(out), lse)


@pytest.mark.parametrize("n,hd", [(700, 64), (400, 128)])
def test_the_bounds_tell_a_missing_term(n, hd):
    """Planted in the oracle: rounded operands pass, and each of a missing key, a missing query and a key taken twice does
    not."""
    terms = _sequence(O.Attn(4, 2, hd, hd**-0.5), n, n, 1)
    good = [bf16(x) for x in terms.results(bf16(terms.p), bf16(terms.g))]
    check_norms(terms, good)
    for mistake in range(3):
        p, g = bf16(terms.p), bf16(terms.g)
        for x in (p, g):
            if mistake == 0:
                x[:, :, n // 3] = 0
            elif mistake == 1:
                x[:, n // 2] = 0
            else:
                x[:, :, n // 3] *= 2
        bad = [bf16(x) for x in terms.results(p, g)]
        for i in range(4):
            with pytest.raises(AssertionError):
                check_norms(terms, [bad[i] if k == i else y for k, y in enumerate(good)])


def test_the_share_tells_a_missing_correction():
    """dQ from score gradients that are rounded once fails, with what the rounding left it passes."""
    for n in (33, 64):
        terms = _sequence(O.Attn(8, 2, 64, 0.125), n, n, 2)
        once = bf16(terms.g)
        check_dq_of_cut_tiles(terms, bf16(terms.results(g=once + bf16(terms.g - once))[1]))
        with pytest.raises(AssertionError):
            check_dq_of_cut_tiles(terms, bf16(terms.results(g=once)[1]))


def _run(heads, kv, hd, lq, lk, causal, window=0, seed=0):
    """(Terms, [O, dQ, dK, dV]) of every sequence."""
    at, mats, dO, out, grads, cu_q, cu_k = A.run(heads, kv, hd, "bf16", lq, lk, causal, window, seed)
    c = O.Attn(heads, kv, hd, float(np.float32(at.desc.scale)), causal, window)
    rows = [A.f64(x) for x in (*mats, dO, out)]
    lse, got = A.f64(at.saved[4]), [A.f64(x) for x in (out, *grads)]
    for a, b, e, f in zip(cu_q[:-1], cu_q[1:], cu_k[:-1], cu_k[1:]):
        yield Terms(c, rows[0][a:b], rows[1][e:f], rows[2][e:f], rows[3][a:b], rows[4][a:b], lse[:, a:b]), [
            got[0][a:b], got[1][a:b], got[2][e:f], got[3][e:f]]


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 150), (False, 90)])
@pytest.mark.parametrize("heads,kv,hd,lq,lk", [
    pytest.param(4, 2, 64, [700, 513], [700, 513], marks=gpu),
    pytest.param(2, 1, 128, [400, 260], [1000, 700], marks=gpu),
    pytest.param(4, 4, 96, [300, 650], [300, 650], marks=gpu),
    pytest.param(4, 1, 75, [500], [700], marks=gpu),  # laid out first
    pytest.param(8, 2, 32, [600], [600], marks=gpu),
    pytest.param(16, 4, 128, [257] * 12, [257] * 12, marks=gpu),  # more workgroups than the card holds at once
])
def test_norms(heads, kv, hd, lq, lk, causal, window):
    for terms, got in _run(heads, kv, hd, lq, lk, causal, window):
        check_norms(terms, got)


@pytest.mark.parametrize("heads,kv,hd", [pytest.param(*x, marks=gpu) for x in ((8, 2, 64), (4, 4, 128), (8, 8, 96), (6, 3, 32))])
def test_dq_of_cut_tiles(heads, kv, hd):
    """Causal sequences of up to 64 tokens have no tile that the mask does not cut."""
    for terms, got in _run(heads, kv, hd, [64] * 6 + [33, 50], [64] * 6 + [33, 50], True):
        check_dq_of_cut_tiles(terms, got[1])
