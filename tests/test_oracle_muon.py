"""Pins of the oracle's orthogonalisation and of its step on packed skew blocks: the polynomial on the singular
values (by an SVD), the closed form of a 2 x 2 skew block, skewness, and the limits of the step."""

import numpy as np
import pytest

import oracle as O


@pytest.mark.parametrize("shape", [(6, 6), (5, 9), (9, 5), (1, 4)])
def test_orthogonalize_is_the_polynomial_on_the_singular_values(shape):
    rng = np.random.default_rng(3)
    M = rng.standard_normal(shape)
    hp = O.NsHP(rms=0.0)
    U, s, Vt = np.linalg.svd(M, full_matrices=False)
    x = s / (np.linalg.norm(s) + hp.eps)
    for _ in range(hp.steps):
        x = hp.a * x + hp.b * x**3 + hp.c * x**5
    np.testing.assert_allclose(O.orthogonalize(M, hp), (U * x) @ Vt, atol=1e-12)
    big = s > 0.01 * np.linalg.norm(s)
    assert np.all((x[big] > 0.68) & (x[big] < 1.21)) and big.sum() >= len(s) - 1


def test_convergent_coefficients_give_the_polar_factor():
    M = np.random.default_rng(4).standard_normal((5, 8))
    U, _, Vt = np.linalg.svd(M, full_matrices=False)
    np.testing.assert_allclose(O.orthogonalize(M, O.NsHP(steps=20, a=1.875, b=-1.25, c=0.375, rms=0.0)), U @ Vt, atol=1e-10)


def test_scale_makes_rms_the_rms_of_an_orthogonal_result():
    M = np.random.default_rng(5).standard_normal((7, 12))
    out = O.orthogonalize(M, O.NsHP(steps=20, a=1.875, b=-1.25, c=0.375, rms=0.2))
    # 7 unit rows over 7 x 12 entries
    np.testing.assert_allclose(np.sqrt((out**2).mean()), 0.2, rtol=1e-9)


def test_skew_block_of_two():
    """One slot u: both singular values are |u|, 1/sqrt(2) after the norm, and O = sign(u) p(...)."""
    hp = O.MuonHP(lr=0.1, beta=0.0, nesterov=False, ns=O.NsHP(rms=0.0))
    x = 1 / np.sqrt(2)
    for _ in range(hp.ns.steps):
        x = hp.ns.a * x + hp.ns.b * x**3 + hp.ns.c * x**5
    for u in (3.0, -1e-3):
        q, m = O.muon_step(np.array([[0.5]]), np.array([[u]]), np.array([[9.0]]), 2, 2, hp)
        np.testing.assert_allclose(q, [[0.5 - 0.1 * np.sign(u) * x]], rtol=2e-4)  # eps against |M| = 1.4e-3
        np.testing.assert_allclose(m, [[u]])


def test_step_keeps_the_unused_slots_and_decays_without_an_update():
    rng = np.random.default_rng(6)
    d, b = 21, 8  # blocks of 8, 8 and 5
    q, g, m = (rng.standard_normal((3, 28)) for _ in range(3))
    hp = O.MuonHP(lr=0.1, weight_decay=0.5, ns=O.NsHP())
    q1, m1 = O.muon_step(q, g, m, d, b, hp)
    dead = np.triu_indices(b, 1)[1] >= 5
    assert np.array_equal(q1[2][dead], q[2][dead]) and np.array_equal(m1[2][dead], m[2][dead])
    assert not np.any(q1[2][~dead] == q[2][~dead])
    q0, m0 = O.muon_step(q, 0 * g, 0 * m, d, b, hp)
    np.testing.assert_allclose(q0[:2], 0.95 * q[:2], rtol=1e-15)
    # the orthogonalised skew matrix is skew: its packed half is all of it
    M = rng.standard_normal((7, 7))
    out = O.orthogonalize(M - M.T, O.NsHP())
    np.testing.assert_allclose(out, -out.T, atol=1e-13)


def test_nesterov_update():
    hp = O.MuonHP(beta=0.9, ns=O.NsHP())
    m, u = O.muon_update(2.0, 1.0, hp)
    assert np.isclose(m, 1.1) and np.isclose(u, 0.9 * 1.1 + 0.2)
    m, u = O.muon_update(2.0, 1.0, O.MuonHP(beta=0.9, nesterov=False, ns=O.NsHP()))
    assert m == u
