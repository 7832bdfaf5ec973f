"""Pins of the oracle's norm: torch's float64 layer norm, the RMS closed form, and central differences of the
forward for every gradient."""

import numpy as np
import pytest
import torch

import oracle as O


def _inputs(T=5, d=7, seed=0):
    rng = np.random.default_rng(seed)
    return rng.standard_normal((T, d)) * 2 + 0.5, rng.standard_normal((T, d)), 1 + 0.3 * rng.standard_normal(d), rng.standard_normal(d)


def test_layer_norm_matches_torch():
    S, _, w, b = _inputs()
    Y, mean, rs = O.norm_forward(S, w, b, "layer", 1e-5)
    ref = torch.nn.functional.layer_norm(torch.tensor(S), (S.shape[1],), torch.tensor(w), torch.tensor(b), 1e-5)
    np.testing.assert_allclose(Y, ref.numpy(), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(mean, S.mean(1), rtol=1e-13)
    np.testing.assert_allclose(rs, 1 / np.sqrt(S.var(1) + 1e-5), rtol=1e-12)


def test_rms_norm_closed_form():
    S, _, w, _ = _inputs(seed=1)
    Y, mean, _ = O.norm_forward(S, w, None, "rms", 1e-6)
    np.testing.assert_allclose(Y, S / np.sqrt((S**2).mean(1, keepdims=True) + 1e-6) * w, rtol=1e-13)
    assert not mean.any()


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("affine", [True, False])
def test_gradients_match_differences(kind, affine):
    S, dY, w, b = _inputs(seed=2)
    w, b = (w, b if kind == "layer" else None) if affine else (None, None)
    loss = lambda S_, w_, b_: float((O.norm_forward(S_, w_, b_, kind, 1e-3)[0] * dY).sum())
    _, mean, rs = O.norm_forward(S, w, b, kind, 1e-3)
    dS, dw, db = O.norm_backward(S, dY, w, mean, rs, kind)
    h = 1e-6

    def diff(a, f):
        out = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            up, dn = a.copy(), a.copy()
            up[i] += h
            dn[i] -= h
            out[i] = (f(up) - f(dn)) / (2 * h)
        return out

    np.testing.assert_allclose(dS, diff(S, lambda x: loss(x, w, b)), rtol=1e-6, atol=1e-7)
    if affine:
        np.testing.assert_allclose(dw, diff(w, lambda x: loss(S, x, b)), rtol=1e-6, atol=1e-7)
        if b is not None:
            np.testing.assert_allclose(db, diff(b, lambda x: loss(S, w, x)), rtol=1e-6, atol=1e-7)
