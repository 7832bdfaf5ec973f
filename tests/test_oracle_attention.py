"""Pins of the oracle's rotary positions, attention and log probabilities: closed forms, torch's float64 functions, and
central differences of the forward for every gradient."""

import numpy as np
import pytest
import torch

import oracle as O


def test_rope_is_a_rotation_by_the_position():
    rng = np.random.default_rng(0)
    f, amp = O.rope_freqs(6, 100.0)
    np.testing.assert_allclose(f, [1.0, 100 ** (-1 / 3), 100 ** (-2 / 3)], rtol=1e-14)
    assert amp == 1.0
    X = rng.standard_normal((5, 2 * 8))
    pos = np.array([0, 1, -3, 7, 100000])
    for layout in ("half", "pairs"):
        Y = O.rope(X, pos, f, 8, layout)
        np.testing.assert_allclose(Y[0], X[0], rtol=1e-15)
        np.testing.assert_allclose(Y.reshape(5, 2, 8)[..., 6:], X.reshape(5, 2, 8)[..., 6:])
        np.testing.assert_allclose((Y**2).sum(1), (X**2).sum(1), rtol=1e-13)
        np.testing.assert_allclose(O.rope(Y, pos, f, 8, layout, inverse=True), X, atol=1e-12)
        # scores of rotated rows depend on the distance alone
        a, b = X[:1], X[1:2]
        s = [float((O.rope(a, np.array([p]), f, 8, layout) * O.rope(b, np.array([p + 5]), f, 8, layout)).sum()) for p in (0, 9, 400)]
        np.testing.assert_allclose(s, s[0], rtol=1e-11)
    Y = O.rope(np.array([[1.0, 0.0]]), np.array([2]), np.array([0.25]), 2, amplitude=3.0)
    np.testing.assert_allclose(Y, [[3 * np.cos(0.5), 3 * np.sin(0.5)]], rtol=1e-14)


def test_rope_scalings():
    f, _ = O.rope_freqs(64)
    for kw in (dict(scaling="linear", factor=4.0),):
        np.testing.assert_allclose(O.rope_freqs(64, **kw)[0], f / 4, rtol=1e-14)
    g, _ = O.rope_freqs(64, scaling="base", factor=4.0)
    np.testing.assert_allclose([g[0], g[-1]], [f[0], f[-1] / 4], rtol=1e-13)  # the last pair turns `factor` times slower
    for scaling in ("bands", "ramp"):
        g, amp = O.rope_freqs(64, scaling=scaling, factor=4.0, original=2048, low=1.0, high=32.0)
        share = (g - f / 4) / (f - f / 4)
        turns = 2048 * f / (2 * np.pi)
        assert share[0] == 1 and abs(share[-1]) < 1e-12 and (np.diff(share) <= 1e-12).all()
        assert (share[turns < 0.7] < 1e-12).all() and (share[turns > 45] > 1 - 1e-12).all()
        assert amp == pytest.approx(1 + 0.1 * np.log(4) if scaling == "ramp" else 1.0)


CASES = [dict(causal=True), dict(causal=False), dict(causal=True, window=3), dict(causal=False, window=2)]


def _attn(seed=0, **kw):
    rng = np.random.default_rng(seed)
    c = O.Attn(4, 2, 3, 0.7, **kw)
    cu_q, cu_k = np.array([0, 3, 3, 8, 9]), np.array([0, 5, 7, 10, 10])
    mats = [rng.standard_normal((9, 12)), rng.standard_normal((10, 6)), rng.standard_normal((10, 6))]
    return c, mats, cu_q, cu_k


@pytest.mark.parametrize("kw", CASES)
def test_attention_matches_torch(kw):
    c, (Q, K, V), cu_q, cu_k = _attn(**kw)
    out, lse = O.attention(c, Q, K, V, cu_q, cu_k)
    for s in range(4):
        nq, nk = cu_q[s + 1] - cu_q[s], cu_k[s + 1] - cu_k[s]
        rows = slice(cu_q[s], cu_q[s + 1])
        if nq == 0 or nk == 0:
            assert not out[rows].any() and np.isneginf(lse[:, rows]).all()
            continue
        t = lambda X, n, cu: torch.tensor(X[cu[s]:cu[s + 1]]).view(-1, n, 3).transpose(0, 1)
        q, k, v = t(Q, 4, cu_q), t(K, 2, cu_k).repeat_interleave(2, 0), t(V, 2, cu_k).repeat_interleave(2, 0)
        on = torch.tensor(c.sees(nq, nk))
        ref = torch.nn.functional.scaled_dot_product_attention(q, k, v, attn_mask=on, scale=0.7)
        ref = torch.where(on.any(1)[None, :, None], ref, torch.zeros_like(ref))
        np.testing.assert_allclose(out[rows], ref.transpose(0, 1).reshape(nq, 12).numpy(), atol=1e-13)
        empty = ~on.any(1).numpy()
        assert np.isneginf(lse[:, rows][:, empty]).all() and np.isfinite(lse[:, rows][:, ~empty]).all()


@pytest.mark.parametrize("kw", CASES)
def test_attention_gradients_by_differences(kw):
    c, mats, cu_q, cu_k = _attn(1, **kw)
    dO = np.random.default_rng(2).standard_normal((9, 12))
    out, lse = O.attention(c, *mats, cu_q, cu_k)
    grads = O.attention_backward(c, dO, *mats, out, lse, cu_q, cu_k)
    for i, g in enumerate(grads):
        num = np.zeros_like(g)
        for at in np.ndindex(*g.shape):
            f = []
            for h in (1e-5, -1e-5):
                m = [x.copy() for x in mats]
                m[i][at] += h
                f.append((O.attention(c, *m, cu_q, cu_k)[0] * dO).sum())
            num[at] = (f[0] - f[1]) / 2e-5
        np.testing.assert_allclose(g, num, atol=3e-9)


def test_log_probabilities_match_torch():
    rng = np.random.default_rng(3)
    X = rng.standard_normal((6, 11)) * 3
    X[1, 4] = -np.inf
    X[2, [3, 7]] = X[2].max() + 1
    X[5] = -np.inf
    t = np.array([0, 5, -1, 11, 10, 3])
    lp, lse, H, ids, tlp = O.token_logprobs(X, t, 0.8, 4)
    ref = torch.log_softmax(torch.tensor(X[:5]) * 0.8, 1)
    np.testing.assert_allclose(lp[[0, 1, 4]], ref[[0, 1, 4], [0, 5, 10]].numpy(), rtol=1e-13)
    assert lp[2] == lp[3] == 0 and np.isneginf(lp[5]) and np.isneginf(lse[5]) and H[5] == 0
    np.testing.assert_allclose(lse[:5], torch.logsumexp(torch.tensor(X[:5]) * 0.8, 1).numpy(), rtol=1e-13)
    np.testing.assert_allclose(H[[0, 2, 3, 4]], torch.distributions.Categorical(logits=torch.tensor(X[[0, 2, 3, 4]]) * 0.8)
                               .entropy().numpy(), rtol=1e-12)
    assert list(ids[2][:2]) == [3, 7] and list(ids[5]) == [0, 1, 2, 3]
    np.testing.assert_allclose(tlp[:5], ref.sort(1, descending=True).values[:, :4].numpy(), rtol=1e-12)


def test_log_probability_gradients_by_differences():
    rng = np.random.default_rng(4)
    X = rng.standard_normal((4, 7)) * 2
    t, a, b = np.array([0, 6, -1, 3]), rng.standard_normal(4), rng.standard_normal(4)
    _, lse, H, _, _ = O.token_logprobs(X, t, 1.3)
    g = O.token_logprobs_backward(X, t, lse, H, a, b, 1.3)
    num = np.zeros_like(X)
    for at in np.ndindex(*X.shape):
        f = []
        for h in (1e-5, -1e-5):
            Y = X.copy()
            Y[at] += h
            lp, _, ent, _, _ = O.token_logprobs(Y, t, 1.3)
            f.append((a * lp).sum() + (b * ent).sum())
        num[at] = (f[0] - f[1]) / 2e-5
    np.testing.assert_allclose(g, num, atol=1e-9)
    X[0, 2] = -np.inf
    X[3] = -np.inf
    _, lse, H, _, _ = O.token_logprobs(X, t, 1.3)
    g = O.token_logprobs_backward(X, t, lse, H, a, b, 1.3)
    assert np.isfinite(g).all() and g[0, 2] == 0 and not g[3].any()
