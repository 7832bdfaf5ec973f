"""Refusals and host helpers of the rotary positions, on the CPU: the C ABI rejects before any device work (the pointers
are never dereferenced), and layer.PoetxRope rejects malformed tensors before any library call."""

import ctypes

import numpy as np
import pytest
import torch

import oracle as O
from orthogonal_reparameterized_cnp_amd import binding as B
from orthogonal_reparameterized_cnp_amd import layer as L

FAKE = 1 << 20


def _call(dsc=None, T=4, pos=FAKE, freqs=FAKE, amp=1.0, inverse=0, X=(2 * FAKE, 3 * FAKE), ldx=(128, 64), heads=(2, 1),
          Y=(4 * FAKE, 5 * FAKE), ldy=(128, 64), count=None, desc_null=False, null=()):
    dsc = dsc or B.rope_desc(64, 64, "half", "bf16")
    n = len(X)
    args = {"X": (ctypes.c_void_p * n)(*X), "ldx": (ctypes.c_int64 * n)(*ldx), "heads": (ctypes.c_int32 * n)(*heads),
            "Y": (ctypes.c_void_p * n)(*Y), "ldy": (ctypes.c_int64 * n)(*ldy)}
    args.update({k: None for k in null})
    return B.lib().poetx_rope(None if desc_null else ctypes.byref(dsc), T, pos, freqs, amp, inverse,
                              n if count is None else count, args["X"], args["ldx"], args["heads"], args["Y"], args["ldy"],
                              None)


def test_refusals():
    assert _call(T=0) == B.POETX_OK
    assert _call(desc_null=True) == B.POETX_E_NULL
    for bad in ((1, 2, 0, 1), (1025, 64, 0, 1), (64, 0, 0, 1), (64, 3, 0, 1), (64, 66, 0, 1), (64, 64, 2, 1)):
        assert _call(B.RopeDesc(*bad)) == B.POETX_E_SHAPE, bad
    assert _call(B.RopeDesc(64, 64, 0, B.POETX_I8)) == B.POETX_E_DTYPE
    for kw in (dict(freqs=None), dict(X=(None, FAKE)), dict(Y=(4 * FAKE, None)), dict(null=("X",)), dict(null=("ldx",)),
               dict(null=("heads",)), dict(null=("Y",)), dict(null=("ldy",))):
        assert _call(**kw) == B.POETX_E_NULL, kw
    for kw in (dict(T=-1), dict(T=(1 << 30) + 1), dict(amp=float("nan")), dict(amp=float("inf")), dict(inverse=2),
               dict(count=0), dict(count=9), dict(heads=(0, 1)), dict(heads=(2, 1 << 15)), dict(ldx=(127, 64)),
               dict(ldy=(128, 63)), dict(X=(2 * FAKE + 1, 3 * FAKE)), dict(freqs=FAKE + 4), dict(pos=FAKE + 2),
               dict(ldx=((1 << 31) + 1, 64))):
        assert _call(**kw) == B.POETX_E_SHAPE, kw


def test_overlap_refusals():
    """A result shares no cell with another operand; columns of one buffer share none."""
    row = 64 * 2
    for Y in ((2 * FAKE + 2, 5 * FAKE), (3 * FAKE, 5 * FAKE), (5 * FAKE, 5 * FAKE), (4 * FAKE, 4 * FAKE + row),
              (4 * FAKE, 2 * FAKE), (FAKE, 5 * FAKE), (4 * FAKE, FAKE - 2)):
        assert _call(Y=Y) == B.POETX_E_SHAPE, Y
    assert _call(X=(2 * FAKE, 2 * FAKE + 1), Y=(2 * FAKE, 2 * FAKE)) == B.POETX_E_SHAPE
    assert _call(Y=(2 * FAKE, 5 * FAKE), ldy=(129, 64)) == B.POETX_E_SHAPE
    wide = dict(ldx=(192, 192), ldy=(192, 192), X=(2 * FAKE, 2 * FAKE + 256))
    for off in (0, 254, 2 * 192 - 2, 2 * 192, 3 * 2 * 192 + 254):
        assert _call(Y=(4 * FAKE, 4 * FAKE + off), **wide) == B.POETX_E_SHAPE, off
        assert _call(Y=(2 * FAKE + off + (off == 0) * 2, 5 * FAKE), **wide) == B.POETX_E_SHAPE, off


@pytest.mark.parametrize("rot", [2, 6, 34, 128])
@pytest.mark.parametrize("kw", [dict(), dict(scaling="linear", factor=3.5), dict(scaling="base", factor=8.0),
                                dict(scaling="bands", factor=8.0, original=8192.0, low=1.0, high=4.0),
                                dict(scaling="ramp", factor=16.0, original=4096.0, low=1.0, high=32.0),
                                dict(scaling="ramp", factor=2.0, original=1.0, low=0.5, high=0.6),
                                dict(scaling="bands", factor=1.0, original=4096.0)])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
def test_frequencies(rot, kw, base):
    if kw.get("scaling") == "base" and rot == 2:
        with pytest.raises(B.PoetxError):
            B.poetx_rope_freqs(rot, B.rope_params(base, **kw))
        return
    f, amp = B.poetx_rope_freqs(rot, B.rope_params(base, **kw))
    ref, ramp = O.rope_freqs(rot, base, **kw)
    np.testing.assert_allclose(f, ref, rtol=1e-11)  # a step of the ramp amplifies a rounding by its slope
    assert amp == pytest.approx(ramp, rel=1e-7)


def test_frequency_refusals():
    ok = dict(base=1e4, scaling="bands", factor=2.0, original=100.0, low=1.0, high=2.0)
    B.poetx_rope_freqs(8, B.rope_params(**ok))
    inf, nan = float("inf"), float("nan")
    for kw in (dict(base=1.0), dict(base=inf), dict(base=nan), dict(factor=0.5), dict(factor=inf), dict(factor=nan),
               dict(original=0.0), dict(original=inf), dict(low=0.0), dict(high=1.0), dict(high=inf), dict(low=nan)):
        with pytest.raises(B.PoetxError) as e:
            B.poetx_rope_freqs(8, B.rope_params(**{**ok, **kw}))
        assert e.value.status == B.POETX_E_SHAPE, kw
    for rot in (0, 3, -2, 1026):
        with pytest.raises(B.PoetxError):
            B.poetx_rope_freqs(rot, B.rope_params())
    bad = B.rope_params()
    bad.scaling = 5
    with pytest.raises(B.PoetxError):
        B.poetx_rope_freqs(8, bad)
    out, amp = (ctypes.c_double * 4)(), ctypes.c_float()
    p = B.rope_params()
    assert B.lib().poetx_rope_freqs(8, None, out, ctypes.byref(amp)) == B.POETX_E_NULL
    assert B.lib().poetx_rope_freqs(8, ctypes.byref(p), None, ctypes.byref(amp)) == B.POETX_E_NULL
    assert B.lib().poetx_rope_freqs(8, ctypes.byref(p), out, None) == B.POETX_E_NULL


bf = lambda *s: torch.zeros(*s, dtype=torch.bfloat16)


def test_layer_rejects(monkeypatch):
    def boom(*a, **k):
        raise AssertionError("a library call was made before the arguments were checked")

    monkeypatch.setattr(B, "poetx_rope", boom)
    for kw, msg in ((dict(layout="both"), "layout"), (dict(scaling="more"), "scaling"), (dict(act="i8"), "act")):
        with pytest.raises(ValueError, match=msg):
            L.PoetxRope(64, device="cpu", **kw)
    with pytest.raises(B.PoetxError):
        L.PoetxRope(64, 3, device="cpu")
    r = L.PoetxRope(64, device="cpu")
    for Xs, kw, msg in (([], {}, "one or more"), ([bf(4, 64)], dict(Ys=[]), "one or more"), ([bf(4, 63)], {}, "2-D"),
                        ([bf(4, 0)], {}, "2-D"), ([bf(64)], {}, "2-D"), ([bf(4, 64)], {}, "GPU"),
                        ([bf(4, 64).float()], {}, "dtype"), ([bf(64, 4).t().contiguous().t().t()], {}, "GPU"),
                        ([bf(4, 64)], dict(pos=torch.zeros(3, dtype=torch.int32)), "shape"),
                        ([bf(4, 64)], dict(pos=torch.zeros(4, dtype=torch.int64)), "dtype")):
        with pytest.raises(ValueError, match=msg):
            r.forward(Xs, **kw)
        with pytest.raises(ValueError):
            r.backward(Xs, kw.get("pos"), kw.get("Ys"))
