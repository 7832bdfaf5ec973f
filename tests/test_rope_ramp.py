"""The ramp of the rotary frequencies, by values worked out from its definition, for the library and for the oracle.

With rot_dim = 8 and base = 256, pair j has f = 4^-j, so within `original` = 2 pi N positions it makes N 4^-j turns, and t
turns are made by pair log4(N / t).  With factor 4 a pair of unscaled share s gets f (s + (1 - s) / 4).  The cases keep
log4(N / t) away from whole numbers, where its rounding up or down would hang on the last digit."""

import numpy as np
import pytest

import oracle as O
from orthogonal_reparameterized_cnp_amd import binding as B

LIBRARY = lambda rot, **kw: B.poetx_rope_freqs(rot, B.rope_params(kw.pop("base"), **kw))

CASES = [
    # N, low, high, share of every pair
    (1024, 1.5, 400.0, [1, 4 / 5, 3 / 5, 2 / 5]),  # from 0.68 to 4.71: the ramp 0 .. 5 ends behind pair 3
    (1024, 3.0, 40.0, [1, 1, 1, 2 / 3]),  # from 2.34 to 4.21: 2 .. 5
    (256, 1.5, 40.0, [1, 1, 2 / 3, 1 / 3]),  # from 1.34 to 3.71: 1 .. 4
    (64, 3.0, 20.0, [1, 2 / 3, 1 / 3, 0]),  # from 0.84 to 2.21: 0 .. 3, within the pairs
    (4, 0.1, 100.0, [1, 2 / 3, 1 / 3, 0]),  # from -2.32, held at 0, to 2.66: 0 .. 3
    (2**20, 1.5, 3e5, [1, 6 / 7, 5 / 7, 4 / 7]),  # from 0.90 to 9.71, held at rot_dim - 1: 0 .. 7
    (2**20, 1.0e3, 3e4, [1, 1, 1, 3 / 4]),  # from 2.56 to 5.02: 2 .. 6
]


@pytest.mark.parametrize("freqs", [LIBRARY, O.rope_freqs], ids=["library", "oracle"])
@pytest.mark.parametrize("N,low,high,share", CASES)
def test_ramp(N, low, high, share, freqs):
    f, amp = freqs(8, base=256.0, scaling="ramp", factor=4.0, original=2 * np.pi * N, low=low, high=high)
    share = np.array(share, dtype=float)
    np.testing.assert_allclose(f, 4.0 ** -np.arange(4) * (share + (1 - share) / 4), rtol=1e-13)
    assert amp == pytest.approx(1 + 0.1 * np.log(4), rel=1e-7)


def test_the_ends_of_the_parameters():
    """Parameters whose quotients and powers leave the range of a double give the frequencies that the formulas name."""
    f = 10.0 ** -np.arange(4)  # rot_dim 8, base 10^4
    for low, high, original in ((1e-310, 1e-309, 1e10), (1e-20, 1e-10, 1e300)):  # every pair makes more than `high` turns
        for scaling in ("ramp", "bands"):
            got, _ = LIBRARY(8, base=1e4, scaling=scaling, factor=4.0, original=original, low=low, high=high)
            np.testing.assert_allclose(got, f, rtol=1e-13)
    for scaling in ("ramp", "bands"):  # and fewer than `low`
        got, _ = LIBRARY(8, base=1e4, scaling=scaling, factor=4.0, original=1.0, low=1e307, high=1.7e308)
        np.testing.assert_allclose(got[scaling == "ramp":], f[scaling == "ramp":] / 4, rtol=1e-13)
    # the last pair turns `factor` times slower, however large the base that this takes
    got, _ = LIBRARY(4, base=1e4, scaling="base", factor=1e200)
    np.testing.assert_allclose(got, [1.0, 1e-202], rtol=1e-13)
