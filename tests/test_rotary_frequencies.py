"""Rotary frequencies at the ends of what the call takes."""
import os

import numpy as np
import pytest

from oracle import rotary


@pytest.fixture(scope="module")
def dsv():
    from serving_draft_verify_gb300 import build as b
    if not os.path.exists(b.LIB):
        b.build()
    import serving_draft_verify_gb300 as m
    return m


@pytest.mark.parametrize("rot,base,factor", [(4, 1e4, 1e160), (64, 1e300, 1e30), (4, 1e308, 1e308), (256, 1e4, 1e306), (64, 1e4, 8.0)])
def test_raised_base_past_doubles(dsv, rot, base, factor):
    """base factor^(rot / (rot - 2)) may leave the doubles; its powers between 1 and 1 / factor do not.
    ln f is at most 2130 and off by 4 parts in 2^53 of that, so f by 2^-39 of itself, and is rounded once."""
    i = np.arange(rot // 2)
    want = np.exp(-2.0 * i / rot * (np.log(base) + rot / (rot - 2.0) * np.log(factor)))
    freq, m = dsv.dspark_rotary_frequencies(rot, base, "base", factor, device="cpu")
    got = freq.double().numpy()
    assert got[0] == 1 and m == 1
    # below float32's normal numbers a rounding is 2^-150
    assert (np.abs(got - want) <= want * (2.0 ** -24 + 2.0 ** -39) + 2.0 ** -150).all()
    if factor == 8.0:
        np.testing.assert_allclose(want, rotary.frequencies(rot, base, "base", factor)[0], rtol=1e-12)


def test_ramp_halfway():
    """4096 positions at base 10^4 and 128 elements: d(32) = 20.9 and d(1) = 45.03, so pairs 20 to 46 are blended, and
    pair 33 keeps one half: 1/2 + 1/2 / 4 of its frequency."""
    ramp, _ = rotary.frequencies(128, 1e4, "ramp", 4, original=4096)
    f = rotary.frequencies(128, 1e4)[0]
    np.testing.assert_allclose(ramp[33], 0.625 * f[33])
    np.testing.assert_allclose(ramp[20:47] / f[20:47], 1 - 0.75 * np.arange(27) / 26)
