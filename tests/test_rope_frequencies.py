"""Frequencies that scaling makes infinite are refused; the largest finite ones turn by their fraction."""
import math

import pytest

import quantized_kv_speculative_gb300 as kvq
from quantized_kv_speculative_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return kvq.load_library()


@pytest.mark.parametrize("kw", [dict(scaling="linear", factor=1e-320), dict(scaling="linear", factor=1e-10, inv_freq=[1e300] * 64),
                                dict(scaling="ramp", factor=5e-324), dict(scaling="bands", factor=1e-300, inv_freq=[-1e-2 * 1e12] * 64, low=1e17, high=1e18)])
def test_frequencies_that_scaling_makes_infinite_are_refused(kw):
    with pytest.raises(kvq.KVQError):
        kvq.Rope(128, **kw)


@pytest.mark.parametrize("kw", [dict(inv_freq=[1.7e308] * 64), dict(scaling="linear", factor=1e-300, inv_freq=[1.0] * 64),
                                dict(scaling="linear", factor=1e300), dict(inv_freq=[-5e-324] * 64)])
def test_finite_ones_are_taken(kw):
    f = [x / (kw.get("factor", 1.0) if "scaling" in kw else 1.0) for x in kw.get("inv_freq", [10000.0 ** (-i / 64) for i in range(64)])]
    turns = [t / 2.0 ** 64 for t in kvq.Rope(128, **kw).struct.turns]
    for t, x in zip(turns, f):
        want = x / 6.283185307179586476925286766559
        want -= math.floor(want)
        assert abs(t - want) <= 2.0 ** -52 or abs(abs(t - want) - 1.0) <= 2.0 ** -52
