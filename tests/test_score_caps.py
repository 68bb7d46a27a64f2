"""Caps from tight to far above the logits, over quantized, residual and pending tokens.

Tolerance: a capped logit is off by what the cap's argument is off and by 2^-20 of its own size, whatever the cap (below 0.7 of the
cap a polynomial within 4.6e-7 of the value; above, two approximations within 2^-22 of the cap each).  |logit| is at most
``size`` = scale sum |q| |k|, so ``extra`` = 2^-20 of that stands in the place of the 2^-20 cap that the comparison allows elsewhere."""
import pytest

import kvq_inputs as ki
import quantized_kv_speculative_gb300 as kvq
from quantized_kv_speculative_gb300 import _build

from plain_attention import assert_close, attend_plain, build

EXTRA = 2.0 ** -20


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kvq.load_library()


def dev(x):
    return ki.f32_to_bf16_tensor(x, "cuda")


def bounded(args, kw, cap):
    """attend_plain under the cap, with the uncapped logits' bound."""
    out, lse, _, vmax = attend_plain(*args, cap=cap, **kw)
    return out, lse, attend_plain(*args, **kw)[2], vmax


CAPS = [65.0, 1e3, 1e4, 1e6, 1e9, 1e30, 1.2e38, 3.4e38]   # (tanh in 64 bits is exact enough for all of them)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("mode,hg,gamma", [("int8", 2, 2), ("int4", 1, 1), ("int2", 4, 2), ("int1", 3, 1)])
def test_loose_caps(lib, mode, hg, gamma, cap):
    gc, ocs = build(kvq.MODE_FORMAT[mode], [500, 77], 2, 64, 32, seed=1)
    q, (pk, pv) = ki.queries(1, 2, gamma, 2 * hg, 64), ki.pending(1, 2, 2, gamma, 64)
    out, lse = kvq.kvq_attend_mod(gc, mode, dev(q), kvq.ScoreMod(cap), dev(pk), dev(pv))
    assert_close(out, lse, bounded((ocs, mode, q, pk, pv), {}, cap), extra=EXTRA)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [1e6, 1e30, 3.4e38])
def test_a_cap_far_above_the_logits_changes_nothing(lib, cap):
    """Against kvq_attend's own results: both within their bounds of the same values."""
    gc, ocs = build("hier8", [900], 2, 128, 32, seed=2)
    q = ki.queries(2, 1, 2, 4, 128)
    a, la = kvq.kvq_attend(gc, "int8", dev(q))
    b, lb = kvq.kvq_attend_mod(gc, "int8", dev(q), kvq.ScoreMod(cap))
    plain = attend_plain(ocs, "int8", q)
    assert_close(a, la, plain), assert_close(b, lb, plain, extra=EXTRA)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [1e-45, 1e-38, 1e-30])
def test_caps_below_every_logit(lib, cap):
    """All logits are 0 to within fp32: the mean of the values."""
    gc, ocs = build("hier8", [300], 2, 64, 32, seed=3)
    q = ki.queries(3, 1, 1, 4, 64)
    assert_close(*kvq.kvq_attend_mod(gc, "int8", dev(q), kvq.ScoreMod(cap)), attend_plain(ocs, "int8", 0 * q))
