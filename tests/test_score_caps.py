"""Caps from tight to far above the logits, over quantized, residual and pending tokens and over a shared prefix.

Tolerance: a capped logit is off by what the cap's argument is off and by 2^-20 of its own size, whatever the cap (below 0.7 of the
cap a polynomial within 4.6e-7 of the value; above, two approximations within 2^-22 of the cap each).  |logit| is at most
``size`` = scale sum |q| |k|, so ``extra`` = 2^-20 of that stands in the place of the 2^-20 cap that the comparison allows elsewhere."""
import numpy as np
import pytest
import torch

import kvq_inputs as ki
import quantized_kv_speculative_gb300 as kvq
from quantized_kv_speculative_gb300 import _build

from plain_attention import assert_close, attend_plain, build

EXTRA = 2.0 ** -20
EXTRA_V = 2.0 ** -9   # the shared pass's values and weights, in fp16 each


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


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [1e-45, 1e-38, 1e-30])
def test_caps_below_every_logit_over_a_prefix(lib, cap):
    pc, (po,) = build("hier8", [200], 2, 64, 32, seed=4, ragged=False)
    gc, ocs = build("hier8", [300], 2, 64, 32, seed=3)
    q = ki.queries(3, 1, 1, 4, 64)
    out, lse = kvq.kvq_attend_shared(pc, gc, "int8", dev(q), mod=kvq.ScoreMod(cap))
    assert_close(out, lse, attend_plain(ocs, "int8", 0 * q, prefix=po), extra_v=EXTRA_V)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", CAPS)
@pytest.mark.parametrize("mode,n0,B,hg", [("int8", 37, 2, 2), ("int4", 300, 3, 1), ("int2", 1000, 11, 4), ("int8", 700, 20, 4)])
def test_loose_caps_over_a_prefix(lib, mode, n0, B, hg, cap):
    """Prefixes that end inside a tile, whose last lanes hold no token."""
    fmt = kvq.MODE_FORMAT[mode]
    pc, (po,) = build(fmt, [n0], 1, 64, 32, seed=5, ragged=False)
    gc, ocs = build(fmt, [40 + i for i in range(B)], 1, 64, 32, seed=6)
    q = ki.queries(5, B, 1, hg, 64)
    out, lse = kvq.kvq_attend_shared(pc, gc, mode, dev(q), mod=kvq.ScoreMod(cap))
    assert_close(out, lse, bounded((ocs, mode, q), dict(prefix=po), cap), extra=EXTRA, extra_v=EXTRA_V)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [1e3, 1e6, 1e30])
def test_a_row_past_the_cap_leaves_the_others_alone(lib, cap):
    """A padded row of the largest values, or one at the cap, beside ordinary rows: the others' log-sum-exps stay within their own
    logits' bound, not the cap's."""
    pc, (po,) = build("hier8", [600], 1, 64, 32, seed=7, ragged=False)
    gc, ocs = build("hier8", [40] * 4, 1, 64, 32, seed=8, ragged=False)
    q = ki.queries(7, 4, 1, 2, 64)
    for odd in (3e38, float(min(cap, 1e37))):
        qd = dev(q)
        qd[1] = odd
        qd[2] = -odd
        out, lse = kvq.kvq_attend_shared(pc, gc, "int8", qd, mod=kvq.ScoreMod(cap))
        good = [0, 3]
        assert_close(out[good], lse[good], bounded(([ocs[b] for b in good], "int8", q[good]), dict(prefix=po), cap), extra=EXTRA, extra_v=EXTRA_V)


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [20.0, 64.0])
def test_ordinary_caps_over_a_prefix_that_ends_inside_a_tile(lib, cap):
    """One key seen: its capped logit is the log-sum-exp, off by 2^-20 of itself also where lanes of the tile hold no token."""
    pc, (po,) = build("hier8", [37], 2, 64, 32, seed=9, ragged=False)
    gc, ocs = build("hier8", [0, 0], 2, 64, 32, seed=9, ragged=False)
    q = ki.queries(9, 2, 1, 4, 64) * np.float32(0.05)
    q = ki.round_bf16(q)
    first = torch.tensor([36, 36], dtype=torch.int32, device="cuda")
    out, lse = kvq.kvq_attend_shared(pc, gc, "int8", dev(q), mod=kvq.ScoreMod(cap, first=first))
    want, want_lse, delta, vmax = bounded((ocs, "int8", q), dict(prefix=po, first=[36, 36]), cap)
    off = np.abs(lse.cpu().numpy().astype(np.float64) - want_lse)
    assert np.all(off <= delta + (2.0 ** -20 + 2.0 ** -22) * np.abs(want_lse) + 2.0 ** -24 * 4), off.max()
    assert_close(out, None, (want, want_lse, delta, vmax), extra=EXTRA, extra_v=EXTRA_V)
