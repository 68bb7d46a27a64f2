"""A ScoreMod whose settings are changed between calls: later calls see them."""
import gc as garbage

import pytest
import torch

import kvq_inputs as ki
import quantized_kv_speculative_gb300 as kvq
from quantized_kv_speculative_gb300 import _build

from plain_attention import build, slopes_of


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return kvq.load_library()


def test_numbers_follow():
    mod = kvq.ScoreMod(30.0, 5)
    mod.softcap, mod.window = 12.5, 77
    assert mod.struct.softcap == 12.5 and mod.struct.window == 77 and (mod.softcap, mod.window) == (12.5, 77)
    assert mod.slopes is None and mod.first is None and not mod.struct.slopes and not mod.struct.first


@pytest.mark.parametrize("window", [2 ** 31, 2 ** 32 + 5, 2 ** 40, -2 ** 31 - 1])
def test_windows_past_32_bits_are_refused(window):
    with pytest.raises(ValueError):
        kvq.ScoreMod(window=window)
    mod = kvq.ScoreMod(window=3)
    with pytest.raises(ValueError):
        mod.window = window
    assert mod.window == 3 and kvq.ScoreMod(window=2 ** 31 - 1).window == 2 ** 31 - 1


def test_a_refused_tensor_changes_nothing():
    mod = kvq.ScoreMod(30.0)
    for name in ("slopes", "first"):
        with pytest.raises(ValueError):
            setattr(mod, name, torch.zeros(4))   # not on the device
        assert getattr(mod, name) is None and not getattr(mod.struct, name)


@pytest.mark.gpu
def test_tensors_follow():
    cache, _ = build("hier8", [500, 500], 2, 64, 32, ragged=False)
    prefix, _ = build("hier8", [300], 2, 64, 32, ragged=False)
    q = ki.f32_to_bf16_tensor(ki.queries(1, 2, 1, 4, 64), "cuda")
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    before = (ints(0, 100), slopes_of(4).cuda())   # (kept: what a stale pointer would read)
    mod = kvq.ScoreMod(30.0, first=before[0], slopes=before[1])
    mod.first, mod.slopes, mod.window = ints(450, 320), 0.5 * slopes_of(4).cuda(), 400
    garbage.collect()
    want = kvq.ScoreMod(30.0, 400, 0.5 * slopes_of(4).cuda(), ints(450, 320))
    for call in (lambda m: kvq.kvq_attend_mod(cache, "int8", q, m), lambda m: kvq.kvq_attend_shared(prefix, cache, "int8", q, mod=m)):
        for a, b in zip(call(mod), call(want)):
            assert torch.equal(a, b)
    mod.first = mod.slopes = None
    for a, b in zip(kvq.kvq_attend_mod(cache, "int8", q, mod), kvq.kvq_attend_mod(cache, "int8", q, kvq.ScoreMod(30.0, 400))):
        assert torch.equal(a, b)
