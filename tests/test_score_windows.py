"""The widest windows, for queries that stand before position 0: more rows than tokens, none of them pending."""
import pytest
import torch

import kvq_inputs as ki
import quantized_kv_speculative_gb300 as kvq
from quantized_kv_speculative_gb300 import _build

from plain_attention import assert_close, attend_plain, build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kvq.load_library()


def dev(x):
    return ki.f32_to_bf16_tensor(x, "cuda")


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 3, 7])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 4, 2 ** 31 - 9, 8, 1])
def test_windows_that_begin_past_32_bits(lib, n, window):
    q = ki.queries(n, 1, 8, 2, 64)
    tokens, ocs = build("hier8", [n], 2, 64, 32, seed=n, ragged=False)
    empty, none = build("hier8", [0], 2, 64, 32, ragged=False)
    mod = kvq.ScoreMod(window=window)
    assert_close(*kvq.kvq_attend_mod(tokens, "int8", dev(q), mod), attend_plain(ocs, "int8", q, window=window))
    out, lse = kvq.kvq_attend_shared(tokens, empty, "int8", dev(q), mod=mod)
    assert_close(out, lse, attend_plain(none, "int8", q, window=window, prefix=ocs[0]), extra_v=2.0 ** -9)
