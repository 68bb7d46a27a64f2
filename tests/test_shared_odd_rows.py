"""Rows of kvq_attend_shared whose logits are no numbers say so, as kvq_attend's do, whatever the sequence's own cache adds."""
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
@pytest.mark.parametrize("n0", [20, 600, 9000])
@pytest.mark.parametrize("lens", [[0, 0, 0], [20, 20, 20], [700, 700, 700]])
@pytest.mark.parametrize("cap", [0.0, 30.0])
def test_queries_that_are_no_numbers(lib, n0, lens, cap):
    pc, (po,) = build("hier8", [n0], 2, 64, 32, seed=1, ragged=False)
    gc, ocs = build("hier8", lens, 2, 64, 32, seed=2, ragged=False)
    q = ki.queries(3, 3, 1, 4, 64)
    qd = dev(q)
    qd[1] = float("nan")
    qd[2, :, :, 5] = float("nan")
    out, lse = kvq.kvq_attend_shared(pc, gc, "int8", qd, mod=kvq.ScoreMod(cap) if cap else None)
    assert torch.all(torch.isnan(out[1:])) and not torch.any(torch.isfinite(lse[1:]))
    assert_close(out[:1], lse[:1], attend_plain(ocs[:1], "int8", q[:1], cap=cap, prefix=po), extra_v=2.0 ** -9)


@pytest.mark.gpu
def test_rows_that_see_nothing_are_zero_beside_them(lib):
    """Hidden is not the same as no number: a query of NaN that sees no key is a row of zeros, as in kvq_attend_mod."""
    pc, _ = build("hier8", [300], 2, 64, 32, seed=1, ragged=False)
    gc, _ = build("hier8", [40, 40], 2, 64, 32, seed=2, ragged=False)
    first = torch.tensor([0, 10 ** 6], dtype=torch.int32, device="cuda")
    q = torch.full((2, 1, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    out, lse = kvq.kvq_attend_shared(pc, gc, "int8", q, mod=kvq.ScoreMod(first=first))
    assert torch.all(torch.isnan(out[0])) and torch.all(out[1] == 0) and torch.all(torch.isneginf(lse[1]))
