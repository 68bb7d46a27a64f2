"""Rotary positions of views whose dimensions of one entry have strides that mean nothing."""
import pytest
import torch

import quantized_kv_speculative_gb300 as kvq
from quantized_kv_speculative_gb300 import _build


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kvq.load_library()


@pytest.mark.gpu
@pytest.mark.parametrize("shape", [(1, 5, 4), (3, 1, 4), (3, 5, 1), (1, 1, 4), (1, 1, 1)])
@pytest.mark.parametrize("stride", [1, 3, 1 << 50, 0])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_dimensions_of_one_entry_may_have_any_stride(lib, shape, stride, layout):
    D = 64
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(shape + (D,), generator=g, device="cuda").bfloat16()
    odd = torch.as_strided(x, x.shape, [s if n > 1 else stride for n, s in zip(shape, x.stride())] + [1])
    rope = kvq.Rope(D, layout=layout)
    want = kvq.kvq_rope_apply(rope, x, x, first_position=7)
    got = kvq.kvq_rope_apply(rope, odd, odd, first_position=7)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    kvq.kvq_rope_apply(rope, odd, q_out=x, first_position=7)   # in place: the same layout
    assert torch.equal(x, want[0])


@pytest.mark.gpu
def test_longer_dimensions_still_need_strides_of_whole_vectors(lib):
    x = torch.zeros(4096, device="cuda", dtype=torch.bfloat16)
    for strides in ((1020, 256, 64), (1024, 252, 64), (1024, 256, 68)):
        with pytest.raises(kvq.KVQError):
            kvq.kvq_rope_apply(kvq.Rope(64), torch.as_strided(x, (2, 2, 2, 64), strides + (1,)))
