"""Small values behind tokens that carry none: the scale by which a run of tokens holds its weights is chosen from the tokens that
count, wherever in the run the first of them stands.

Tolerance: ``assert_close`` is relative to the largest |v| that a row sees, so it is the same for values of any size."""
import numpy as np
import pytest
import torch

import kvq_inputs as ki
import oracle
import quantized_kv_speculative_gb300 as kvq
from quantized_kv_speculative_gb300 import _build

from plain_attention import assert_close, attend_plain

HEADS = 256   # so many that a split is long: each of its warps runs through several steps of 32 tokens
LOOK = [0, 100, 255]


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kvq.load_library()


def dev(x):
    return ki.f32_to_bf16_tensor(x, "cuda")


def build(mode, n, D, G, size, flat=0, seed=0):
    """One sequence of n tokens and HEADS KV heads with values of about ``size``, the first ``flat`` of them zero; the oracle holds
    the heads LOOK."""
    fmt = kvq.MODE_FORMAT[mode]
    g = torch.Generator(device="cuda").manual_seed(seed)
    K, V = (torch.randn((1, HEADS, n, D), generator=g, device="cuda") for _ in range(2))
    K, V = K.bfloat16(), (V * size).bfloat16()
    V[:, :, :flat] = 0
    gc, oc = kvq.QuantizedKVCache(1, HEADS, D, G, fmt, n // G * G), oracle.OracleCache(1, len(LOOK), D, G, fmt, n // G * G)
    kvq.kvq_quantize_append(gc, K, V)
    oc.append(ki.bf16_tensor_to_f32(K[:, LOOK]), ki.bf16_tensor_to_f32(V[:, LOOK]))
    return gc, oc


def rows(hg):
    return [h * hg + i for h in LOOK for i in range(hg)]


def queries(seed, gamma, hg, D):
    """For all heads on the device, and for those of LOOK."""
    q = ki.queries(seed, 1, gamma, HEADS * hg, D)
    return dev(q), q[:, :, rows(hg)]


def check(out, lse, plain, hg):
    assert_close(out[:, :, rows(hg)], lse[:, :, rows(hg)], plain)


SHAPES = [("int8", 4, 128, 32, 2), ("int8", 1, 128, 128, 1), ("int4", 1, 64, 32, 4), ("int4", 8, 128, 64, 1), ("int2", 4, 128, 32, 2),
          ("int1", 4, 128, 128, 1), ("int1c", 2, 64, 64, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("mode,hg,D,G,gamma", SHAPES)
@pytest.mark.parametrize("size", [1e-3, 1e-6])
@pytest.mark.parametrize("edge", [32, 64, 100, 127])
def test_hidden_tokens_ahead_of_small_values(lib, mode, hg, D, G, gamma, size, edge):
    """The first visible position stands ``edge`` tokens behind a split's start: 32-token steps that no row sees come first."""
    n, low = 3000, 512 + edge
    gc, oc = build(mode, n, D, G, size)
    qd, q = queries(1, gamma, hg, D)
    window = n - gamma - low + 1   # the first row's reaches down to ``low``
    for kw, mod in ((dict(first=[low]), kvq.ScoreMod(first=torch.tensor([low], dtype=torch.int32, device="cuda"))),
                    (dict(window=window), kvq.ScoreMod(window=window))):
        out, lse = kvq.kvq_attend_mod(gc, mode, qd, mod)
        check(out, lse, attend_plain([oc], mode, q, **kw), hg)


@pytest.mark.gpu
@pytest.mark.parametrize("mode,hg,D,G,gamma", SHAPES)
@pytest.mark.parametrize("size", [1e-3, 1e-6])
def test_zero_values_ahead_of_small_ones(lib, mode, hg, D, G, gamma, size):
    """A padded prompt's values are zero, and so are their scales: in every form of the attention."""
    gc, oc = build(mode, 2500, D, G, size, flat=70)
    qd, q = queries(2, gamma, hg, D)
    plain = attend_plain([oc], mode, q)
    check(*kvq.kvq_attend(gc, mode, qd), plain, hg)
    check(*kvq.kvq_attend_mod(gc, mode, qd, kvq.ScoreMod()), plain, hg)
    if mode != "int8":
        out, lse, _, _ = kvq.kvq_attend_topk(gc, mode, qd, 8, score_row=0)
        check(out, lse, plain, hg)


@pytest.mark.gpu
def test_values_that_are_all_equal(lib):
    """No token has a scale: the zero points alone make the output."""
    n, D = 700, 64
    K, _ = ki.kv_stream(3, 1, 2, n, D)
    V = np.full_like(K, 0.75)
    gc, oc = kvq.QuantizedKVCache(1, 2, D, 32, "hier8", 704), oracle.OracleCache(1, 2, D, 32, "hier8", 704)
    kvq.kvq_quantize_append(gc, dev(K), dev(V))
    oc.append(K, V)
    q = ki.queries(4, 1, 2, 4, D)
    plain = attend_plain([oc], "int8", q)
    for out, lse in (kvq.kvq_attend(gc, "int8", dev(q)), kvq.kvq_attend_mod(gc, "int8", dev(q), kvq.ScoreMod())):
        assert_close(out, lse, plain)
        assert torch.all(out == 0.75)
