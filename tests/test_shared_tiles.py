"""The pass over a shared prefix with many tiles in one CTA: as many KV heads as the device has SMs leave each CTA the whole prefix
(or half of it, where two CTAs share an SM), so that the rings of codes and of zero terms go round several times, both value buffers
are used again and again, and references move in late tiles.  Every row shape, from 16 to 160 rows.

Tolerance: as in the other tests of kvq_attend_shared (``EXTRA_V`` = 2^-9 of the largest |v|)."""
import pytest
import torch

import kvq_inputs as ki
import oracle
import quantized_kv_speculative_gb300 as kvq
from quantized_kv_speculative_gb300 import _build

from plain_attention import assert_close, attend_plain, slopes_of

EXTRA_V = 2.0 ** -9
HG = 8


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kvq.load_library()


def host(t):
    return ki.bf16_tensor_to_f32(t)


def heads_looked_at(H):
    return [0, H // 2, H - 1]


def filled(fmt, B, H, D, G, n, g, ramp=None):
    """A device cache of n tokens a sequence, and the oracle caches of each sequence's heads looked at."""
    K, V = (torch.randn((B, H, n, D), generator=g, device="cuda") for _ in range(2))
    if ramp is not None:
        K *= ramp[:, None]
    # one sign for each channel and 128 tokens: a tile that is lost, stale or counted twice shows in the outputs
    sign = torch.randint(0, 2, (B, H, n // 128 + 1, D), generator=g, device="cuda") * 2.0 - 1.0
    V = 0.2 * V + sign.repeat_interleave(128, 2)[:, :, :n]
    K, V = K.bfloat16(), V.bfloat16()
    cap = max(G, n // G * G)
    gc = kvq.QuantizedKVCache(B, H, D, G, fmt, cap)
    kvq.kvq_quantize_append(gc, K, V)
    ocs = []
    for b in range(B):
        ocs.append(oracle.OracleCache(1, 3, D, G, fmt, cap))
        ocs[b].append(host(K[b:b + 1, heads_looked_at(H)]), host(V[b:b + 1, heads_looked_at(H)]))
    return gc, ocs


def run(mode, D, G, rows, kind, seed):
    H = torch.cuda.get_device_properties(0).multi_processor_count
    B, fmt = rows // HG, kvq.MODE_FORMAT[mode]
    n0 = (40 if rows <= 32 else 22) * 128 + 77
    g = torch.Generator(device="cuda").manual_seed(seed)
    ramp = torch.linspace(0.3, 10.0, n0, device="cuda") if kind == "growing" else None
    pc, (po,) = filled(fmt, 1, H, D, G, n0, g, ramp)
    gc, ocs = filled(fmt, B, H, D, G, 2, g)
    q = torch.randn((B, 1, H * HG, D), generator=g, device="cuda").bfloat16()
    look = [h * HG + i for h in heads_looked_at(H) for i in range(HG)]
    kw, mod = {}, None
    if kind == "modified":
        first, slopes = [(211 * b) % n0 for b in range(B)], slopes_of(H * HG)
        kw = dict(cap=5.0, window=n0 - 500, slopes=slopes[look], first=first)
        mod = kvq.ScoreMod(5.0, n0 - 500, slopes.cuda(), torch.tensor(first, dtype=torch.int32, device="cuda"))
    ws = kvq.make_shared_workspace(pc, gc, H * HG, 1)
    out, lse = kvq.kvq_attend_shared(pc, gc, mode, q, mod=mod, workspace=ws)
    assert kvq.kvq_workspace_status(ws) == 0
    assert_close(out[:, :, look], lse[:, :, look], attend_plain(ocs, mode, host(q[:, :, look]), prefix=po, **kw), extra_v=EXTRA_V)


@pytest.mark.gpu
@pytest.mark.parametrize("rows", [16, 32, 64, 96, 128, 160])
@pytest.mark.parametrize("mode,D,G", [("int8", 64, 64), ("int4", 64, 32), ("int2", 128, 32), ("int8", 128, 128), ("int1", 128, 64)])
@pytest.mark.parametrize("kind", ["flat", "growing", "modified"])
def test_many_tiles_in_one_cta(lib, mode, D, G, rows, kind):
    """``flat``: all tokens count; ``growing``: the logits' spread grows from 0.3 to 10 along the prefix, so late tiles raise the
    maxima by more than a weight may hold and sums and outputs are rescaled; ``modified``: cap, slopes, window, first positions."""
    run(mode, D, G, rows, kind, seed=rows)
