"""Long prefixes: the tensor cores' fp32 accumulators cut off towards zero at every step, so a chain of steps must not grow with the
prefix.

The values are +a in the first half of the prefix and -a in the second, exact in every format the pass holds them in, so the sums climb
and fall back and the output is a small difference: what the steps cut off stays visible beside its rounding.

Tolerance of an output element: a chain of n steps cuts off at most n 2^-23 of its largest sum, a times the weights of one half, on the
way up and down: n 2^-24 a of the output.  64 tiles of 128 tokens in steps of 16 are n = 512 steps.  Weights are rounded to fp16, each
off by 2^-12 of itself at random: the sum's root mean square is 2^-12 sqrt(sum w^2), six of which are allowed.  The logits' own errors
are 2^-19 sum |q| |k| of a weight at most (and of either sign), times sqrt(sum w^2) as well.  Half a bf16 step: 2^-8 of the element."""
import math

import pytest
import torch

import quantized_kv_speculative_gb300 as kvq
from quantized_kv_speculative_gb300 import _build

A = 1.3359375   # eight bits, as bf16 holds them


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kvq.load_library()


def keys_of(pc, h, G, n):
    """Head h's keys in 64 bits: 2-bit codes, lowest bits first, then the residual."""
    lq = pc.quantized_len
    w = pc.k_plane(0)[h, :lq]
    codes = torch.stack([(w >> (2 * i)) & 3 for i in range(4)], -1).flatten(-2).double()
    s, z = (pc.k_scale_zero()[h, :lq // G, i].double().repeat_interleave(G, 0) for i in range(2))
    r, at = pc.residual_len, torch.arange(pc.residual_len, device="cuda") + pc.residual_start
    k = torch.cat((codes * s + z, pc.residual()[0][h][at % (2 * G)].double()))
    assert k.shape[0] == n == lq + r
    return k, torch.cat((codes * s.abs() + z.abs(), k[lq:].abs()))


@pytest.mark.gpu
@pytest.mark.parametrize("rows,n", [(64, 131072), (16, 262144), (160, 65536 + 77)])
def test_sums_over_a_long_prefix(lib, rows, n):
    sms, D, G, hg = torch.cuda.get_device_properties(0).multi_processor_count, 64, 64, 8
    H = (2 if rows <= 32 else 1) * sms // 2 + 1   # one split of each head fills the device
    B = rows // hg
    g = torch.Generator(device="cuda").manual_seed(n)
    pc = kvq.QuantizedKVCache(1, H, D, G, "int2", n // G * G)
    sign = torch.where(torch.arange(n, device="cuda") < n // 2, 1.0, -1.0)
    for at in range(0, n, 16384):   # (in pieces: the whole as fp32 would take gigabytes)
        m = min(16384, n - at)
        K = torch.randn((1, H, m, D), generator=g, device="cuda", dtype=torch.bfloat16)
        V = (A * sign[at:at + m]).bfloat16()[None, None, :, None].expand(1, H, m, D).contiguous()
        kvq.kvq_quantize_append(pc, K, V)
    gc = kvq.QuantizedKVCache(B, H, D, G, "int2", G)
    q = torch.randn((B, 1, H * hg, D), generator=g, device="cuda").bfloat16()
    out, _ = kvq.kvq_attend_shared(pc, gc, "int2", q)
    chain = 512 * 2.0 ** -24 * A
    for h in (0, H - 1):
        k, size = keys_of(pc, h, G, n)
        for b in range(B):
            for i in range(hg):
                qr = q[b, 0, h * hg + i].double()
                x = k @ qr / math.sqrt(D)
                w = torch.softmax(x, 0)
                want = float((w * sign.double()).sum()) * A
                spread = float((w * w).sum().sqrt()) * A
                logit = 2.0 ** -19 * float((size @ qr.abs()).max()) / math.sqrt(D)
                off = (out[b, 0, h * hg + i].double() - want).abs().max()
                tol = 2.0 ** -8 * abs(want) + chain + (6 * 2.0 ** -12 + logit) * spread
                assert float(off) <= tol, f"head {h} row {b * hg + i}: off by {float(off):.2e} > {tol:.2e} (output {want:.2e})"
