// Rotary positions of the queries and keys of new tokens (kvq_rope_init,
// kvq_rope_apply): what runs between a model's projections and
// kvq_quantize_append / kvq_attend.
//
// Pair i of a head (channels i and i + rd/2, or 2i and 2i + 1) turns by the
// angle p f_i at position p:
//   a' = m (a cos - b sin),  b' = m (a sin + b cos).
// Angles are kept in turns as 64-bit fixed-point fractions: with
// T_i = frac(f_i / 2 pi) 2^64, the low 64 bits of p T_i are the fraction of a
// turn at position p, whatever whole turns were made, in one integer product.
// The upper 32 bits become a signed fp32 fraction of a turn, so the angle in
// (-pi, pi] is off by 2^-32 of a turn and 2^-24 of itself at every position, and
// by what T_i's 53 bits leave, 2^-53 of a turn a position at most (an fp32 product
// p f_i would be off by 0.03 radians at position 500,000).
//
// Bound by memory: each query and key value is read and written once.  The
// cosines and sines of a token are shared by its heads, so a CTA first fills a
// table of its tokens' pairs (a thread per pair) while its first rows are in
// flight, then rotates whole 16-byte vectors from registers.
//
// Measured on the GB300 (8,192 tokens of 32 + 32 heads of 128 channels, 268 MB):
// CTAs of 128 threads with two vectors each 46.4 us (5.8 TB/s, 0.85 of the
// measured copy rate); of 256 threads with two 50.8 us, with four 55.2 us (short
// CTAs keep more loads in flight around the table's barrier).  Streaming cache
// hints changed nothing.  One token of 64 heads: 1.9 us, its launch.
#include <cmath>
#include <cstring>

#include "kvq_device.cuh"

using namespace kvq;

namespace {

constexpr uint32_t kRopeMagic = 0x52505131u;   // "RPQ1"
constexpr int kMaxPairs = 64;
constexpr int kRopeThreads = 128;
constexpr int kRopeTokens = 16;                // tokens of a CTA at most (bounds the table)
constexpr int kRopeItems = 2;                  // vectors of a thread in flight

struct RopeParams {
  const uint16_t* in[2];     // queries, keys
  uint16_t* out[2];          // [B][n][Hq][D], [B][Hkv][n][D]
  long long sb[2], st[2], sh[2];   // input strides in elements: sequence, token, head
  int heads[2];
  const int32_t* pos;        // [B][n] or null
  long long pos0;            // null positions: token i is at pos0 + i
  int B, n, D, rd;
  int tokens;                // tokens per CTA
  int slice;                 // heads per CTA
  float magnitude;
  uint64_t turns[kMaxPairs];
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// A vector is VW pairs of one head (VW = 8 where the rotated part has a
// multiple of 16 channels, else 4), or 2 VW channels past the rotated part.
template <int VW>
struct Vec {
  uint32_t w[VW];
};

template <int N>   // N 32-bit words, 8- or 16-byte aligned
__device__ __forceinline__ void load_words(const uint16_t* p, uint32_t* w) {
  if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x; w[1] = v.y;
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint4 v = reinterpret_cast<const uint4*>(p)[i];
      w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
    }
  }
}
template <int N>
__device__ __forceinline__ void store_words(uint16_t* p, const uint32_t* w) {
  if constexpr (N == 2) {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  } else {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  }
}

template <int VW, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
  // (m cos, m sin) of token x pair, read two pairs at a time
  __shared__ __align__(sizeof(float4)) float2 table[kRopeTokens * kMaxPairs];
  static_assert(__alignof__(table) >= sizeof(float4) && kMaxPairs % 2 == 0, "a token's pairs start at a vector of four floats");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int tid = threadIdx.x;
  const int pairs = p.rd / 2, rot = p.rd / (2 * VW);
  const int lv = __ffs(p.D / (2 * VW)) - 1;                 // log2 of the vectors of a head
  const int H = p.heads[0] + p.heads[1];
  const unsigned n = p.n, ntok = static_cast<unsigned>(p.B) * n, tok0 = blockIdx.x * static_cast<unsigned>(p.tokens);   // below 2^31
  const int nt = static_cast<int>(min(static_cast<unsigned>(p.tokens), ntok - tok0));
  const int h0 = blockIdx.y * p.slice, nh = min(p.slice, H - h0);
  const int total = nt * nh << lv;

  bool filled = false;
  for (int base = tid; base - tid < total; base += kRopeThreads * kRopeItems) {
    Vec<VW> x[kRopeItems];
    uint16_t* dst[kRopeItems];
    int tv[kRopeItems];      // token << 8 | vector; -1: none
#pragma unroll
    for (int k = 0; k < kRopeItems; ++k) {
      const int e = base + k * kRopeThreads;
      tv[k] = -1;
      if (e >= total) continue;
      const int r = e >> lv, v = e - (r << lv);
      const int t = nt == 1 ? 0 : r / nh, hh = h0 + (r - t * nh);
      const int which = hh >= p.heads[0], h = hh - (which ? p.heads[0] : 0);
      const unsigned tok = tok0 + t, b = tok / n, i = tok - b * n;
      const uint16_t* src = p.in[which] + b * p.sb[which] + i * p.st[which] + h * p.sh[which];
      const long long row = which ? (static_cast<long long>(b) * p.heads[1] + h) * n + i : static_cast<long long>(tok) * p.heads[0] + h;
      dst[k] = p.out[which] + row * p.D;
      tv[k] = t << 8 | v;
      if (INTER || v >= rot) {
        load_words<VW>(src + v * 2 * VW, x[k].w);
      } else {
        load_words<VW / 2>(src + v * VW, x[k].w);
        load_words<VW / 2>(src + pairs + v * VW, x[k].w + VW / 2);
      }
    }
    if (!filled) {   // the same in every thread; the first rows are in flight
      for (int e = tid; e < nt * pairs; e += kRopeThreads) {
        const int t = e / pairs, i = e - t * pairs;
        const unsigned tok = tok0 + t;
        const long long pos = p.pos ? p.pos[tok] : p.pos0 + tok % n;
        const uint64_t ph = static_cast<uint64_t>(pos) * p.turns[i];
        const float turn = static_cast<float>(static_cast<int32_t>(ph >> 32)) * 0x1p-31f;   // half turns in [-1, 1)
        float s, c;
        sincospif(turn, &s, &c);
        table[t * kMaxPairs + i] = make_float2(c * p.magnitude, s * p.magnitude);
      }
      __syncthreads();
      filled = true;
    }
#pragma unroll
    for (int k = 0; k < kRopeItems; ++k) {
      if (tv[k] < 0) continue;
      const int t = tv[k] >> 8, v = tv[k] & 255;
      if (v >= rot) {
        store_words<VW>(dst[k] + v * 2 * VW, x[k].w);
        continue;
      }
      const float4* cs = reinterpret_cast<const float4*>(table + t * kMaxPairs + v * VW);
      uint32_t y[VW];
#pragma unroll
      for (int j = 0; j < VW / 2; ++j) {   // pairs 2j, 2j + 1
        const float4 f = cs[j];
        if constexpr (INTER) {
          const float a0 = bf_lo(x[k].w[2 * j]), b0 = bf_hi(x[k].w[2 * j]);
          const float a1 = bf_lo(x[k].w[2 * j + 1]), b1 = bf_hi(x[k].w[2 * j + 1]);
          y[2 * j] = pack_bf16(a0 * f.x - b0 * f.y, a0 * f.y + b0 * f.x);
          y[2 * j + 1] = pack_bf16(a1 * f.z - b1 * f.w, a1 * f.w + b1 * f.z);
        } else {
          const uint32_t a = x[k].w[j], b = x[k].w[VW / 2 + j];
          y[j] = pack_bf16(bf_lo(a) * f.x - bf_lo(b) * f.y, bf_hi(a) * f.z - bf_hi(b) * f.w);
          y[VW / 2 + j] = pack_bf16(bf_lo(a) * f.y + bf_lo(b) * f.x, bf_hi(a) * f.w + bf_hi(b) * f.z);
        }
      }
      if constexpr (INTER) {
        store_words<VW>(dst[k] + v * 2 * VW, y);
      } else {
        store_words<VW / 2>(dst[k] + v * VW, y);
        store_words<VW / 2>(dst[k] + pairs + v * VW, y + VW / 2);
      }
    }
  }
}

template <int VW, bool INTER>
cudaError_t launch_rope(const RopeParams& p, dim3 grid, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kRopeThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rope_kernel<VW, INTER>, p);
}

bool finite_positive(double x) { return std::isfinite(x) && x > 0; }

bool valid_rope_desc(const kvq_rope_desc* d) {
  if (d->head_dim != 64 && d->head_dim != 128) return false;
  if (d->rotary_dim < 8 || d->rotary_dim > d->head_dim || d->rotary_dim % 8) return false;
  if (d->layout != KVQ_ROPE_HALF && d->layout != KVQ_ROPE_INTERLEAVED) return false;
  if (d->scaling < KVQ_ROPE_UNSCALED || d->scaling > KVQ_ROPE_BANDS) return false;
  if (!finite_positive(d->base) || d->base <= 1.0 || !std::isfinite(static_cast<float>(d->magnitude))) return false;
  if (d->scaling != KVQ_ROPE_UNSCALED && !finite_positive(d->factor)) return false;
  if (d->scaling == KVQ_ROPE_RAMP || d->scaling == KVQ_ROPE_BANDS) {
    if (!finite_positive(d->original_len) || !finite_positive(d->low) || !finite_positive(d->high) || d->high <= d->low) return false;
  }
  return true;
}

constexpr double kTwoPi = 6.283185307179586476925286766559;

constexpr int64_t kMaxStride = int64_t{1} << 40;   // elements
constexpr double kMaxExtent = 0x1p47;             // bytes of an input, first to last

// Extent of a strided [B][n][heads][D] tensor in bytes; its strides are at most kMaxStride.
double extent_bytes(const int64_t* st, int B, int n, int heads, int D) {
  return 2.0 * ((B - 1.0) * st[0] + (n - 1.0) * st[1] + (heads - 1.0) * st[2] + D);
}

struct Range {
  uintptr_t lo, hi;
};
bool overlap(const Range& a, const Range& b) { return a.lo < b.hi && b.lo < a.hi; }

}  // namespace

extern "C" {

kvq_status kvq_rope_init(kvq_rope* rope, const kvq_rope_desc* d, const double* inv_freq) {
  if (!rope || !d || !valid_rope_desc(d)) return KVQ_ERR_INVALID_ARG;
  const int rd = d->rotary_dim, pairs = rd / 2;
  double f[kMaxPairs];
  for (int i = 0; i < pairs; ++i) {
    f[i] = inv_freq ? inv_freq[i] : std::pow(d->base, -2.0 * i / rd);
    if (!std::isfinite(f[i])) return KVQ_ERR_INVALID_ARG;
  }
  // w: the share of the unscaled frequency that a pair keeps
  const double span = 2.0 * std::log(d->base);
  const double at_high = rd * std::log(d->original_len / (d->high * kTwoPi)) / span;
  const double at_low = rd * std::log(d->original_len / (d->low * kTwoPi)) / span;
  for (int i = 0; i < pairs; ++i) {
    double w = 1.0;
    if (d->scaling == KVQ_ROPE_LINEAR) {
      w = 0.0;
    } else if (d->scaling == KVQ_ROPE_RAMP) {
      const double lo = std::fmax(0.0, std::floor(at_high)), hi = std::fmin(rd - 1.0, std::ceil(at_low));
      w = 1.0 - std::fmin(1.0, std::fmax(0.0, (i - lo) / std::fmax(hi - lo, 1e-3)));
    } else if (d->scaling == KVQ_ROPE_BANDS) {
      w = std::fmin(1.0, std::fmax(0.0, (d->original_len * std::fabs(f[i]) / kTwoPi - d->low) / (d->high - d->low)));
    }
    if (w < 1.0) f[i] = f[i] * w + f[i] / d->factor * (1.0 - w);
    if (!std::isfinite(f[i])) return KVQ_ERR_INVALID_ARG;   // a factor near 0
  }
  std::memset(rope, 0, sizeof(*rope));
  rope->desc = *d;
  for (int i = 0; i < pairs; ++i) {
    // frac(f / 2 pi) as a 64-bit fraction: the upper 32 bits, then the rest (both steps exact)
    double t = f[i] / kTwoPi;
    t -= std::floor(t);
    const double up = std::floor(t * 0x1p32);
    rope->turns[i] = (static_cast<uint64_t>(up) << 32) + static_cast<uint64_t>((t * 0x1p32 - up) * 0x1p32);
  }
  rope->magic = kRopeMagic;
  return KVQ_OK;
}

kvq_status kvq_rope_apply(const kvq_rope* rope, const void* q, const int64_t* q_strides, int32_t num_q_heads, void* q_out,
                          const void* k, const int64_t* k_strides, int32_t num_kv_heads, void* k_out,
                          const int32_t* positions, int64_t first_position, int32_t batch, int32_t n_tokens,
                          kvq_stream_t stream) {
  if (!rope || rope->magic != kRopeMagic) return KVQ_ERR_NOT_INITIALIZED;
  const int D = rope->desc.head_dim;
  const int heads[2] = {num_q_heads, num_kv_heads};
  const void* in[2] = {q, k};
  void* out[2] = {q_out, k_out};
  const int64_t* strides[2] = {q_strides, k_strides};
  if (batch < 1 || n_tokens < 0 || heads[0] < 0 || heads[1] < 0 || heads[0] > 65536 || heads[1] > 65536 || heads[0] + heads[1] < 1)
    return KVQ_ERR_INVALID_ARG;
  if (static_cast<int64_t>(batch) * n_tokens >= (int64_t{1} << 31)) return KVQ_ERR_INVALID_ARG;
  if (positions && (reinterpret_cast<uintptr_t>(positions) & 3u)) return KVQ_ERR_INVALID_ARG;
  if (!positions && (first_position < 0 || first_position > (int64_t{1} << 31))) return KVQ_ERR_INVALID_ARG;
  RopeParams p{};
  Range rin[2] = {}, rout[2] = {};
  for (int w = 0; w < 2; ++w) {
    if (heads[w] == 0) continue;
    if (n_tokens == 0) continue;
    if (!in[w] || !out[w] || !strides[w] || (reinterpret_cast<uintptr_t>(in[w]) & 15u) || (reinterpret_cast<uintptr_t>(out[w]) & 15u))
      return KVQ_ERR_INVALID_ARG;
    int64_t st[3];   // nothing steps along a dimension of one entry, whatever its stride
    const int size[3] = {batch, n_tokens, heads[w]};
    for (int a = 0; a < 3; ++a) {
      st[a] = size[a] > 1 ? strides[w][a] : 0;
      if (st[a] < 0 || st[a] % 8 || st[a] > kMaxStride) return KVQ_ERR_INVALID_ARG;
    }
    const double ext = extent_bytes(st, batch, n_tokens, heads[w], D);
    if (ext > kMaxExtent) return KVQ_ERR_INVALID_ARG;
    p.in[w] = static_cast<const uint16_t*>(in[w]);
    p.out[w] = static_cast<uint16_t*>(out[w]);
    p.sb[w] = st[0];
    p.st[w] = st[1];
    p.sh[w] = st[2];
    rin[w] = {reinterpret_cast<uintptr_t>(in[w]),
              reinterpret_cast<uintptr_t>(in[w]) + static_cast<uintptr_t>(ext)};
    rout[w] = {reinterpret_cast<uintptr_t>(out[w]),
               reinterpret_cast<uintptr_t>(out[w]) + 2ull * batch * n_tokens * heads[w] * D};
  }
  if (n_tokens == 0) return KVQ_OK;
  // An output may take the place of its own input in the same layout and
  // touches no other tensor of the call.
  for (int w = 0; w < 2; ++w) {
    if (heads[w] == 0) continue;
    if (overlap(rout[w], rin[w])) {
      const int64_t hs = w ? static_cast<int64_t>(n_tokens) * D : D, ts = w ? D : static_cast<int64_t>(heads[w]) * D;
      const bool same = in[w] == out[w] && (heads[w] == 1 || p.sh[w] == hs) && (n_tokens == 1 || p.st[w] == ts) &&
                        (batch == 1 || p.sb[w] == static_cast<int64_t>(heads[w]) * n_tokens * D);
      if (!same) return KVQ_ERR_INVALID_ARG;
    }
    if (heads[1 - w] > 0 && (overlap(rout[w], rin[1 - w]) || overlap(rout[w], rout[1 - w]))) return KVQ_ERR_INVALID_ARG;
  }
  p.heads[0] = heads[0];
  p.heads[1] = heads[1];
  p.pos = positions;
  p.pos0 = first_position;
  p.B = batch;
  p.n = n_tokens;
  p.D = D;
  p.rd = rope->desc.rotary_dim;
  p.magnitude = static_cast<float>(rope->desc.magnitude);
  std::memcpy(p.turns, rope->turns, sizeof(p.turns));
  const int vw = p.rd % 16 == 0 ? 8 : 4;
  const long long vph = D / (2 * vw), H = heads[0] + heads[1], ntok = static_cast<long long>(batch) * n_tokens;
  // A CTA takes 256 vectors (two a thread): several tokens of few heads, or some
  // of a token's heads; calls that would leave SMs idle take 128.
  const long long sms = device_sm_count() > 0 ? device_sm_count() : 152;
  const long long per = ntok * H * vph >= sms * kRopeThreads * kRopeItems ? kRopeThreads * kRopeItems : kRopeThreads;
  p.tokens = static_cast<int>(std::fmin(kRopeTokens, std::fmax(1, per / (H * vph))));
  p.slice = static_cast<int>(std::fmin(static_cast<double>(H), std::fmax(1, per / vph)));
  const dim3 grid(static_cast<unsigned>((ntok + p.tokens - 1) / p.tokens), static_cast<unsigned>((H + p.slice - 1) / p.slice), 1);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool inter = rope->desc.layout == KVQ_ROPE_INTERLEAVED;
  const cudaError_t e = vw == 8 ? (inter ? launch_rope<8, true>(p, grid, s) : launch_rope<8, false>(p, grid, s))
                                : (inter ? launch_rope<4, true>(p, grid, s) : launch_rope<4, false>(p, grid, s));
  return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA;
}

}  // extern "C"
