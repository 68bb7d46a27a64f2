// The rows of every sequence against one shared prefix cache, on the 5th
// generation tensor cores (the first part of kvq_attend_shared).
//
// For a KV head the B gamma (Hq / Hkv) query rows attend the same tokens.  A CTA
// takes a tile of up to 160 rows and a split of the prefix's tiles of 128
// tokens.  Both products put the low-bit operand on the 128 TMEM lanes:
//   S^T [token, row]   = K [token, channel] Q^T          (A = keys, B = queries)
//   O^T [channel, row] = V^T [channel, token] P^T        (A = values, B = weights)
// so the codes go from shared memory through registers straight into TMEM as
// the A operand (one lane a token, or a channel: the planes' own layouts), and
// the cost of a product falls with the rows down to N = 16.  (Measured, 64
// products back to back: 19, 20, 34 and 63 cycles each at N = 16, 32, 64 and
// 128 with A in TMEM; 41 to 65 with A in shared memory.)
//
// Phases.  Eight warps (up to 32 rows, two CTAs an SM) or sixteen (one) turn the
// values of tile j into f16, take the softmax of its logits, then turn the keys
// of tile j + 1, all of them the same code at a time; one warp issues the
// products and one copies tiles ahead (1-D bulk copies into a ring).  S(j + 1)
// runs on the tensor cores while the values of j + 1 are turned, P V (j) while
// its keys are.  Warps of fixed roles instead (dequantizers, softmax groups)
// took twice the time: their code together does not fit the SM's instruction
// cache, and waiting warps' polls took a quarter of the issue slots.  Keys and
// values turned in one phase, or two halves of the warps in opposite phases,
// took 5 to 20% longer.
//
// Bound by the phases' latency: of the 4,500 cycles of a tile at 96 rows (INT2,
// G = 32) some 1,250 each go to keys, values and the softmax, one after another, at
// 2.4 instructions a cycle of an SM (of 4); the tensor cores are busy for a fifth,
// HBM for less.  Fewer instructions alone no longer help (35 of 800 a warp and tile:
// nothing); phases that overlap would.  Measured on the GB300 in a
// graph (both launches): 16 rows x 32 heads over 8K INT4 tokens 32 us; 288 rows x
// 8 heads over 32K INT2 tokens 102 us (0.38 PFLOP/s of the two products, 0.57 with
// the keys' second part; in tiles of 96 rows, each of which turns the codes again,
// 111); 128 rows x 8 heads over 128K INT8 tokens, capped, 217 us
// (1.3 TB/s; 0.32 and 0.48 PFLOP/s).
//
// Precision.  With c' = c - c0 (c0 the middle code), a key is
// s c' + (z + c0 s).  The part s c' is held exactly to 22 bits: hi = f16(c' s_hi)
// and lo = f16(c' s_hi - hi + c' s_lo), the first difference exact by one fused
// multiply-add, both multiplied with Q.  The part q.(z + c0 s) is one number
// per row and key group: a small launch ahead (zero_kernel) leaves them in the
// workspace, and each tile's arrive with its codes.  Q is bf16, exact in f16
// after a power of two of the row's own.  Values and weights are one f16 each: off by
// 2^-12 to 2^-11 of themselves at random, where the splits of kvq_attend keep codes
// exact and weights in two parts.  Against 64 bits that makes the output 1% less
// exact (1.66e-3 -> 1.68e-3 of its size at 32K, nearly all of it bf16's rounding);
// second parts would double the products and the stores into TMEM.  Weighted values
// are summed in TMEM over a split, in steps of 16 tokens that are cut off towards
// zero: at most 2^-23 of the sum each, 2e-5 of |v| measured over 512 steps, 7e-5 over
// 8,192 and 1.4e-4 over 16,384 (sums that climb and fall back).  The plan keeps a
// split at 512 steps as long as 64 splits allow (270,000 tokens at least).
//
// Softmax.  Row maxima run across lanes here, so they are looked at only when
// needed: a row keeps a reference m and its weights are 2^(x - m), m set 4 below
// the maximum when it was last looked at; a thread that meets x - m > 15.5 votes
// for a new look (one barrier a tile carries the votes), upon which the maxima
// are reduced and sums and outputs rescaled.  Weights stay below f16's 2^16, and
// those 2^-28 below the largest still count.
#include <limits.h>

#include "kvq_modes.cuh"

namespace kvq {
namespace {

constexpr int kTile = kSharedTile;
// A CTA's shape by the rows that it can hold.  Up to 32 rows: 8 working warps,
// half of the TMEM and of the shared memory, two CTAs an SM, whose phases fill
// each other's waits.  More: 16 working warps, one CTA an SM.  Past 128 rows the
// TMEM holds one value buffer, not two.
template <int NR>
struct Shape {
  static constexpr int WORK = NR <= 32 ? 8 : 16, GROUPS = WORK / 4;   // working warps, in groups of four
  static constexpr int MMA = WORK, COPY = WORK + 1, THREADS = (WORK + 2) * 32;
  static constexpr int CTAS = NR <= 32 ? 2 : 1, VB = NR <= 32 || NR > 128 ? 1 : 2;   // CTAs an SM, value buffers
  // TMEM columns: K hi and lo parts, values, S, O
  static constexpr uint32_t T_K = 0, T_V = 128, T_S = T_V + VB * 64, T_O = T_S + (NR <= 32 ? 32 : NR <= 128 ? 128 : NR), T_ALL = 512 / CTAS;
  static_assert(T_O + (T_O - T_S) <= T_ALL, "TMEM columns");
};
constexpr float kRefBelow = 4.f;        // a row's reference lies this far below its maximum when set
constexpr float kVoteAbove = 15.5f;     // an exponent above this asks for a new reference
constexpr float kNoRef = -1e30f;        // no token seen yet

// ------------------------------------------------------------------------------
// tcgen05
// ------------------------------------------------------------------------------
__device__ __forceinline__ void tm_alloc(uint32_t* dst, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
}
__device__ __forceinline__ void tm_dealloc(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void tm_ld8(uint32_t addr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]));   // no memory clobber: loads move past it
}
// The loaded registers become valid here (the asm ties them to the wait).
__device__ __forceinline__ void tm_wait_ld(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}
__device__ __forceinline__ void tm_st8(uint32_t addr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]),
               "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tm_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// D [128 lanes x N columns] (+)= A (TMEM, 128 x 16 f16) * B (shared memory, 16 x N f16)
__device__ __forceinline__ void tm_mma(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(add))
      : "memory");
}
__device__ __forceinline__ void tm_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// Shared-memory matrix descriptor, 128-byte swizzle: `sbo` bytes between the
// 8-row (K-major) or 8-k (row-major) blocks, `lbo` between row-major blocks of 64 rows.
__device__ __forceinline__ uint64_t mat_desc(uint32_t addr, uint32_t sbo, uint32_t lbo) {
  return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lbo >> 4) << 16) | (static_cast<uint64_t>(sbo >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// f16 inputs, fp32 result, M = 128; B row-major (its rows contiguous) if `mn`.
__device__ __forceinline__ uint32_t instr_desc(int n, bool mn) {
  return (1u << 4) | (mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(n / 8) << 17) | (8u << 24);
}

// Tries until the phase completes, at most 64 times: few instructions a try,
// since the waiting warps share their issue slots with the working ones.
__device__ __forceinline__ bool try_wait_64(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, 64;\n\t"
      "AGAIN%=:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "sub.u32 n, n, 1;\n\t"
      "setp.ne.and.u32 q, n, 0, !p;\n\t"
      "@q bra AGAIN%=;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Further tries, up to the limit; gives up once another thread has.
__device__ __noinline__ void wait_slow(uint64_t* bar, uint32_t parity, long long limit, int* status, volatile int* abort_flag) {
  const long long t0 = clock64();
  while (!try_wait_64(bar, parity)) {
    if (*abort_flag) return;
    if (clock64() - t0 > limit) {
      record_status(status, KVQ_ERR_DEVICE_TIMEOUT);
      *abort_flag = 1;
      return;
    }
  }
}

__device__ __forceinline__ void named_sync(int id) { asm volatile("bar.sync %0, 128;" ::"r"(id) : "memory"); }
__device__ __forceinline__ bool named_or(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(v)), "r"(id)
      : "memory");
  return r != 0;
}

__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<__half2*>(&v); }
__device__ __forceinline__ uint32_t as_u32(__half2 v) { return *reinterpret_cast<uint32_t*>(&v); }

// The power of two 2^e with x 2^-e in [2^13, 2^14) (1 for zero), e within
// [-100, 100]; NaN and infinity give the largest.
__device__ __forceinline__ int norm_exp(float x) {
  const int b = static_cast<int>((__float_as_uint(x) >> 23) & 0xFF);
  return x == 0.f ? 0 : max(-100, min(100, b - 127 - 13));
}

// ------------------------------------------------------------------------------
// Codes to centred f16 pairs.  A 16-bit word 0x6400 | m is 1024 + m, so an AND
// and OR (one LOP3) with the code at bits 2^k gives 1024 + c 2^k, and one fused
// multiply-add c - c0, exactly.  Index kk of a row of 8 / pb codes a byte holds
// code perm(kk); `code_slot` is the inverse.
// ------------------------------------------------------------------------------
template <int MODE>
struct Codes {
  static constexpr int C0 = MODE == KVQ_MODE_INT8 ? 128 : (MODE == KVQ_MODE_INT4 ? 8 : (MODE == KVQ_MODE_INT2 ? 2 : 0));
  static constexpr int CMAX = MODE == KVQ_MODE_INT8 ? 255 : (MODE == KVQ_MODE_INT4 ? 15 : (MODE == KVQ_MODE_INT2 ? 3 : 1));
  static constexpr int CABS = MODE == KVQ_MODE_INT1 ? 1 : C0;            // largest |c - c0|
  static constexpr int WPC = MODE == KVQ_MODE_INT8 ? 4 : Mode<MODE>::PB;   // words (a plane) of 32 codes
};

template <int MODE>
__device__ __forceinline__ constexpr int code_slot(int c) {
  if constexpr (MODE == KVQ_MODE_INT8) return (c & ~7) + ((c & 1) << 2) + ((c & 7) >> 1);
  else if constexpr (MODE == KVQ_MODE_INT4) return (c & ~7) + ((c & 3) << 1) + ((c >> 2) & 1);
  else if constexpr (MODE == KVQ_MODE_INT2) return (c & ~15) + ((c & 7) << 1) + ((c >> 3) & 1);
  else return (c & ~31) + ((c & 15) << 1) + ((c >> 4) & 1);
}
// The inverse: code of slot kk.
template <int MODE>
__device__ __forceinline__ constexpr int slot_code(int kk) {
  const int e = kk & 1;
  if constexpr (MODE == KVQ_MODE_INT8) return (kk & ~7) + 2 * (kk & 3) + ((kk >> 2) & 1);
  else if constexpr (MODE == KVQ_MODE_INT4) return (kk & ~7) + ((kk & 7) >> 1) + 4 * e;
  else if constexpr (MODE == KVQ_MODE_INT2) return (kk & ~15) + ((kk & 15) >> 1) + 8 * e;
  else return (kk & ~31) + ((kk & 31) >> 1) + 16 * e;
}

// 32 codes (the words of one or both planes) to 16 pairs c - c0 in slot order.
template <int MODE>
__device__ __forceinline__ void centred(const uint32_t* h, const uint32_t* l, uint32_t (&c)[16]) {
  constexpr uint32_t M = 0x64006400u;
  if constexpr (MODE == KVQ_MODE_INT8) {
    const __half2 off = __float2half2_rn(-1024.f - Codes<MODE>::C0);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const uint32_t E = ((h[w] << 4) & 0xF0F0F0F0u) | (l[w] & 0x0F0F0F0Fu);
      const uint32_t O = (h[w] & 0xF0F0F0F0u) | ((l[w] >> 4) & 0x0F0F0F0Fu);
      c[4 * w] = as_u32(__hadd2(as_half2(__byte_perm(E, M, 0x7170)), off));
      c[4 * w + 1] = as_u32(__hadd2(as_half2(__byte_perm(E, M, 0x7372)), off));
      c[4 * w + 2] = as_u32(__hadd2(as_half2(__byte_perm(O, M, 0x7170)), off));
      c[4 * w + 3] = as_u32(__hadd2(as_half2(__byte_perm(O, M, 0x7372)), off));
    }
  } else {
    constexpr int PB = Mode<MODE>::PB, PW = 16 / PB;   // pairs of a word
    constexpr int LOW = 8 / PB;                        // of them below bit 8
#pragma unroll
    for (int w = 0; w < 16 / PW; ++w) {
      const uint32_t t = h[w] >> 8;
#pragma unroll
      for (int n = 0; n < PW; ++n) {
        const int k = PB * (n % LOW);
        const uint32_t mask = ((1u << PB) - 1u) * 0x00010001u << k;
        const uint32_t x = ((n < LOW ? h[w] : t) & mask) | M;
        const float f = 1.f / static_cast<float>(1 << k);
        c[PW * w + n] = as_u32(__hfma2(as_half2(x), __float2half2_rn(f), __float2half2_rn(-1024.f * f - Codes<MODE>::C0)));
      }
    }
  }
}

// The words of 32 codes at `src`, both planes.
template <int MODE>
__device__ __forceinline__ void load_codes(const uint8_t* src, int plane, uint32_t (&h)[4], uint32_t (&l)[4]) {
  if constexpr (Codes<MODE>::WPC == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(src);
    h[0] = v.x; h[1] = v.y; h[2] = v.z; h[3] = v.w;
    if constexpr (Mode<MODE>::NP == 2) {
      const uint4 w = *reinterpret_cast<const uint4*>(src + plane);
      l[0] = w.x; l[1] = w.y; l[2] = w.z; l[3] = w.w;
    }
  } else if constexpr (Codes<MODE>::WPC == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(src);
    h[0] = v.x; h[1] = v.y;
  } else {
    h[0] = *reinterpret_cast<const uint32_t*>(src);
  }
}

// ------------------------------------------------------------------------------
// Shared memory
// ------------------------------------------------------------------------------
template <int D, int NR>   // NR: rows of a CTA (16, 32, 64, 96, 128 or 160)
struct SharedSmem {
  static constexpr int ZB = 4;                          // tiles of zero terms in their ring
  static constexpr int Q_OFF = 0;                       // [D / 64][NR rows][128 B], swizzled
  static constexpr int W = Shape<NR>::WORK;
  static constexpr int P_OFF = Q_OFF + NR * D * 2;      // [NR / 64][128 tokens][64 rows] f16, swizzled
  static constexpr int P_BLOCK = kTile * 64 * 2;
  static constexpr int Z_OFF = P_OFF + (NR + 63) / 64 * P_BLOCK;   // [ZB][4 groups][NR] f32
  static constexpr int Z_BUF = 4 * NR * 4;
  static constexpr int ZC_OFF = Z_OFF + ZB * Z_BUF;         // two constant rows: zeros, minus infinity
  static constexpr int KT_OFF = ZC_OFF + 2 * NR * 4;        // [16 warps][16] (s_hi, s_lo) pairs
  static constexpr int VT_OFF = KT_OFF + W * 128;       // [16 warps][16] (s, z) pairs
  static constexpr int KF_OFF = VT_OFF + W * 128;       // [2][128] logit factor of a tile's lane
  static constexpr int ROW_OFF = KF_OFF + 2 * 128 * 4;      // [6][NR]: minus the reference, alpha, low, query position, slope, query factor
  static constexpr int WM_OFF = ROW_OFF + 6 * NR * 4;       // [4 warps][NR]
  static constexpr int MISC_OFF = WM_OFF + 4 * NR * 4;      // scalars, then the barriers
  static constexpr int BAR_OFF = MISC_OFF + 128;
  static constexpr int STAGE_OFF = (BAR_OFF + 256 + 127) / 128 * 128;
  static constexpr int LIMIT = Shape<NR>::CTAS == 2 ? 113 * 1024 : 227 * 1024;
  static constexpr int MAX_STAGES = 8;
  static_assert(W * 8 * 33 * 4 <= (NR + 63) / 64 * P_BLOCK + ZB * Z_BUF, "the last sums fit the weights' buffer and the zero terms behind it");
};

// Byte offsets inside a stage; G is a run-time value.
template <int MODE, int D>
struct StageMap {
  static constexpr int KROW = D * Mode<MODE>::PB / 8, VROW = 32 * Mode<MODE>::PB / 8;
  static constexpr int KPLANE = kTile * KROW, VPLANE = (kTile / 32) * D * VROW;
  static constexpr int V_OFF = Mode<MODE>::NP * KPLANE, KSZ_OFF = V_OFF + Mode<MODE>::NP * VPLANE;
  __host__ __device__ static constexpr int vsz_off(int lg) { return KSZ_OFF + (kTile >> lg) * 2 * D * 4; }
  __host__ __device__ static constexpr int bytes(int lg) { return vsz_off(lg) + kTile * 2 * (D >> lg) * 4; }
};

// ------------------------------------------------------------------------------
// The kernel
// ------------------------------------------------------------------------------
template <int MODE, int D, int NR, bool MOD>
__global__ void __launch_bounds__(Shape<NR>::THREADS, Shape<NR>::CTAS) shared_kernel(const __grid_constant__ SharedParams p) {
  using L = SharedSmem<D, NR>;
  using M = Mode<MODE>;
  using C = Codes<MODE>;
  using SM = StageMap<MODE, D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  using H = Shape<NR>;
  constexpr uint32_t T_K = H::T_K, T_V = H::T_V, T_S = H::T_S, T_O = H::T_O;
  constexpr int VB = H::VB, GROUPS = H::GROUPS;
  constexpr int KSTEPS = D / 16;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the own attention may take each SM that is done
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int split = blockIdx.y, kvh = blockIdx.z;
  constexpr int N = NR;                            // rows of the tile, padded
  const int row0 = blockIdx.x * N;
  const int nrow = min(N, p.rows - row0);
  const int lg = __ffs(p.c.G) - 1, G = 1 << lg, NJ = D >> lg;   // (the loops divide by neither G nor the ring)
  const int stage_bytes = SM::bytes(lg), vsz_off = SM::vsz_off(lg);
  const int nst = p.stages;
  float* rowf = reinterpret_cast<float*>(smem + L::ROW_OFF);
  uint32_t* tm_slot = reinterpret_cast<uint32_t*>(smem + L::MISC_OFF);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L::MISC_OFF + 4);
  int* lo_all_s = reinterpret_cast<int*>(smem + L::MISC_OFF + 8);
  int* lo_any_s = lo_all_s + 1;
  int* sent = reinterpret_cast<int*>(smem + L::MISC_OFF + 16);   // tiles of codes, of zero terms whose copies were issued
  unsigned* vmax_s = reinterpret_cast<unsigned*>(smem + L::MISC_OFF + 32);   // largest value scale and |zero point|
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L::BAR_OFF);
  uint64_t *full = bars, *empty = bars + 8, *zfull = bars + 16, *zempty = bars + 20, *kfull = bars + 24, *sfull = bars + 25,
           *pfull = bars + 26, *drained = bars + 27, *pvdone = bars + 28;   // pvdone: one for each value buffer
  constexpr int cw = N / GROUPS;   // a softmax group: 128 threads, one a token, and its share of the rows

  if (tid == 0) {
    *abort_flag = 0;
    *lo_all_s = INT_MAX;
    *lo_any_s = INT_MIN;
    vmax_s[0] = vmax_s[1] = 0u;
    sent[0] = sent[1] = 0;
    for (int i = 0; i < nst; ++i) {
      mbar_init(full + i, 1);
      mbar_init(empty + i, H::WORK);
    }
    for (int i = 0; i < L::ZB; ++i) {
      mbar_init(zfull + i, 1);
      mbar_init(zempty + i, H::WORK);
    }
    mbar_init(kfull, H::WORK);
    mbar_init(sfull, 1);
    mbar_init(pfull, H::WORK);
    mbar_init(drained, 1);
    mbar_init(pvdone, 1);
    mbar_init(pvdone + 1, 1);
    fence_mbar_init();
  }
  if (warp == H::MMA) tm_alloc(tm_slot, H::T_ALL);
  __syncthreads();

  // ---- rows: what each sees, and its query, exact in f16 after a power of two of its own ----
  // (Positions beside a slope count from the prefix's end: a key's is negative
  // and a query's is not, so a distance keeps its 24 bits at any length.)
  const int n0 = static_cast<int>(p.c.Lq) + p.c.r;
  for (int e = tid; e < NR; e += H::THREADS) {
    float* f = rowf + e;
    int lo = INT_MAX, qp = 0;
    float slope = 0.f;
    if (e < nrow) {
      const int row = row0 + e, b = row / p.R, rho = row % p.R;
      qp = n0 + static_cast<int>(seq_lq(p.own, b)) + seq_r(p.own, b) + p.P - p.gamma + rho / p.HG;
      lo = p.first ? p.first[b] : INT_MIN;
      if (p.window > 0) lo = max(lo, qp - (p.window - 1));
      if (p.slopes) slope = p.slopes[kvh * p.HG + rho % p.HG] * 1.4426950408889634f;
      atomicMin(lo_all_s, lo);
      atomicMax(lo_any_s, lo);
    }
    f[0] = -kNoRef;
    f[NR] = 1.f;
    reinterpret_cast<int*>(f)[2 * NR] = max(lo, 0);
    f[3 * NR] = static_cast<float>(qp - n0);
    f[4 * NR] = slope;
    float* zc = reinterpret_cast<float*>(smem + L::ZC_OFF) + e;
    zc[0] = 0.f;
    zc[NR] = neg_inf();
  }
  // A row's own power of two, so that no row's values touch another's: D / 8
  // adjacent lanes hold a row.
  constexpr int QI = NR * D / 8;                       // 16-byte slices of the queries
#pragma unroll 1
  for (int e = tid; e < QI; e += H::THREADS) {         // (whole warps)
    const int r = e / (D / 8), c8 = 8 * (e % (D / 8));
    uint4 v = make_uint4(0u, 0u, 0u, 0u);
    if (r < nrow) {
      const int row = row0 + r, b = row / p.R, rho = row % p.R;
      v = *reinterpret_cast<const uint4*>(p.q + ((static_cast<long long>(b) * p.gamma + rho / p.HG) * p.Hq + kvh * p.HG + rho % p.HG) * D + c8);
    }
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xFFFF0000u))));
#pragma unroll
    for (int o = 1; o < D / 8; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const int eq = norm_exp(mx);
    const float f = pow2f_exact(-eq);
    if (c8 == 0) rowf[5 * NR + r] = pow2f_exact(eq);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16) * f;
      const int kk = code_slot<MODE>(c8 + i);
      const int off = (kk / 64) * (NR * 128) + r * 128 + ((((kk % 64) / 8) ^ (r & 7)) << 4) + (kk % 8) * 2;
      *reinterpret_cast<__half*>(smem + L::Q_OFF + off) = __float2half_rn(x);
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  tm_fence_before();
  __syncthreads();
  tm_fence_after();
  const uint32_t tm = *tm_slot;
  const int lo_all = max(0, *lo_all_s), lo_any = *lo_any_s;

  // ---- this CTA's tiles: those before the first visible token are left out ----
  const int lq = static_cast<int>(p.c.Lq);
  int first_tile = split * p.per;
  const int end_tile = min(p.tiles, first_tile + p.per);
  if (lo_all > p.t_begin) {
    const int hid = lo_all >= lq ? p.tiles_q + (lo_all - lq >= p.c.r ? p.tiles - p.tiles_q : (lo_all - lq) / kTile)
                                 : (lo_all - p.t_begin) / kTile;
    first_tile = max(first_tile, hid);
  }
  const int nt = max(0, end_tile - first_tile);
  const int tok0 = p.t_begin + first_tile * kTile;     // first quantized token (if any tile is)
  const int nq = max(0, min(end_tile, p.tiles_q) - first_tile);   // quantized tiles
  const long long u_tok = static_cast<long long>(kvh) * p.c.C;

  // A bounded wait, by whole warps, which leaves them converged.  On giving up
  // (or once another thread has) every warp runs through its remaining steps
  // without waiting, so that the named barriers stay matched and nothing is
  // left behind.
  auto wait_warp = [&](uint64_t* bar, uint32_t parity) {
    if (!try_wait_64(bar, parity)) wait_slow(bar, parity, p.wait_limit, p.status, abort_flag);
    __syncwarp();
  };
  const float mult = MODE == KVQ_MODE_INT1 ? p.smul : static_cast<float>(M::MULT);
  auto value_exp = [&]() {   // values lie within |zero point| + (cmax mult + shift) scale
    return norm_exp(fmaf(C::CMAX * mult + fabsf(p.zshift), __uint_as_float(vmax_s[0]), __uint_as_float(vmax_s[1])));
  };

  if (warp == H::COPY) {
    // =============================== copies ===============================
    // Operands are computed by the whole warp from warp-uniform values and the
    // copies issued by one elected lane.
    const uint64_t pol = __shfl_sync(0xffffffffu, policy_evict_first(), 0);
    const long long tok_u = u_tok + tok0;
    const uint8_t *kp = p.c.kplane[0] + tok_u * SM::KROW, *vp = p.c.vplane[0] + tok_u / 32 * (D * SM::VROW);
    const long long kp1 = p.c.kplane[1] - p.c.kplane[0], vp1 = p.c.vplane[1] - p.c.vplane[0];   // the lower plane (INT8)
    const float *ksz = p.c.ksz + (static_cast<long long>(kvh) * (p.c.C >> lg) + (tok0 >> lg)) * 2 * D, *vsz = p.c.vsz + tok_u * 2 * NJ;
    const float* zsrc = p.zt + ((static_cast<long long>(kvh) * gridDim.x + blockIdx.x) * p.groups + ((tok0 - p.t_begin) >> lg)) * NR;
    int zi = 0;   // tiles whose zero terms are on their way
    int s = 0, round = 0, t = 0;
#pragma unroll 1
    for (; t < nq; ++t) {
      if (round > 0) wait_warp(empty + s, (round - 1) & 1);
      if (__any_sync(0xffffffffu, *abort_flag)) break;
      const int n = min(kTile, lq - (tok0 + t * kTile));
      uint8_t* st = smem + L::STAGE_OFF + s * stage_bytes;
      const uint32_t kb = n * SM::KROW, vb = n / 32 * (D * SM::VROW);
      const uint32_t kszb = static_cast<uint32_t>((n + G - 1) >> lg) * 2 * D * 4, vszb = n * 2 * NJ * 4;
      if (elect_one()) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive_expect_tx(full + s, M::NP * (kb + vb) + kszb + vszb);
        bulk_g2s(st, kp, kb, full + s, pol);
        bulk_g2s(st + SM::V_OFF, vp, vb, full + s, pol);
        if constexpr (M::NP == 2) {
          bulk_g2s(st + SM::KPLANE, kp + kp1, kb, full + s, pol);
          bulk_g2s(st + SM::V_OFF + SM::VPLANE, vp + vp1, vb, full + s, pol);
        }
        bulk_g2s(st + SM::KSZ_OFF, ksz, kszb, full + s, pol);
        bulk_g2s(st + vsz_off, vsz, vszb, full + s, pol);
      }
      __syncwarp();
      kp += kTile * SM::KROW;
      vp += kTile / 32 * (D * SM::VROW);
      ksz += (kTile >> lg) * 2 * D;
      vsz += kTile * 2 * NJ;
      if (++s == nst) {
        s = 0;
        ++round;
      }
      // The zero terms follow once the launch that makes them is done: waited
      // for when the ring of codes is on its way.
      if (t + 1 >= min(nst, nq)) {
        if (zi == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll 1
        for (; zi <= t; ++zi) {
          const int z = zi % L::ZB;
          const uint32_t zb = static_cast<uint32_t>((min(kTile, lq - (tok0 + zi * kTile)) + G - 1) >> lg) * NR * 4;
          if (zi >= L::ZB) wait_warp(zempty + z, (zi / L::ZB - 1) & 1);
          if (elect_one()) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            mbar_arrive_expect_tx(zfull + z, zb);
            bulk_g2s(smem + L::Z_OFF + z * L::Z_BUF, zsrc, zb, zfull + z, pol);
          }
          __syncwarp();
          zsrc += (kTile >> lg) * NR;
        }
      }
    }
    if (zi == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (lane == 0) {
      sent[0] = t;
      sent[1] = zi;
    }
  } else if (warp == H::MMA) {
    // =============================== products ===============================
    // The whole warp walks the steps with warp-uniform descriptors; one elected
    // lane issues (a product issued from a divergent lane costs 50 cycles and
    // more, one of N = 64 itself 34).
    const uint32_t tmu = __shfl_sync(0xffffffffu, tm, 0);
    const uint32_t idesc_s = instr_desc(N, false), idesc_o = instr_desc(N, true);
    const uint64_t qdesc = mat_desc(smem_u32(smem + L::Q_OFF), 1024, 16), pdesc = mat_desc(smem_u32(smem + L::P_OFF), 1024, L::P_BLOCK);
#pragma unroll 1
    for (int i = 0; i < nt; ++i) {
      wait_warp(kfull, i & 1);
      tm_fence_after();
      if (elect_one()) {
        // hi parts, then lo parts (the columns behind them)
#pragma unroll
        for (int k = 0; k < 2 * KSTEPS; ++k)
          tm_mma(tmu + T_S, tmu + T_K + k * 8, qdesc + (((k % KSTEPS / 4) * (NR * 128) + (k % 4) * 32) >> 4), idesc_s, k > 0);
        tm_commit(sfull);
      }
      __syncwarp();
      wait_warp(pfull, i & 1);
      tm_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k)
          tm_mma(tmu + T_O, tmu + T_V + (i % VB) * 64 + k * 8, pdesc + k * (2048 >> 4), idesc_o, i > 0 || k > 0);
        tm_commit(pvdone + i % VB);
      }
      __syncwarp();
    }
    // No product is under way when the CTA leaves, whatever the other warps gave up.
    if (elect_one()) tm_commit(drained);
    __syncwarp();
    mbar_wait_bounded(drained, 0, 1 << 24);
    __syncwarp();
  } else {
    // =============================== codes and softmax ===============================
    const int g = warp / 4, w4 = warp & 3, ln = 32 * w4 + lane;   // group; warp of the group; TMEM lane: token or channel
    const uint32_t lane_base = static_cast<uint32_t>(32 * w4) << 16;
    float* kfac = reinterpret_cast<float*>(smem + L::KF_OFF);
    {
      // The largest value scale and |zero point| that this CTA reads bound its
      // values, for their power of two.
      float ms = 0.f, mz = 0.f;
      const int t_lo = max(tok0, lo_all), t_hi = min(lq, tok0 + nq * kTile);
      if (t_lo < t_hi) {
        const float* v = p.c.vsz + (u_tok + t_lo) * 2 * NJ;
        int n = (t_hi - t_lo) * 2 * NJ;                 // floats; rows of s [NJ], z [NJ]
        if (NJ == 1 && (t_lo & 1)) {                    // to a 16-byte boundary
          ms = fabsf(v[0]);
          mz = fabsf(v[1]);
          v += 2;
          n -= 2;
        }
        const float4* v4 = reinterpret_cast<const float4*>(v);
#pragma unroll 4
        for (int i = tid; i < n / 4; i += H::WORK * 32) {
          const float4 a = v4[i];
          const float lo2 = fmaxf(fabsf(a.x), fabsf(NJ == 1 ? a.z : a.y)), hi2 = fmaxf(fabsf(NJ == 1 ? a.y : a.z), fabsf(a.w));
          const bool zrow = NJ == 4 && (i & 1);         // a whole row of zero points
          ms = fmaxf(ms, NJ == 4 ? (zrow ? 0.f : fmaxf(lo2, hi2)) : lo2);
          mz = fmaxf(mz, NJ == 4 ? (zrow ? fmaxf(lo2, hi2) : 0.f) : hi2);
        }
        if (NJ == 1 && (n & 2) && tid == 0) {
          ms = fmaxf(ms, fabsf(v[n - 2]));
          mz = fmaxf(mz, fabsf(v[n - 1]));
        }
      }
      if (nt > nq) {
        const int r_lo = max((first_tile + nq - p.tiles_q) * kTile, lo_all - lq), r_hi = min(p.c.r, (end_tile - p.tiles_q) * kTile);
        const uint4* src = reinterpret_cast<const uint4*>(p.c.res_v + static_cast<long long>(kvh) * 2 * G * D);
#pragma unroll 4
        for (int i = tid; i < 2 * G * D / 8; i += H::WORK * 32) {
          const int t = (i / (D / 8) - p.c.res_start) & (2 * G - 1);
          const uint4 a = t >= r_lo && t < r_hi ? src[i] : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mz = fmaxf(mz, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
        }
      }
      const unsigned rs = __reduce_max_sync(0xffffffffu, __float_as_uint(ms)), rz = __reduce_max_sync(0xffffffffu, __float_as_uint(mz));
      if (lane == 0) {
        atomicMax(vmax_s, rs);
        atomicMax(vmax_s + 1, rz);
      }
      asm volatile("bar.sync 1, %0;" ::"n"(H::WORK * 32) : "memory");
    }
    const float vf = pow2f_exact(-value_exp());

    // A lane's place in a table of 32 codes' factors: slot `lane`, of code `perm`.
    const int perm = slot_code<MODE>(lane);
    __half* ktab = reinterpret_cast<__half*>(smem + L::KT_OFF + warp * 128) + 4 * (lane / 2) + (lane & 1);

    // ---- keys of a quantized tile: this warp's 32 tokens (lanes) and group's channels ----
    int ks = 0;              // stage of the next tile's keys
    uint32_t kround = 0;     // times the ring went round
    auto key_ready = [&]() {
      tm_wait_st();
      tm_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(kfull);
    };
    auto k_tile = [&](int t) {
      wait_warp(full + ks, kround & 1);
      const uint8_t* st = smem + L::STAGE_OFF + ks * stage_bytes;
      if (++ks == nst) {
        ks = 0;
        ++kround;
      }
      {
        const bool live = 32 * w4 < lq - (tok0 + t * kTile);
        const float* sc = reinterpret_cast<const float*>(st + SM::KSZ_OFF) + (32 * w4 >> lg) * 2 * D;   // its key group's scales
        // the power of two of all channels' scales, then each chunk's in slot pairs
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) mx = fmaxf(mx, live ? sc[lane + 32 * i] : 0.f);
        const int e = norm_exp(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx))) * (mult * C::CABS));
        const float f = pow2f_exact(-e);
        if (g == 0) kfac[(t & 1) * 128 + ln] = pow2f_exact(e) * p.qscale;
        const float mf = mult * f;    // (powers of two)
#pragma unroll 1
        for (int c = g; c < D / 32; c += GROUPS) {   // 32 channels at a time
          uint32_t h[4], l[4], x[16];
          load_codes<MODE>(st + ln * SM::KROW + c * (C::WPC * 4), SM::KPLANE, h, l);
          const float a = live ? sc[32 * c + perm] * mf : 0.f;
          const __half ah = __float2half_rn(a);
          __syncwarp();
          ktab[0] = ah;
          ktab[2] = __float2half_rn(a - __half2float(ah));
          centred<MODE>(h, l, x);
          __syncwarp();
          uint32_t hi[16], lo[16];
          const uint4* t4 = reinterpret_cast<const uint4*>(smem + L::KT_OFF) + warp * 8;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 w = t4[i];   // (s_hi, s_lo) of two pairs
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const __half2 cc = as_half2(x[2 * i + k]), sh = as_half2(k ? w.z : w.x), sl = as_half2(k ? w.w : w.y);
              const __half2 hv = __hmul2(cc, sh);
              hi[2 * i + k] = as_u32(hv);
              lo[2 * i + k] = as_u32(__hfma2(cc, sl, __hfma2(cc, sh, __hneg2(hv))));
            }
          }
          tm_st16(tm + T_K + lane_base + 16 * c, hi);
          tm_st16(tm + T_K + D / 2 + lane_base + 16 * c, lo);
        }
      }
      key_ready();
    };
    auto k_residual = [&](int t, int t0) {   // residual tokens t0 .. t0 + 127: bf16 keys, exact in f16 after a power of two
      {
        const int tk = t0 + ln;
        const bool on = tk < p.c.r;
        const uint4* src = reinterpret_cast<const uint4*>(
            p.c.res_k + (static_cast<long long>(kvh) * 2 * G + ((p.c.res_start + (on ? tk : 0)) & (2 * G - 1))) * D);
        float mx = 0.f;
        if (on) {
#pragma unroll 4
          for (int i = 0; i < D / 8; ++i) {
            const uint4 v = src[i];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(w[k] << 16)), fabsf(__uint_as_float(w[k] & 0xFFFF0000u))));
          }
        }
        const int e = norm_exp(mx);
        const float f = on ? pow2f_exact(-e) : 0.f;
        if (g == 0) kfac[(t & 1) * 128 + ln] = pow2f_exact(e) * p.qscale;
        const uint32_t zero[16] = {};
#pragma unroll 1
        for (int c = g; c < D / 32; c += GROUPS) {
          uint32_t hi[16], w[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 v = on ? src[4 * c + i] : make_uint4(0u, 0u, 0u, 0u);
            w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
          }
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int c0 = slot_code<MODE>(2 * i), c1 = slot_code<MODE>(2 * i + 1);
            const float a = __uint_as_float(c0 & 1 ? w[c0 / 2] & 0xFFFF0000u : w[c0 / 2] << 16);
            const float b = __uint_as_float(c1 & 1 ? w[c1 / 2] & 0xFFFF0000u : w[c1 / 2] << 16);
            hi[i] = pack_half2(a * f, b * f);
          }
          __syncwarp();
          tm_st16(tm + T_K + lane_base + 16 * c, hi);
          tm_st16(tm + T_K + D / 2 + lane_base + 16 * c, zero);
        }
      }
      key_ready();
    };

    // ---- values: this warp's 32 channels (lanes) and group's tokens ----
    int vs = 0;              // stage of the next tile's values
    auto value_wait = [&](int t) {
      // (two buffers: the softmax of the tile before waited for this one's last use)
      if (VB == 1 && t > 0) wait_warp(pvdone, (t - 1) & 1);
      tm_fence_after();
    };
    auto v_tile = [&](int t) {   // (its stage was waited for with the keys)
      const uint8_t* st = smem + L::STAGE_OFF + vs * stage_bytes;
      uint64_t* done = empty + vs;
      if (++vs == nst) vs = 0;
      value_wait(t);
      if (32 * w4 < D) {
#pragma unroll 1
        for (int c = g; c < kTile / 32; c += GROUPS) {   // 32 tokens at a time
          uint32_t h[4], l[4], x[16];
          load_codes<MODE>(st + SM::V_OFF + (c * D + ln) * SM::VROW, SM::VPLANE, h, l);
          // scales and zero points of the tokens for this warp's channel block, in
          // slot pairs; those of tokens that no row sees are zero
          const int tok = 32 * c + perm, pos = tok0 + t * kTile + tok;
          const float* v = reinterpret_cast<const float*>(st + vsz_off) + tok * 2 * NJ + (32 * w4 >> lg);
          const bool on = pos < lq && pos >= lo_all;
          const float s0 = on ? v[0] : 0.f, z0 = on ? v[NJ] : 0.f, se = s0 * mult;
          __half* vtab = ktab + (L::VT_OFF - L::KT_OFF) / 2;
          __syncwarp();
          vtab[0] = __float2half_rn(se * vf);
          vtab[2] = __float2half_rn((fmaf(p.zshift, s0, z0) + C::C0 * se) * vf);
          centred<MODE>(h, l, x);
          __syncwarp();
          const uint4* t4 = reinterpret_cast<const uint4*>(smem + L::VT_OFF) + warp * 8;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 w = t4[i];   // (s, z) of two pairs
            x[2 * i] = as_u32(__hfma2(as_half2(x[2 * i]), as_half2(w.x), as_half2(w.y)));
            x[2 * i + 1] = as_u32(__hfma2(as_half2(x[2 * i + 1]), as_half2(w.z), as_half2(w.w)));
          }
          tm_st16(tm + T_V + (t % VB) * 64 + lane_base + 16 * c, x);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(done);
    };
    auto v_residual = [&](int t, int t0) {
      value_wait(t);
      if (32 * w4 < D) {
        const uint16_t* src = p.c.res_v + static_cast<long long>(kvh) * 2 * G * D + ln;
#pragma unroll 1
        for (int c = g; c < kTile / 32; c += GROUPS) {
          uint32_t x[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float v[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int tk = t0 + 32 * c + slot_code<MODE>(2 * i + e);
              v[e] = tk < p.c.r && lq + tk >= lo_all ? bf16_to_f32(src[((p.c.res_start + tk) & (2 * G - 1)) * D]) * vf : 0.f;
            }
            x[i] = pack_half2(v[0], v[1]);
          }
          __syncwarp();
          tm_st16(tm + T_V + (t % VB) * 64 + lane_base + 16 * c, x);
        }
      }
      __syncwarp();
    };

    // ---- softmax: this thread's token, its group's rows ----
    const int c0 = g * cw;                     // first row of the group
    float* nref = rowf + c0;
    float* alpha = nref + NR;
    const int* low = reinterpret_cast<const int*>(nref + 2 * NR);
    const float* qpos = nref + 3 * NR;
    const float* slope = nref + 4 * NR;
    const float* qfac = nref + 5 * NR;
    float* wm = reinterpret_cast<float*>(smem + L::WM_OFF) + c0;
    const uint32_t ts = tm + T_S + lane_base + c0, to = tm + T_O + lane_base + c0;
    const int kk0 = code_slot<MODE>(ln);
    uint8_t* prow = smem + L::P_OFF + kk0 * 128;   // this token's weights: 16-byte pieces of 8 rows, swizzled, in blocks of 64 rows
    constexpr int CH = NR / GROUPS / 8;             // chunks of 8 rows at most
    float2 l2[4 * CH];                         // sums of this lane's weights, two rows at a time
#pragma unroll
    for (int i = 0; i < 4 * CH; ++i) l2[i] = make_float2(0.f, 0.f);

    auto softmax = [&](int i) {
      const bool quant = i < nq;
      const int t0 = quant ? tok0 + i * kTile : lq + (first_tile + i - p.tiles_q) * kTile;   // position of the tile's first token
      const int n = min(kTile, (quant ? lq : lq + p.c.r) - t0), pos = t0 + ln;
      const bool valid = ln < n;
      // What is added to the lane's products: its group's zero terms; zeros for a
      // residual token; minus infinity past the last token (whose products are 0).
      const int zs = i % L::ZB;
      const float* zrow = reinterpret_cast<const float*>(smem + (!valid ? L::ZC_OFF + NR * 4 : quant ? L::Z_OFF + zs * L::Z_BUF : L::ZC_OFF)) +
                          (valid && quant ? (32 * w4 >> lg) * NR : 0) + c0;
      const float kf = kfac[(i & 1) * 128 + ln];

      // The logits of 8 rows from the group's row 8 c on, from their products `a`.
      auto logits_of = [&](int c, const uint32_t (&a)[8], float2 (&x)[4]) {
        const float2 kf2 = make_float2(kf, kf);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 z = *reinterpret_cast<const float4*>(zrow + 8 * c + 4 * k), f = *reinterpret_cast<const float4*>(qfac + 8 * c + 4 * k);
          x[2 * k] = fma2(mul2(make_float2(__uint_as_float(a[4 * k]), __uint_as_float(a[4 * k + 1])), make_float2(f.x, f.y)), kf2, make_float2(z.x, z.y));
          x[2 * k + 1] = fma2(mul2(make_float2(__uint_as_float(a[4 * k + 2]), __uint_as_float(a[4 * k + 3])), make_float2(f.z, f.w)), kf2, make_float2(z.z, z.w));
        }
        if constexpr (MOD) {
          if (p.cap2 > 0.f) {
            // The polynomial alone where no row comes near the cap; else each logit by
            // the form that suits its size, so that none is touched by its neighbours'.
            // (Lanes past the last token hold minus infinity and ask for nothing.)
            float big = 0.f;
#pragma unroll
            for (int k = 0; k < 4; ++k) big = fmaxf(big, fmaxf(fabsf(x[k].x), fabsf(x[k].y)));
            if (__any_sync(0xffffffffu, valid && big > kCapPoly * p.cap2)) {
#pragma unroll
              for (int k = 0; k < 4; ++k) x[k] = any_cap2(x[k], p.cap2, p.cap_f);
            } else {
              const float inv = cap_inverse(p.cap_f);
#pragma unroll
              for (int k = 0; k < 4; ++k) x[k] = cap_poly(x[k], make_float2(inv, inv));
            }
          }
          if (p.slopes) {
            const float2 at = make_float2(static_cast<float>(pos - n0), static_cast<float>(pos - n0));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 qp = *reinterpret_cast<const float2*>(qpos + 8 * c + 2 * k);
              x[k] = fma2(*reinterpret_cast<const float2*>(slope + 8 * c + 2 * k), add2(at, make_float2(-qp.x, -qp.y)), x[k]);
            }
          }
          if (t0 < lo_any || n < kTile) {
            const int at = valid ? pos : -1;   // below every row's first
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (at < low[8 * c + 2 * k]) x[k].x = neg_inf();
              if (at < low[8 * c + 2 * k + 1]) x[k].y = neg_inf();
            }
          }
        }
      };
      auto logits = [&](int c, float2 (&x)[4]) {
        uint32_t a[8];
        tm_ld8(ts + 8 * c, a);
        tm_wait_ld(a);
        logits_of(c, a, x);
      };

      // New references where a row's maximum has grown: sums and outputs follow.
      auto look = [&]() {
#pragma unroll 1
        for (int c = 0; c < cw / 8; ++c) {
          float2 x[4];
          logits(c, x);
          float mine = neg_inf();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            // the largest of the lanes' values, as integers that order like them
            const int b = __float_as_int((k & 1) ? x[k / 2].y : x[k / 2].x);
            const int m = __reduce_max_sync(0xffffffffu, b ^ ((b >> 31) & 0x7FFFFFFF));
            if (lane == k) mine = __int_as_float(m ^ ((m >> 31) & 0x7FFFFFFF));
          }
          if (lane < 8) wm[w4 * NR + 8 * c + lane] = mine;
        }
        named_sync(2 + g);
        if (ln < cw) {
          const float m = fmaxf(fmaxf(wm[ln], wm[NR + ln]), fmaxf(wm[2 * NR + ln], wm[3 * NR + ln])) - kRefBelow;
          const float old = -nref[ln];
          alpha[ln] = m > old ? fast_exp2(old - m) : 1.f;
          if (m > old) nref[ln] = -m;
        }
        named_sync(2 + g);
#pragma unroll
        for (int k = 0; k < 4 * CH; ++k) {
          if (2 * k < cw) {
            l2[k].x *= alpha[2 * k];
            l2[k].y *= alpha[2 * k + 1];
          }
        }
        if (i > 0) {
#pragma unroll 1
          for (int c = 0; c < cw / 8; ++c) {
            uint32_t a[8];
            tm_ld8(to + 8 * c, a);
            tm_wait_ld(a);
#pragma unroll
            for (int k = 0; k < 8; ++k) a[k] = __float_as_uint(__uint_as_float(a[k]) * alpha[8 * c + k]);
            tm_st8(to + 8 * c, a);
          }
          tm_wait_st();
        }
      };

      // A second pass follows a vote.
      bool again = i == 0;   // the first tile's references
      for (int pass = 0;; ++pass) {
        if (again) look();
        float top = neg_inf();
        uint32_t a8[2][8];   // the next 8 rows' products load while these are turned
        tm_ld8(ts, a8[0]);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          if (8 * c < cw) {
            tm_wait_ld(a8[c & 1]);
            if (8 * c + 8 < cw) tm_ld8(ts + 8 * c + 8, a8[(c + 1) & 1]);
            float2 x[4];
            logits_of(c, a8[c & 1], x);
            uint32_t pk[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float4 m = *reinterpret_cast<const float4*>(nref + 8 * c + 4 * k);
              const float2 a = add2(x[2 * k], make_float2(m.x, m.y)), b = add2(x[2 * k + 1], make_float2(m.z, m.w));
              top = fmaxf(fmaxf(top, fmaxf(a.x, a.y)), fmaxf(b.x, b.y));
              const float2 ea = make_float2(fast_exp2(a.x), fast_exp2(a.y)), eb = make_float2(fast_exp2(b.x), fast_exp2(b.y));
              pk[2 * k] = pack_half2(ea.x, ea.y);
              pk[2 * k + 1] = pack_half2(eb.x, eb.y);
              l2[4 * c + 2 * k] = add2(l2[4 * c + 2 * k], ea);
              l2[4 * c + 2 * k + 1] = add2(l2[4 * c + 2 * k + 1], eb);
            }
            const int col = c0 + 8 * c;
            *reinterpret_cast<uint4*>(prow + (col / 64) * L::P_BLOCK + (((col / 8 % 8) ^ (kk0 & 7)) << 4)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
          }
        }
        again = named_or(2 + g, top > kVoteAbove);
        if (!again || pass == 1) break;
        // Take this tile's weights out of the sums again, then look.  What
        // that loses is 2^-24 of the weight, which the new reference makes
        // 2^4 at most; a sum beside a weight of 2^100 counts for nothing.
        float part[8 * CH];   // rare: rolled, in local memory
#pragma unroll
        for (int k = 0; k < 8 * CH; ++k) part[k] = (k & 1) ? l2[k / 2].y : l2[k / 2].x;
#pragma unroll 1
        for (int c = 0; c < cw / 8; ++c) {
          float2 x[4];
          logits(c, x);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float a = ((k & 1) ? x[k / 2].y : x[k / 2].x) + nref[8 * c + k];
            part[8 * c + k] = a > 100.f ? 0.f : part[8 * c + k] - fast_exp2(a);
          }
        }
#pragma unroll
        for (int k = 0; k < 4 * CH; ++k) l2[k] = make_float2(part[2 * k], part[2 * k + 1]);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      if (quant && lane == 0) mbar_arrive(zempty + zs);
    };

    if (nt > 0) {
      if (nq > 0) k_tile(0);
      else k_residual(0, (first_tile - p.tiles_q) * kTile);
    }
#pragma unroll 1
    for (int i = 0; i < nt; ++i) {
      if (i < nq) v_tile(i);
      else v_residual(i, (first_tile + i - p.tiles_q) * kTile);
      if (i < nq) wait_warp(zfull + i % L::ZB, (i / L::ZB) & 1);
      if (VB == 2 && i > 0) wait_warp(pvdone + (i - 1) % VB, ((i - 1) / VB) & 1);   // the weights' buffer and the outputs are free
      wait_warp(sfull, i & 1);
      tm_fence_after();
      softmax(i);
      tm_wait_st();       // values (and rescaled outputs) are in TMEM
      tm_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pfull);
      if (i + 1 < nt) {   // the keys' buffer is free: S (i) is done
        if (i + 1 < nq) k_tile(i + 1);
        else k_residual(i + 1, (first_tile + i + 1 - p.tiles_q) * kTile);
      }
    }

    // ---- partials: sums over the tokens, outputs from TMEM ----
    if (nt > 0) wait_warp(pvdone + (nt - 1) % VB, ((nt - 1) / VB) & 1);
    tm_fence_after();
    // every warp is done with the weights' buffer and the zero terms: [row][lane + 1] of 8 rows
    asm volatile("bar.sync 1, %0;" ::"n"(H::WORK * 32) : "memory");
    {
      float* lsum = reinterpret_cast<float*>(smem + L::P_OFF) + warp * (8 * 33);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        if (8 * c < cw) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            lsum[(2 * k) * 33 + lane] = l2[4 * c + k].x;
            lsum[(2 * k + 1) * 33 + lane] = l2[4 * c + k].y;
          }
          __syncwarp();
          float a = 0.f;
#pragma unroll
          for (int k = 0; k < 8; ++k) a += lsum[(lane & 7) * 33 + (lane & 24) + k];
          a += __shfl_xor_sync(0xffffffffu, a, 8);
          a += __shfl_xor_sync(0xffffffffu, a, 16);
          if (lane < 8) wm[w4 * NR + 8 * c + lane] = a;
          __syncwarp();
        }
      }
      named_sync(2 + g);
      const long long part = (static_cast<long long>(kvh) * p.S + split) * p.rows + row0 + c0;
      const int mine = min(cw, nrow - c0);     // rows of this group (may be negative)
      if (ln < mine) {
        const float sum = (wm[ln] + wm[NR + ln]) + (wm[2 * NR + ln] + wm[3 * NR + ln]);
        // (a sum that is no number keeps its reference, and so its place among the partials)
        reinterpret_cast<float2*>(p.ml)[part + ln] = make_float2(sum == 0.f ? neg_inf() : -nref[ln], sum);
      }
      if (nt > 0) {
        const float f = pow2f_exact(value_exp());
#pragma unroll 1
        for (int c = 0; c < cw / 8; ++c) {
          uint32_t a[8];
          tm_ld8(to + 8 * c, a);
          tm_wait_ld(a);
          if (ln < D) {
#pragma unroll
            for (int k = 0; k < 8; ++k)
              if (8 * c + k < mine) p.o[(part + 8 * c + k) * D + ln] = __uint_as_float(a[k]) * f;
          }
        }
      }
    }
    tm_fence_before();
  }

  __syncwarp();
  __syncthreads();
  if (*abort_flag) {   // copies still in flight land before the CTA leaves
    if (tid == 0) {
      for (int t = max(0, sent[0] - nst); t < sent[0]; ++t) mbar_wait_bounded(full + t % nst, (t / nst) & 1, 1 << 24);
      for (int t = max(0, sent[1] - L::ZB); t < sent[1]; ++t) mbar_wait_bounded(zfull + t % L::ZB, (t / L::ZB) & 1, 1 << 24);
    }
    __syncthreads();
  }
  if (warp == H::MMA) {
    tm_fence_after();
    tm_dealloc(tm, H::T_ALL);
  }
}

// ------------------------------------------------------------------------------
// The rows' zero terms: q.(z + c0 s) qscale of each key group, which the pass
// above adds to the logits of the group's tokens.  A CTA takes 32 groups and up
// to 64 rows of a row tile; a warp keeps its 8 groups' fragments in registers and walks the
// rows, 16 at a time, by bf16 m16n8k16 products.  A term z + c0 s goes in as
// three bf16 parts (24 bits), so nothing is lost at any size.  The products'
// k order is permuted so that a lane's operands are 8 adjacent channels: k-step
// 2 j + i, register halves e of lane q hold channels 32 j + 8 q + 4 i + 2 e.
// Bound by its loads' latency: 3 to 12 us, most of them beside the start of the
// pass.  (288 rows over 1,025 groups x 8 heads, whole call, when it took three row
// tiles of 96, which two of 160 have replaced (134 us): CTAs of 64 rows 143.9 us, of
// 32 rows 146.4; a loop over all row tiles 143.2 to 148 by its grid.)
// ------------------------------------------------------------------------------
template <int D, int NR>
__global__ void __launch_bounds__(128) zero_kernel(const __grid_constant__ SharedParams p, float add) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ int qoff[NR];   // each row's place among the queries (in rows of D), -1: none
  const int lane = threadIdx.x % 32, g = lane >> 2, q = lane & 3;
  constexpr int PARTS = (NR + 63) / 64;   // CTAs over a tile's rows
  const int rt = blockIdx.y / PARTS, m0 = blockIdx.y % PARTS * 64, kvh = blockIdx.z, G = p.c.G;
  for (int e = threadIdx.x; e < NR; e += 128) {
    const int row = rt * NR + e;
    int off = -1;
    if (row < p.rows) {
      const int b = row / p.R, rho = row % p.R;
      off = static_cast<int>((static_cast<long long>(b) * p.gamma + rho / p.HG) * p.Hq + kvh * p.HG + rho % p.HG);
    }
    qoff[e] = off;
  }
  const int g0 = blockIdx.x * 32 + threadIdx.x / 32 * 8;
  const int grp = min(g0 + g, p.groups - 1);
  const float4* sp = reinterpret_cast<const float4*>(p.c.ksz + (static_cast<long long>(kvh) * (p.c.C / G) + p.t_begin / G + grp) * 2 * D) + 2 * q;
  uint32_t b[D / 16][3][2];
#pragma unroll
  for (int j = 0; j < D / 32; ++j)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float4 s = sp[8 * j + i], z = sp[D / 4 + 8 * j + i];
      float v[4] = {fmaf(add, s.x, z.x), fmaf(add, s.y, z.y), fmaf(add, s.z, z.z), fmaf(add, s.w, z.w)};
#pragma unroll
      for (int part = 0; part < 3; ++part)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const __nv_bfloat162 w = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
          const uint32_t u = *reinterpret_cast<const uint32_t*>(&w);
          b[2 * j + i][part][e] = u;
          v[2 * e] -= __uint_as_float(u << 16);
          v[2 * e + 1] -= __uint_as_float(u & 0xFFFF0000u);
        }
    }
  __syncthreads();
  float* out = p.zt + ((static_cast<long long>(kvh) * (gridDim.y / PARTS) + rt) * p.groups + g0 + 2 * q) * (NR) + g;
  const bool on0 = g0 + 2 * q < p.groups, on1 = g0 + 2 * q + 1 < p.groups;
#pragma unroll 2
  for (int m = m0; m < min(NR, m0 + 64); m += 16) {
    uint4 a[2][D / 32];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int off = qoff[m + g + 8 * e];
      const uint4* src = reinterpret_cast<const uint4*>(p.q + static_cast<long long>(max(off, 0)) * D) + q;
#pragma unroll
      for (int j = 0; j < D / 32; ++j) a[e][j] = off >= 0 ? src[4 * j] : make_uint4(0u, 0u, 0u, 0u);
    }
    float pa[3][4] = {};   // a part each: three short chains of products
#pragma unroll
    for (int j = 0; j < D / 32; ++j) {
      const uint32_t a0[4] = {a[0][j].x, a[1][j].x, a[0][j].y, a[1][j].y}, a1[4] = {a[0][j].z, a[1][j].z, a[0][j].w, a[1][j].w};
#pragma unroll
      for (int part = 0; part < 3; ++part) mma16816_bf16(pa[part], a0, b[2 * j][part][0], b[2 * j][part][1]);
#pragma unroll
      for (int part = 0; part < 3; ++part) mma16816_bf16(pa[part], a1, b[2 * j + 1][part][0], b[2 * j + 1][part][1]);
    }
    float acc[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[i] = pa[0][i] + (pa[1][i] + pa[2][i]);
    if (on0) {
      out[m] = acc[0] * p.qscale;
      out[m + 8] = acc[2] * p.qscale;
    }
    if (on1) {
      out[NR + m] = acc[1] * p.qscale;
      out[NR + m + 8] = acc[3] * p.qscale;
    }
  }
}

template <int MODE, int D, int NR, bool MOD>
cudaError_t launch_shared_t(SharedParams p, const SharedPlan& plan, cudaStream_t s) {
  using L = SharedSmem<D, NR>;
  const int stage = StageMap<MODE, D>::bytes(p.c.G == 128 ? 7 : (p.c.G == 64 ? 6 : 5));
  p.stages = (L::LIMIT - L::STAGE_OFF) / stage < L::MAX_STAGES ? (L::LIMIT - L::STAGE_OFF) / stage : L::MAX_STAGES;
  const int smem = L::STAGE_OFF + p.stages * stage;
  if (p.stages < 2) return cudaErrorInvalidValue;
  const cudaError_t e = set_smem_once(reinterpret_cast<const void*>(&shared_kernel<MODE, D, NR, MOD>), L::LIMIT);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(plan.row_tiles, plan.S, p.c.Hkv);
  cfg.blockDim = dim3(Shape<NR>::THREADS, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at = {};
  if (p.tiles_q > 0) {
    const float add = p.zshift + Codes<MODE>::C0 * (MODE == KVQ_MODE_INT1 ? p.smul : static_cast<float>(Mode<MODE>::MULT));
    zero_kernel<D, NR><<<dim3((p.groups + 31) / 32, plan.row_tiles * ((NR + 63) / 64), p.c.Hkv), 128, 0, s>>>(p, add);
    const cudaError_t z = cudaGetLastError();
    if (z != cudaSuccess) return z;
    // the pass starts beside that launch, whose own start was after all earlier
    // work, and waits for it before it reads the terms
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, shared_kernel<MODE, D, NR, MOD>, p);
}

template <int MODE, int NR, bool MOD>
cudaError_t launch_shared_d(const SharedParams& p, const SharedPlan& plan, cudaStream_t s) {
  return p.c.D == 128 ? launch_shared_t<MODE, 128, NR, MOD>(p, plan, s) : launch_shared_t<MODE, 64, NR, MOD>(p, plan, s);
}

}  // namespace

// MOD: the variants with modified scores, compiled apart so that the plain ones stay small.
template <int MODE, bool MOD>
cudaError_t shared_launch_m(const SharedParams& p, const SharedPlan& plan, cudaStream_t s) {
  switch (plan.cols) {
    case 16: return launch_shared_d<MODE, 16, MOD>(p, plan, s);
    case 32: return launch_shared_d<MODE, 32, MOD>(p, plan, s);
    case 64: return launch_shared_d<MODE, 64, MOD>(p, plan, s);
    case 96: return launch_shared_d<MODE, 96, MOD>(p, plan, s);
    case 128: return launch_shared_d<MODE, 128, MOD>(p, plan, s);
    default: return launch_shared_d<MODE, 160, MOD>(p, plan, s);
  }
}
}  // namespace kvq
