// Plan and dispatch of the shared-prefix pass (kvq_attend_shared's first
// launch).  The kernel is in kvq_shared_kernel.cuh; each mode's variants are
// compiled in kvq_shared_<mode>.cu.
#include <algorithm>

#include "kvq_internal.h"

namespace kvq {
template <int MODE, bool MOD>
cudaError_t shared_launch_m(const SharedParams& p, const SharedPlan& plan, cudaStream_t s);

namespace {

int ceil_div_i(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

// Row tiles of up to 160 rows (what the TMEM holds), all alike, padded to 16 rows
// or to a multiple of 32: each tile turns the prefix's codes again, so few and
// large ones (288 rows over 32K INT2 tokens: two of 160 134 us, three of 96 145).
void shared_rows(int rows, SharedPlan* pl) {
  pl->row_tiles = ceil_div_i(rows, 160);
  const int per = ceil_div_i(rows, pl->row_tiles);
  pl->cols = per <= 16 ? 16 : ceil_div_i(per, 32) * 32;
}

// The most splits for a number of tiles.  A unit is a KV head's row tile.  One CTA
// fits an SM (two with up to 32 rows); a wave has as many splits of each unit as fit
// the SMs together, rounded down (96 units leave 56 of 152 SMs without work), and
// there are as many whole waves as keep each split's chain of sums short.
int most_splits(int heads, const SharedPlan& pl, long long tiles) {
  const int sms = device_sm_count() > 0 ? device_sm_count() : 152;
  const long long units = static_cast<long long>(heads) * pl.row_tiles;
  const int wave = static_cast<int>(std::max(1LL, std::min<long long>(kMaxSharedSplits, sms * (pl.cols <= 32 ? 2 : 1) / units)));
  return wave * std::min(kMaxSharedSplits / wave, std::max(1, ceil_div_i(tiles, static_cast<long long>(kSharedChainTiles) * wave)));
}

}  // namespace

int shared_splits_max(const kvq_cache_desc& prefix, int rows) {
  SharedPlan pl{};
  shared_rows(rows, &pl);
  // the most tiles: all of the capacity, and the residual's up to 2 G - 1 tokens
  return most_splits(prefix.num_kv_heads, pl, ceil_div_i(prefix.capacity_tokens, kSharedTile) + ceil_div_i(2 * prefix.group_size - 1, kSharedTile));
}

int shared_zero_floats(int rows) {
  SharedPlan pl{};
  shared_rows(rows, &pl);
  return pl.row_tiles * pl.cols;
}

SharedPlan shared_plan(const kvq_cache_desc& prefix, int rows, int tiles) {
  SharedPlan pl{};
  shared_rows(rows, &pl);
  pl.per = std::max(1, ceil_div_i(tiles, most_splits(prefix.num_kv_heads, pl, tiles)));
  pl.S = ceil_div_i(tiles, pl.per);
  return pl;
}

cudaError_t launch_shared(const SharedParams& p, int mode, const SharedPlan& plan, cudaStream_t s) {
  const bool mod = p.cap2 > 0.f || p.slopes || p.first || p.window > 0;
  switch (mode) {
    case KVQ_MODE_INT8: return mod ? shared_launch_m<KVQ_MODE_INT8, true>(p, plan, s) : shared_launch_m<KVQ_MODE_INT8, false>(p, plan, s);
    case KVQ_MODE_INT4: return mod ? shared_launch_m<KVQ_MODE_INT4, true>(p, plan, s) : shared_launch_m<KVQ_MODE_INT4, false>(p, plan, s);
    case KVQ_MODE_INT2: return mod ? shared_launch_m<KVQ_MODE_INT2, true>(p, plan, s) : shared_launch_m<KVQ_MODE_INT2, false>(p, plan, s);
    case KVQ_MODE_INT1: return mod ? shared_launch_m<KVQ_MODE_INT1, true>(p, plan, s) : shared_launch_m<KVQ_MODE_INT1, false>(p, plan, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
