// cache_mma.cu -- which form the tensor-core attention over the 8-bit cache takes (host).
#include <algorithm>
#include <cmath>

#include "cache_common.cuh"

namespace attn {
namespace cache {

bool mma_supported(int D) { return D <= 256; }

// The columns that the kernel for head dim D is compiled for.  Measured at 4 rows of some 115,000 keys, 8 kv
// heads, 4 queries to each: D = 96 138 us (5.5 TB/s; one such row on FFMA 587), D = 192 300 us (5.1 TB/s), D = 80
// 218 us (2.9 TB/s: rows of 80 bytes do not lie on the 32-byte sectors).
int mma_columns(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

// Rows of a work item: 16, or 32 where there are more rows than that and the accumulators fit
// (bf16, head dims up to 128), so that widening a code serves two row tiles.
int mma_row_tile(int dtype, int D, int R) { return dtype == kBF16 && R > 16 && D <= 128 ? 32 : 16; }

int mma_unit_shift(int D) { return D <= 64 ? 8 : D <= 128 ? 7 : 6; }  // four slices

int mma_ctas_per_sm(int D, int row_tile) {
  return row_tile == 32 || D > 128 ? 2 : 3;  // Cfg's CTAS
}

// How the work is spread.  A cluster of CTAs for each item (sequence, kv head, row tile) joins its parts in
// shared memory: one launch, and a CTA has one run, but the longest row decides.  Splitting all items' keys
// evenly over one wave of CTAs balances any lengths, at the cost of a plan, of parts through memory and of a
// second launch.  The host knows the table's width, not the lengths: it takes clusters where one wave of
// them ends before the split would, counted in slices of a warp (1.1 us each, whatever the head dim), full
// rows against rows half full.  kStart: a CTA's start and end; kSplit: the plan and the join.  Measured (us,
// cluster / split): 1 x 1531 keys at D = 256 12.4 / 14.4; at D = 128 with 8 kv heads 4 x 2000 12.4 / 14.4,
// 4 x 8000 22.6 / 24.7, 2 x 16000 31.1 / 24.5 (split taken); clusters in several waves lose (32 x 4000:
// 53 to 78 / 55; 64 ragged rows at D = 64 46 to 99 / 47).
int mma_cluster(const FwdParams &p) {
  constexpr double kStart = 4, kSplit = 6;
  const long long items = (long long)p.NG * p.c.Hkv;
  long long keys = (long long)p.c.max_pages << p.c.page_shift;
  if (p.window > 0) keys = std::min(keys, (long long)p.window + p.Sq);
  const double units = (double)((keys >> p.unit_shift) + 1);  // a unit: a slice for each warp
  const long long slots = (long long)mma_ctas_per_sm(p.c.D, p.row_tile) * device_sm_count();
  double best = kStart + kSplit + std::ceil(0.5 * items * units / slots);
  int cluster = 0;
  for (int c = 1; c <= 8 && items * c <= slots; c *= 2) {
    const double t = kStart + std::ceil(units / c);
    if (t < best) {
      best = t;
      cluster = c;
    }
  }
  return cluster;
}

cudaError_t launch_fwd_mma(const FwdParams &p, int dtype, int kind, cudaStream_t st) {
  return kind == ATTN_CACHE_E4M3 ? launch_mma_e4m3(p, dtype, st) : launch_mma_int8(p, dtype, st);
}

}  // namespace cache
}  // namespace attn
