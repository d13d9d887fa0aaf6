// cache_common.cuh -- what the kernels of the 8-bit paged cache share: the cache's view, code
// conversions, the scale rule, and the plan that spreads attention over the grid.
#pragma once

#include <cuda.h>  // CUtensorMap (type only)
#include <cuda_fp16.h>
#include <limits.h>
#include <math_constants.h>

#include "../../include/attn_cache_gb300.h"
#include "common.cuh"
#include "internal.h"

namespace attn {
namespace cache {

// Device status bits, beside those of common.cuh.
enum : unsigned {
  kStatusBadPage = 8u,        // a page id outside the cache, or a length outside the table
  kStatusNonFinite = 16u,     // an appended value was infinite or NaN
};

// The cache and the sequences of a call, as kernels take them.
struct View {
  int num_pages, page_shift, page, Hkv, D;
  uint8_t *k, *v;
  float *k_scale, *v_scale;
  unsigned *status;
  int B, max_pages;
  const int *table;
  long long table_stride;
  const int *lengths;
};

// Length of sequence b, brought into [0, table's end]; *bad is set when it was outside.
__device__ __forceinline__ int seq_len(const View &c, int b, bool *bad) {
  const int n = c.lengths[b];
  const long long cap = (long long)c.max_pages << c.page_shift;
  *bad = n < 0 || n > cap;
  return n < 0 ? 0 : (int)(n > cap ? cap : n);
}
__device__ __forceinline__ int seq_len(const View &c, int b) {
  bool bad;
  return seq_len(c, b, &bad);
}

// Page that holds position pos of sequence b, or -1 (recorded) if its id is outside the cache.
__device__ __forceinline__ int page_of(const View &c, int b, int pos) {
  const int id = c.table[b * c.table_stride + (pos >> c.page_shift)];
  if ((unsigned)id < (unsigned)c.num_pages) return id;
  set_status(c.status, kStatusBadPage);
  return -1;
}

// Row of codes (in elements) of slot `slot` of a page, for kv head h: 64-bit, as a cache may hold
// more than 2^32 codes.
__device__ __forceinline__ size_t row_at(const View &c, int page, int h, int slot) {
  return ((((size_t)page * c.Hkv + h) << c.page_shift) + slot) * c.D;
}

constexpr int kMinScaleExp = -60;  // least scale 2^-60: smaller magnitudes round to coarser steps or 0
constexpr float kMinScale = 8.673617379884035e-19f;

template <int KIND> __device__ __forceinline__ constexpr float qmax() { return KIND == ATTN_CACHE_E4M3 ? 448.f : 127.f; }

// The least power of two s >= 2^-60 with amax <= qmax * s (amax finite, >= 0): the exponent of
// amax / qmax rounded up, taken from amax's own bits.  448 = 1.75 * 2^8 and 127 = 1.984375 * 2^6,
// so amax = m * 2^e (1 <= m < 2) needs e - 8 (e - 6), and one more if m is above that mantissa.
template <int KIND> __device__ __forceinline__ float need_scale(float amax) {
  const unsigned u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127;  // below -126 for subnormals: the lower bound takes over
  const unsigned m = u & 0x7fffffu;
  int x = KIND == ATTN_CACHE_E4M3 ? e - 8 + (m > 0x600000u) : e - 6 + (m > 0x7e0000u);
  if (x < kMinScaleExp) x = kMinScaleExp;
  return __uint_as_float((unsigned)(x + 127) << 23);
}

// 1 / s for a power of two s in [2^-60, 2^120]: exact.
__device__ __forceinline__ float pow2_inverse(float s) { return __uint_as_float(0x7f000000u - __float_as_uint(s)); }

// Two codes from two values already in units of their scale: rounded to nearest even, saturated.
template <int KIND> __device__ __forceinline__ unsigned encode2(float lo, float hi) {
  if (KIND == ATTN_CACHE_E4M3) {
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
  }
  // Adding 1.5 * 2^23 leaves the rounded integer in the low bits (a conversion would go to a slower unit).
  const float a = fminf(fmaxf(lo == lo ? lo : 0.f, -127.f), 127.f) + 12582912.f;
  const float b = fminf(fmaxf(hi == hi ? hi : 0.f, -127.f), 127.f) + 12582912.f;
  return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040) & 0xffffu;
}

// Four codes of a word as floats.  e4m3 by way of fp16, which holds it exactly; int8: code + 128 under
// the bits of 2^23, less 2^23 + 128.
template <int KIND> __device__ __forceinline__ void decode4(unsigned w, float *x) {
  if (KIND == ATTN_CACHE_E4M3) {
    unsigned lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo)), b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  } else {
    const unsigned u = w ^ 0x80808080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = __uint_as_float(__byte_perm(u, 0x4b000000u, 0x7540 + i)) - 8388736.f;
  }
}

// Maximum that keeps a NaN, so that a row with a NaN logit ends as NaN and not as an empty row.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// ---------------------------------------------------------------- attention

struct FwdParams {
  View c;
  int Sq, Hq, G, R;      // R = G * Sq: query rows of one (sequence, kv head); row r is query r / G,
                         // head h * G + r % G
  int row_tile, NG, RT;  // rows per work item; RT = ceil(R / row_tile); NG = B * RT groups (b, tile)
  int splits;            // shares of every item's keys (tcgen05 path), or 0
  int cluster;           // CTAs of the cluster that has an item (tensor-core path), or 0: items split over the grid
  int unit_shift;        // keys of one unit of work: a slice for each warp of a CTA
  int max_ctas;
  int causal, window;
  float cap, inv_cap, scale;
  const void *q;
  long long q_sb, q_ss, q_sh;
  const float *sink;
  int off_by_one;
  void *O;
  float *LSE;
  const float *w_in;
  float *w_out;
  long long w_sb, w_sh;
  // workspace
  int *prefix;           // [NG + 1]: units of the groups before each; prefix[NG]: units of one kv head
  float *o_part;         // [2 * max_ctas or items * splits, row_tile, D]: unnormalised partial outputs
  float2 *ml_part;       // [the same, row_tile]: exponent reference (base 2) and sum
  float *scores;         // [B * Hkv, R, Lpad]: logits times log2(e), -inf where unseen
  long long Lpad;
};

// The query of row r (a division only where there is more than one).
__device__ __forceinline__ int query_of(const FwdParams &p, int r) { return p.Sq == 1 ? 0 : r / p.G; }

// The keys [lo, hi) that some row of a group's tile sees; lo rounded down to 64 keys (the slices of a
// warp, 16 to 64 keys, start on multiples of their size, so that they lie in one page or in whole pages).
struct Range {
  int lo, hi, len;
};
__device__ __forceinline__ Range group_range(const FwdParams &p, int b, int rt) {
  Range g;
  g.len = seq_len(p.c, b);
  g.hi = g.len;
  g.lo = 0;
  if (p.causal | (p.window > 0)) {
    const int r0 = rt * p.row_tile, r1 = min(p.R, r0 + p.row_tile) - 1, q0 = g.len - p.Sq;  // position of query 0
    if (p.causal) g.hi = max(0, min(g.len, q0 + query_of(p, r1) + 1));
    if (p.window > 0) g.lo = min(g.hi, max(0, q0 + query_of(p, r0) - p.window + 1) & ~63);
  }
  return g;
}
__device__ __forceinline__ int range_units(const FwdParams &p, const Range &g) { return (g.hi - g.lo + (1 << p.unit_shift) - 1) >> p.unit_shift; }

// U units over at most max_ctas CTAs, as evenly as they go: the first `extra` CTAs have one more.
struct Shares {
  int C, each, extra;
  __device__ __forceinline__ Shares(int U, int max_ctas) {
    C = min(U, max_ctas);
    each = C ? U / C : 0;
    extra = U - each * C;
  }
  __device__ __forceinline__ int begin(int c) const { return c * each + min(c, extra); }
  __device__ __forceinline__ int owner(int u) const {  // the CTA whose share holds unit u
    const int big = extra * (each + 1);
    return u < big ? u / (each + 1) : extra + (u - big) / each;
  }
};

// log2 of the exponentials' unit: logits are kept in base 2.
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

cudaError_t launch_fwd_simt(const FwdParams &p, int dtype, int kind, cudaStream_t st);
int simt_row_tile();
int simt_unit_shift();

// Tensor-core path.
bool mma_supported(int D);
int mma_columns(int D);
int mma_row_tile(int dtype, int D, int R);
int mma_ctas_per_sm(int D, int row_tile);
int mma_unit_shift(int D);
int mma_cluster(const FwdParams &p);
cudaError_t launch_fwd_mma(const FwdParams &p, int dtype, int kind, cudaStream_t st);
cudaError_t launch_mma_e4m3(const FwdParams &p, int dtype, cudaStream_t st);
cudaError_t launch_mma_int8(const FwdParams &p, int dtype, cudaStream_t st);
// tcgen05 path (many rows).
bool tc_supported_rows(int dtype, int D, int R, int B, int Hkv);
int tc_row_tile();
int tc_unit_shift();
int tc_splits(const FwdParams &p);
cudaError_t launch_fwd_tc(const FwdParams &p, int kind, cudaStream_t st);
bool make_tmap_codes(CUtensorMap *m, const void *base, int D, int page, long long heads, int box_cols, int box_rows);

cudaError_t launch_fwd_join(const FwdParams &p, int dtype, cudaStream_t st);
cudaError_t launch_weights(const FwdParams &p, cudaStream_t st);

// Launches a kernel that may begin before the one ahead of it in the stream has ended (programmatic
// dependent launch): it has to call grid_wait() before it touches anything of an earlier kernel, in every
// block, so that what follows it is ordered behind both.
template <typename... P, typename... A>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return counted(cudaLaunchKernelEx(&cfg, kernel, args...));
}
// Waits until the kernels ahead have ended and their writes are visible.
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// Lets the next kernel's blocks start (they wait above for this grid's end).
__device__ __forceinline__ void grid_launch_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// A kernel's limit of dynamic shared memory, raised once per device.
template <typename K> cudaError_t raise_smem(K kernel, std::atomic<unsigned long long> &done, size_t bytes) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (bit && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

struct AppendParams {
  View c;
  int S, span;  // span: pages that S tokens can touch
  const void *k, *v;
  long long k_sb, k_ss, k_sh, v_sb, v_ss, v_sh;
  const int *counts;
  int *lengths_out;
  float *weights;
  long long w_sb, w_sh;
};
cudaError_t launch_append(const AppendParams &p, int dtype, int kind, cudaStream_t st);

struct EvictParams {
  View c;
  int keep, first, recent, out_pages;
  const float *weights;
  long long w_sb, w_sh;
  const int *table_out;
  long long table_out_stride;
  int *kept, *lengths_out;
  float *weights_out;
  long long wo_sb, wo_sh;
};
cudaError_t launch_evict(const EvictParams &p, int kind, cudaStream_t st);

}  // namespace cache
}  // namespace attn
