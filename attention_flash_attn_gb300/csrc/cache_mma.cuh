// cache_mma.cuh -- attention over the 8-bit cache on the tensor cores, head dims up to 256 (instantiated for
// each kind of code in its own file).  Compiled for 64, 128 and 256 columns; a head dim in between takes the
// next larger form, whose further columns TMA fills with zeros: they cost products, but no bytes of memory.
//
// Decoding reads 2 D bytes of codes per key and kv head and does 4 D flops per byte and query row, so
// with the few rows of a step (G heads share a kv head) it is bound by memory; what can keep it from
// that is the work per byte: widening codes, loads from shared memory, softmax.  Hence:
//   - Each warp works alone.  It owns a ring of slices (SK keys of K and V), lane 0 fills it by TMA
//     (the table's page ids and the scales of 32 slices ahead sit one per lane in registers), and no
//     warp waits for another until a run of units ends.
//   - Codes go from shared memory to registers 16 at a time in the order in which the MMA wants its B
//     operand, whatever that does to the order of d (both products are free to permute what they sum
//     over, and Q is laid out to match), and are widened there to fp16, exactly; no shuffles, no second
//     copy.  m16n8k16 with fp16 operands: rows of Q (or P) as A, 8 keys (or 8 columns of V) as B.
//   - TMA's swizzle makes both 16-byte access patterns free of bank conflicts.
//   - Q is scaled per row by a power of two into fp16's range: exact for elements within 2^-31 of the
//     row's largest.
//   - P is rounded to fp16 (half a step: 2^-11 of each probability, eight times finer than the bf16 result), times
//     2^14, so that the many small probabilities beside a large one keep their bits down to 2^-28 of it (held
//     as they are, from 2^-14 on they did not, and below 2^-25 they were 0, while the sum counted them).
//   - float queries take the same way in two terms each: q = hi + lo in fp16 (22 bits), p 2^14 = hi + lo, both
//     terms multiplied into the same accumulators.  Twice the MMAs; a call on the FFMA kernel took 39 us where
//     it took 26 with this one, now 25 (9 ragged rows up to 9001 keys, one kv head, a join and a weights pass in each).
// Measured at 4 rows of some 115,000 keys, 8 kv heads, 4 bf16 queries to each: 5.0 TB/s at D = 64, 6.0 at 128, 6.5
// at 256 (a copy reaches 6.8); float queries at D = 128 5.3.  Registers: most forms of 64 and 128 columns spill, up to
// 92 bytes a thread, within what two or three CTAs to an SM leave them.  Short calls are bound by the fixed parts, some 12 us:
// launch, plan and first loads, the last run's end, the join.  With a row tile of 32, or D = 64 (half the bytes
// per score), the warps' issue slots and latencies bound it, not the memory.
#pragma once
#include "cache_work.cuh"
#include "tc_common.cuh"

namespace attn {
namespace cache {
namespace {

using namespace attn::tc;

constexpr int kWarps = kThreads / 32;
constexpr float kZeroLog = kMinScaleExp - 1;
constexpr float kPShift = 14;  // probabilities (at most 1) are held times 2^14: fp16 is normal down to 2^-28 of the row's largest

template <typename T, int D_, int MT_>
struct Cfg {
  static constexpr int D = D_, MT = MT_;
  static constexpr int TERMS = sizeof(T) == 4 ? 2 : 1;  // fp16 terms of a query element and of a probability
  static constexpr int SK = D == 256 ? 16 : D == 128 ? 32 : 64;  // keys of a slice: 8 KB of codes
  static constexpr int NH = SK / 16;                   // groups of 16 keys: each lies in one page
  static constexpr int BLK = D < 128 ? D : 128;        // columns of one TMA box row
  static constexpr int NB = D / BLK;                   // boxes per row
  static constexpr int CH = BLK / 64;                  // 16-byte chunks per lane and key for Q K^T
  static constexpr int KS = D / 16;                    // k-steps of Q K^T
  static constexpr int NT = D / 8;                     // n-tiles of P V
  static constexpr int QG = SK < 32 ? SK / 8 : 4;      // n-tiles of Q K^T whose codes are in registers at once
  static constexpr bool SPLIT = D == 256;               // scores in two accumulators
  static constexpr int STAGE = 2 * SK * D;             // bytes of a slice, K then V
  static constexpr int DEPTH = 2;
  static constexpr int CTAS = MT == 1 && D <= 128 ? 3 : 2;
  static constexpr bool QREG = D * MT * TERMS <= 64;   // Q fragments in registers, else in shared memory
  static constexpr int ROWS = 16 * MT;
  static_assert(NB == 1 || NH == 1, "a slice of several pages has one box per page");
  static constexpr size_t RING = (size_t)kWarps * DEPTH * STAGE;
  static_assert(DEPTH * STAGE >= ROWS * D * 4, "a warp's output fits its ring at the end of a run");
  static constexpr size_t Q_BYTES = QREG ? 0 : (size_t)TERMS * MT * KS * 32 * 16;
  static constexpr size_t ML_BYTES = (size_t)kWarps * ROWS * 8;
  static constexpr size_t NAN_BYTES = (size_t)ROWS * D / 8;  // one bit per output of the run
  static constexpr size_t SMEM = 1024 + RING + Q_BYTES + ML_BYTES + ROWS * 8 + NAN_BYTES + kWarps * DEPTH * 8;
};

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

// Reads of another cluster CTA's shared memory (`at`: this CTA's address of the same thing).
__device__ __forceinline__ uint32_t dsmem_at(uint32_t at, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(at), "r"(rank));
  return r;
}
__device__ __forceinline__ float2 dsmem_f2(uint32_t at, int rank) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(dsmem_at(at, rank)));
  return v;
}
__device__ __forceinline__ float4 dsmem_f4(uint32_t at, int rank) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(dsmem_at(at, rank)));
  return v;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ void mma_f16(float *c, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(const uint8_t *at) { return *reinterpret_cast<const uint4 *>(at); }
__device__ __forceinline__ uint2 lds64(const uint8_t *at) { return *reinterpret_cast<const uint2 *>(at); }

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// What a pair in fp16 leaves of the values it was rounded from, in fp16 (0 where they are not finite, so
// that the sum is what it would be without).
__device__ __forceinline__ uint32_t rest_h2(uint32_t h, float lo, float hi) {
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  const float a = lo - f.x, b = hi - f.y;
  return pack_h2(fabsf(a) <= 3.402823466e38f ? a : 0.f, fabsf(b) <= 3.402823466e38f ? b : 0.f);
}

// Elements x and x + 1 (x even) of a lane's part of a query row.
template <typename T> __device__ __forceinline__ void q_pair(const uint4 *raw, int x, float &a, float &b) {
  if (sizeof(T) == 4) {
    const uint4 &u = raw[x / 4];
    a = __uint_as_float(x % 4 ? u.z : u.x);
    b = __uint_as_float(x % 4 ? u.w : u.y);
  } else {
    const uint4 &u = raw[x / 8];
    const uint32_t w = x % 8 == 0 ? u.x : x % 8 == 2 ? u.y : x % 8 == 4 ? u.z : u.w;
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
  }
}

// Four codes of a word widened to two fp16 pairs, exactly.  int8: code + 128 under the bits of 1024
// is 1152 + code in fp16.
template <int KIND> __device__ __forceinline__ void widen4(uint32_t w, uint32_t &lo, uint32_t &hi) {
  if (KIND == ATTN_CACHE_E4M3) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(w));
  } else {
    const uint32_t u = w ^ 0x80808080u;
    const __half2 bias = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));  // 1152
    uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
    __half2 x = __hsub2(*reinterpret_cast<__half2 *>(&a), bias), y = __hsub2(*reinterpret_cast<__half2 *>(&b), bias);
    lo = *reinterpret_cast<uint32_t *>(&x);
    hi = *reinterpret_cast<uint32_t *>(&y);
  }
}

// cap * tanh(u / cap) * log2(e) with y = 2 log2(e) u / cap: 1 - 2 / (1 + 2^y).  Absolute error some
// steps of the cap; saturates cleanly (2^y = inf gives 1, 0 gives -1).
__device__ __forceinline__ float softcap_log2(float y, float cap_log2) {
  return cap_log2 - __fdividef(2.f * cap_log2, 1.f + ex2(y));
}

__device__ __forceinline__ void put4(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
__device__ __forceinline__ void put4(__nv_bfloat16 *p, float4 x) {
  __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
}

// Byte offset of 16-byte chunk `ch` of key row `row` in a box, under TMA's swizzle.
template <int BLK> __device__ __forceinline__ uint32_t swz(int row, int ch) {
  if (BLK == 128) return row * 128 + ((ch ^ (row & 7)) << 4);
  return row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
}

// A 16-byte chunk of values of key `pos` (columns d ..) with e4m3 NaNs in it: the outputs that they belong
// to -- of the rows that see the key -- are marked in s_nan, and they become 0.
template <int D>
__device__ __noinline__ void mark_nans(const FwdParams &p, uint4 *at, int pos, int d, int len, int r0, int rows, uint32_t *s_nan, int *s_any) {
  uint8_t *code = reinterpret_cast<uint8_t *>(at);
  for (int x = 0; x < 16; ++x) {
    if ((code[x] & 0x7f) != 0x7f) continue;
    code[x] = 0;
    for (int r = 0; r < rows; ++r)
      if (within(row_sees(p, len, query_of(p, r0 + r)), pos)) {
        atomicOr(s_nan + (r * D + d + x) / 32, 1u << ((d + x) % 32));
        *s_any = 1;
      }
  }
}

// Makes a slice's values fit to be multiplied by P where some row does not see every key: rows of
// keys that no row sees (slots behind the last token may hold anything) become 0, and so do e4m3 NaNs,
// whose outputs are marked.  A run's first and last slices come here.
template <typename T, int KIND, int D, int MT>
__device__ __forceinline__ void scrub_values(const FwdParams &p, uint8_t *sv, int pos, int key1, unsigned gone, int len, int r0, int rows,
                                             uint32_t *s_nan, int *s_any) {
  using C = Cfg<T, D, MT>;
  constexpr int kChunks = C::SK * D / 16 / 32;  // per lane
  const int lane = threadIdx.x & 31;
  auto at = [&](int i, int *row, int *c) {
    const int x = lane + 32 * i;
    *row = x / (D / 16);
    *c = x % (D / 16);
    return reinterpret_cast<uint4 *>(sv + (*c / (C::BLK / 16)) * (C::SK * C::BLK) + swz<C::BLK>(*row, *c % (C::BLK / 16)));
  };
  unsigned nans = 0;
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    int row, c;
    uint4 *u = at(i, &row, &c);
    if (pos + row >= key1 || ((gone >> (row >> 4)) & 1u)) {
      *u = make_uint4(0, 0, 0, 0);
    } else if (KIND == ATTN_CACHE_E4M3) {
      const uint4 v = *u;  // a byte of 0x7f, and no other, carries into its top bit
      const uint32_t any = ((v.x & 0x7f7f7f7fu) + 0x01010101u) | ((v.y & 0x7f7f7f7fu) + 0x01010101u) |
                           ((v.z & 0x7f7f7f7fu) + 0x01010101u) | ((v.w & 0x7f7f7f7fu) + 0x01010101u);
      if (any & 0x80808080u) nans |= 1u << i;
    }
  }
  while (nans) {
    const int i = __ffs(nans) - 1;
    nans &= nans - 1;
    int row, c;
    uint4 *u = at(i, &row, &c);
    mark_nans<D>(p, u, pos + row, c * 16, len, r0, rows, s_nan, s_any);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the stage's next fill comes by TMA
  __syncwarp();
}

// recount for rows r0 .. r0 + rows - 1 of (kv head, sequence) pair `hb`, whose references and sums lie in ml.  Called by a warp.
template <typename T, int KIND>
__device__ __noinline__ void recount_rows(const FwdParams &p, int hb, int r0, int len, Keys keys, float2 *ml, int rows) {
  const int hk = hb / p.c.B, b = hb - hk * p.c.B;
  if (!far_apart(p, b, hk, keys)) return;
#pragma unroll 1
  for (int r = 0; r < rows; ++r) {
    const float sum = recount<T, KIND>(p, b, hk, r0 + r, len, keys, ml[r].x);
    if ((threadIdx.x & 31) == 0) ml[r].y = sum;
  }
}

template <typename T, int KIND, int D, int MT>
__global__ void __launch_bounds__(kThreads, (Cfg<T, D, MT>::CTAS))
cache_fwd_mma_kernel(const __grid_constant__ FwdParams p, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap) {
  using C = Cfg<T, D, MT>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ int s_any, s_large;  // s_large: a value scale so large that others may be too far below it (see cache_work.cuh)
  const uint32_t raw = smem_u32(smem_raw), ring0 = (raw + 1023u) & ~1023u;
  uint8_t *base = smem_raw + (ring0 - raw);
  uint4 *s_q = reinterpret_cast<uint4 *>(base + C::RING);                                      // [TERMS][MT][KS][32]
  float2 *s_ml = reinterpret_cast<float2 *>(base + C::RING + C::Q_BYTES);                      // [kWarps][ROWS]
  float2 *s_cta = s_ml + kWarps * C::ROWS;                                                     // [ROWS]: the CTA's, for its cluster
  uint32_t *s_nan = reinterpret_cast<uint32_t *>(s_cta + C::ROWS);                             // [ROWS][D / 32]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t ring = ring0 + warp * (C::DEPTH * C::STAGE);
  const uint32_t bars = ring0 + C::RING + C::Q_BYTES + C::ML_BYTES + C::ROWS * 8 + C::NAN_BYTES + warp * (C::DEPTH * 8);
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < C::DEPTH; ++s) mbar_init(bars + 8 * s, 1);
    fence_barrier_init();
    tma_prefetch_desc(&kmap);
    tma_prefetch_desc(&vmap);
  }
  for (int x = tid; x < C::ROWS * D / 32; x += kThreads) s_nan[x] = 0u;
  if (tid == 0) s_any = 0, s_large = 0;
  __syncthreads();  // a warp may mark NaNs as soon as its own first slice has come: not before every warp has cleared its part

  __shared__ Groups s_groups;
  Cursor cur;
  Run run;
  int rank = 0;  // in the item's cluster
  if (p.cluster) {
    const int item = blockIdx.x / p.cluster;
    rank = blockIdx.x - item * p.cluster;
    run.hk = item / p.NG;
    const int gr = item - run.hk * p.NG;
    run.b = p.RT == 1 ? gr : gr / p.RT;
    run.rt = gr - run.b * p.RT;
    run.range = group_range(p, run.b, run.rt);
    run.n = range_units(p, run.range);
    const int each = run.n / p.cluster, extra = run.n - each * p.cluster;
    run.off = rank * each + min(rank, extra);
    run.cnt = each + (rank < extra);
    if (rank == 0 && run.hk == 0 && run.rt == 0 && tid == 0) {
      bool bad;
      seq_len(p.c, run.b, &bad);
      if (bad) set_status(p.c.status, kStatusBadPage);
    }
  } else if (!cursor_begin(p, &s_groups, cur) || !cursor_next(p, &s_groups, cur, run)) {
    grid_launch_next();
    return;
  }
  uint32_t phases = 0;  // parity of each stage's next completion
  int stage = 0;
  bool dead = false;    // a wait gave up: recorded; this warp computes no further
  const float cap_log2 = p.cap * kLog2e;
  int id_nxt[C::NH];
  bool first = true;    // (id_nxt holds the page ids of every run but the first)
#pragma unroll 1
  do {
    const int r0 = run.rt * C::ROWS, rows = min(C::ROWS, p.R - r0);
    const int key0 = run.range.lo + (run.off << p.unit_shift), key1 = min(run.range.hi, key0 + (run.cnt << p.unit_shift));
    // This warp's slices: key0 + (warp + 4 x) SK for x < n_slices.
    const int n_slices = (key1 - key0 - warp * C::SK + kWarps * C::SK - 1) / (kWarps * C::SK);  // <= 0: none

    // Page ids and scales of 32 slices, one per lane, and the following batch's page ids.
    int id_now[C::NH];
    float ks_now[C::NH], lv_now[C::NH];
    unsigned odd_now = 0;  // bit x: slice x of the batch has a half without a page, or whose values count as 0
    auto load_ids = [&](int b, int from, int to, int batch, int *ids) {  // of the warp's slices in [from, to)
#pragma unroll
      for (int h = 0; h < C::NH; ++h) {
        const int pos = from + (warp + kWarps * (batch * 32 + lane)) * C::SK + 16 * h;
        ids[h] = pos < to ? page_of(p.c, b, pos) : -1;
      }
    };
    // The page ids that follow batch `batch`: of this run's next one, or of the next run's first.
    auto load_next_ids = [&](int batch) {
      if (n_slices > batch * 32 + 32) {
        load_ids(run.b, key0, key1, batch + 1, id_nxt);
      } else if (!p.cluster) {
        Cursor peek = cur;
        Run next;
        if (cursor_next(p, &s_groups, peek, next)) {
          const int from = next.range.lo + (next.off << p.unit_shift);
          load_ids(next.b, from, min(next.range.hi, from + (next.cnt << p.unit_shift)), 0, id_nxt);
        }
      }
    };
    // The scales of the batch in id_now, in two steps, so that nothing waits for them before the first
    // slice has come.  A value scale that counts as 0 has kZeroLog for its logarithm: any reference does for
    // values of 0, as long as the sum undoes it.
    auto fetch_scales = [&]() {
#pragma unroll
      for (int h = 0; h < C::NH; ++h) {
        ks_now[h] = lv_now[h] = 0.f;
        if (id_now[h] >= 0) {
          const size_t at = (size_t)id_now[h] * p.c.Hkv + run.hk;
          ks_now[h] = p.c.k_scale[at];
          lv_now[h] = p.c.v_scale[at];
        }
      }
    };
    auto take_scales = [&]() {
      bool odd = false;
#pragma unroll
      for (int h = 0; h < C::NH; ++h) {
        odd |= !(lv_now[h] >= kMinScale);
        lv_now[h] = lv_now[h] >= kMinScale ? log2f(lv_now[h]) : kZeroLog;
        if (lv_now[h] > kFarTop) s_large = 1;
      }
      odd_now = __ballot_sync(~0u, odd);
    };
    // Fills ring stage `st` with slice x (ids: its batch).  All lanes call it; lane 0 issues, or, where a
    // slice spans several pages, a lane for each.  `hold` is 0, known only once the stage's loads have come.
    auto issue = [&](int x, int st, const int *ids, uint32_t hold) {
      const uint32_t bar = bars + 8 * st + hold, dst = ring + st * C::STAGE + hold;
      const int pos = key0 + (warp + kWarps * x) * C::SK;
      const int slot = pos & (p.c.page - 1);
      int id = __shfl_sync(~0u, ids[0], x & 31);
      if (C::NH == 1 || p.c.page >= C::SK) {
        if (lane == 0) {
          mbar_arrive_expect_tx(bar, id >= 0 ? C::STAGE : 0);
          if (id >= 0) {
            const int head = id * p.c.Hkv + run.hk;
#pragma unroll
            for (int j = 0; j < C::NB; ++j) {
              tma_load_3d(dst + j * (C::SK * C::BLK), &kmap, bar, j * C::BLK, slot, head);
              tma_load_3d(dst + C::SK * D + j * (C::SK * C::BLK), &vmap, bar, j * C::BLK, slot, head);
            }
          }
        }
      } else {
        const int boxes = C::SK >> p.c.page_shift, groups = C::NH / boxes;  // (each slice begins a page)
#pragma unroll
        for (int h = 1; h < C::NH; ++h) {
          const int other = __shfl_sync(~0u, ids[h], x & 31);
          if (h == lane * groups) id = other;
        }
        const bool has = lane < boxes && id >= 0;
        const unsigned count = __popc(__ballot_sync(~0u, has));
        if (lane == 0) mbar_arrive_expect_tx(bar, count * (2 * D << p.c.page_shift));
        __syncwarp();
        if (has) {
          const int head = id * p.c.Hkv + run.hk;
          const uint32_t to = dst + ((lane * C::BLK) << p.c.page_shift);
          tma_load_3d(to, &kmap, bar, 0, 0, head);
          tma_load_3d(to + C::SK * D, &vmap, bar, 0, 0, head);
        }
      }
    };

    // Queries: rows g and g + 8 of each 16, this lane's columns; asked for before anything that waits.
    constexpr int kQW = D * (int)sizeof(T) / 64;  // 16-byte words of a row's quarter
    uint4 raw_q[MT][2][kQW];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int r = r0 + mt * 16 + 8 * y + g, i = query_of(p, r), h = run.hk * p.G + (r - i * p.G);
        const T *row = static_cast<const T *>(p.q) + run.b * p.q_sb + i * p.q_ss + h * p.q_sh + t * (C::BLK / 4);
#pragma unroll
        for (int z = 0; z < kQW; ++z) {
          constexpr int kPerBlk = kQW / C::NB, kEl = 16 / (int)sizeof(T);
          raw_q[mt][y][z] = make_uint4(0, 0, 0, 0);
          const int at = (z / kPerBlk) * C::BLK + (z % kPerBlk) * kEl;
          if (r < p.R && at + t * (C::BLK / 4) < p.c.D) raw_q[mt][y][z] = *reinterpret_cast<const uint4 *>(row + at);
        }
      }

    if (first) load_ids(run.b, key0, key1, 0, id_nxt);
    first = false;
#pragma unroll
    for (int h = 0; h < C::NH; ++h) id_now[h] = id_nxt[h];
    int filled = dead ? 0 : min(C::DEPTH, n_slices);  // slices asked for
#pragma unroll 1
    for (int s = 0; s < filled; ++s) issue(s, stage + s >= C::DEPTH ? stage + s - C::DEPTH : stage + s, id_now, 0u);
    fetch_scales();
    if (n_slices <= 0) load_next_ids(0);

    // The queries scaled into fp16.
    uint32_t qf[C::QREG ? MT : 1][C::QREG ? C::KS : 1][4];
    float q_mul[MT][2];  // what undoes the scaling, times the softmax scale (and log2 e without a cap)
    int see_lo[MT][2], see_n[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      float up[2];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int2 see = row_sees(p, run.range.len, query_of(p, r0 + mt * 16 + 8 * y + g));
        see_lo[mt][y] = see.x;
        see_n[mt][y] = max(0, min(see.y, key1) - see.x);
        float amax = 0.f;
#pragma unroll
        for (int x = 0; x < D / 4; x += 2) {
          float q0, q1;
          q_pair<T>(raw_q[mt][y], x, q0, q1);
          amax = max_nan(amax, fabsf(q0), fabsf(q1));
        }
        amax = max_nan(amax, __shfl_xor_sync(~0u, amax, 1));
        amax = max_nan(amax, __shfl_xor_sync(~0u, amax, 2));
        // 2^x that brings the largest element into [2^14, 2^15); 1 for rows that are 0 or not finite.
        int x = 14 - ((int)(__float_as_uint(amax) >> 23) - 127);
        if (!(amax > 0.f) || !(amax <= 3.402823466e38f)) x = 0;
        x = x > 126 ? 126 : x;
        up[y] = copysignf(__uint_as_float((unsigned)(x + 127) << 23), p.scale);
        // (The capped logit's argument: of 2^y for bf16, see softcap_log2, of tanh for float.)
        const float unit = p.cap > 0.f ? (C::TERMS == 1 ? 2.f * kLog2e * p.inv_cap : p.inv_cap) : kLog2e;
        q_mul[mt][y] = __uint_as_float((unsigned)(127 - x) << 23) * fabsf(p.scale) * unit;
      }
      // A fragment of k-step s: columns 4 s .. 4 s + 3 of this lane's, of rows g and g + 8.
#pragma unroll
      for (int s = 0; s < C::KS; ++s) {
        uint32_t f[C::TERMS][4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float q0, q1;
          q_pair<T>(raw_q[mt][e & 1], 4 * s + 2 * (e >> 1), q0, q1);
          q0 *= up[e & 1];
          q1 *= up[e & 1];
          f[0][e] = pack_h2(q0, q1);
          if (C::TERMS == 2) f[C::TERMS - 1][e] = rest_h2(f[0][e], q0, q1);
        }
#pragma unroll
        for (int w = 0; w < C::TERMS; ++w) {
          if (C::QREG) {
#pragma unroll
            for (int e = 0; e < 4; ++e) qf[C::QREG ? mt : 0][C::QREG ? s : 0][e] = f[w][e];
          } else if (warp == 0) {
            s_q[((w * MT + mt) * C::KS + s) * 32 + lane] = make_uint4(f[w][0], f[w][1], f[w][2], f[w][3]);
          }
        }
      }
    }
    if (!C::QREG) __syncthreads();  // (the previous run's reads of s_q ended before its own barriers)

    float m[MT][2], l[MT][2], o[MT][C::NT][4];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        m[mt][y] = -CUDART_INF_F;
        l[mt][y] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < C::NT; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x) o[mt][n][x] = 0.f;
    }
    // The keys that every row of the tile sees (rows' positions ascend).
    const int all_from = row_sees(p, run.range.len, query_of(p, r0 + rows - 1)).x;
    const int all_below = min(key1, row_sees(p, run.range.len, query_of(p, r0)).y);

#pragma unroll 1
    for (int x = 0; x < n_slices; ++x) {
      const int pos = key0 + (warp + kWarps * x) * C::SK;
      if (x > 0 && (x & 31) == 0) {
#pragma unroll
        for (int h = 0; h < C::NH; ++h) id_now[h] = id_nxt[h];
        fetch_scales();
      }
      uint8_t *const sk = base + (warp * C::DEPTH + stage) * C::STAGE, *const sv = sk + C::SK * D;
      // (Copies in flight are waited for even then: they end in this CTA's memory.)
      if (x < filled) dead |= !mbar_wait_warp(bars + 8 * stage, (phases >> stage) & 1u, p.c.status);
      phases ^= 1u << stage;
      if ((x & 31) == 0) {
        take_scales();
        load_next_ids(x >> 5);
      }
      // This slice's scales.
      float ks[C::NH], lv[C::NH];
#pragma unroll
      for (int h = 0; h < C::NH; ++h) {
        ks[h] = __shfl_sync(~0u, ks_now[h], x & 31);
        lv[h] = __shfl_sync(~0u, lv_now[h], x & 31);
      }
      const bool partial = ((odd_now >> (x & 31)) & 1u) || pos + C::SK > all_below || pos < all_from;
      if (!dead) {
        // (Two accumulators where few n-tiles would make the k-steps one long chain.)
        float s[MT][C::SK / 8][4], s2[MT][C::SPLIT ? C::SK / 8 : 1][4];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int n = 0; n < C::SK / 8; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[mt][n][e] = s2[mt][C::SPLIT ? n : 0][e] = 0.f;
        // Scores: n-tile n holds keys 8 n .. 8 n + 7, key 8 n + g on the lanes of group g.
#pragma unroll
        for (int j = 0; j < C::NB; ++j)
#pragma unroll
          for (int c = 0; c < C::CH; ++c)
#pragma unroll
            for (int n0 = 0; n0 < C::SK / 8; n0 += C::QG) {
              uint4 kw[C::QG];
#pragma unroll
              for (int n = 0; n < C::QG; ++n)
                kw[n] = lds128(sk + j * (C::SK * C::BLK) + (n0 + n) * (8 * C::BLK) + swz<C::BLK>(g, t * C::CH + c));
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                const int step = (j * C::CH + c) * 4 + w;
                uint4 qs[C::TERMS][MT];
#pragma unroll
                for (int z = 0; z < C::TERMS; ++z)
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt)
                    if (!C::QREG) qs[z][mt] = s_q[((z * MT + mt) * C::KS + step) * 32 + lane];
#pragma unroll
                for (int n = 0; n < C::QG; ++n) {
                  const uint32_t word = w == 0 ? kw[n].x : w == 1 ? kw[n].y : w == 2 ? kw[n].z : kw[n].w;
                  uint32_t b0, b1;
                  widen4<KIND>(word, b0, b1);
#pragma unroll
                  for (int z = 0; z < C::TERMS; ++z)
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                      if (C::QREG) {
                        mma_f16(s[mt][n0 + n], qf[C::QREG ? mt : 0][C::QREG ? step : 0], b0, b1);
                      } else {
                        const uint32_t a[4] = {qs[z][mt].x, qs[z][mt].y, qs[z][mt].z, qs[z][mt].w};
                        mma_f16(C::SPLIT && (w & 1) ? s2[mt][C::SPLIT ? n0 + n : 0] : s[mt][n0 + n], a, b0, b1);
                      }
                    }
                }
              }
            }
        if (C::SPLIT) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int n = 0; n < C::SK / 8; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[mt][n][e] += s2[mt][C::SPLIT ? n : 0][e];
        }
        // Softmax.  A probability is 2^(f s + lv - m): f takes a raw score to a logit in base 2 (it is not
        // negative, so that the largest raw score gives the largest logit), lv is the values' scale.  With a cap
        // or a mask the logits are formed first, and f is 1.
        float f[MT][2][C::NH];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int y = 0; y < 2; ++y)
#pragma unroll
            for (int h = 0; h < C::NH; ++h) f[mt][y][h] = q_mul[mt][y] * ks[h];
        if (partial || p.cap > 0.f) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int n = 0; n < C::SK / 8; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) s[mt][n][e] *= f[mt][e >> 1][n / 2];
          if (p.cap > 0.f) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int n = 0; n < C::SK / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[mt][n][e] = C::TERMS == 1 ? softcap_log2(s[mt][n][e], cap_log2) : cap_log2 * tanhf(s[mt][n][e]);
          }
          if (partial) {
            unsigned gone = 0, zero = 0;  // bit h: half h has no page; its values count as 0
#pragma unroll
            for (int h = 0; h < C::NH; ++h) {
              gone |= (__shfl_sync(~0u, id_now[h], x & 31) < 0 ? 1u : 0u) << h;
              zero |= (lv[h] == kZeroLog ? 1u : 0u) << h;
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int n = 0; n < C::SK / 8; ++n)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int key = pos + 8 * n + 2 * t + (e & 1);
                  if ((gone >> (n / 2) & 1u) || (unsigned)(key - see_lo[mt][e >> 1]) >= (unsigned)see_n[mt][e >> 1])
                    s[mt][n][e] = -CUDART_INF_F;
                }
            scrub_values<T, KIND, D, MT>(p, sv, pos, key1, gone | zero, run.range.len, r0, rows, s_nan, &s_any);
          }
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int y = 0; y < 2; ++y)
#pragma unroll
              for (int h = 0; h < C::NH; ++h) f[mt][y][h] = 1.f;
        }
        if (p.scores) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int y = 0; y < 2; ++y)
              if (mt * 16 + 8 * y + g < rows) {
                float *row = scores_row(p, run.b, run.hk, r0 + mt * 16 + 8 * y + g) + pos + 2 * t;
#pragma unroll
                for (int n = 0; n < C::SK / 8; ++n)
                  *reinterpret_cast<float2 *>(row + 8 * n) =
                      make_float2(f[mt][y][n / 2] * s[mt][n][2 * y], f[mt][y][n / 2] * s[mt][n][2 * y + 1]);
              }
        }
        uint32_t pf[C::TERMS][MT][C::NH][4];
        bool moved = false;
        float mn[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            float top = m[mt][y];
#pragma unroll
            for (int h = 0; h < C::NH; ++h) {
              const float a = max_nan(s[mt][2 * h][2 * y], s[mt][2 * h][2 * y + 1], s[mt][2 * h + 1][2 * y]);
              top = max_nan(top, fmaf(f[mt][y][h], max_nan(a, s[mt][2 * h + 1][2 * y + 1]), lv[h]));
            }
            top = max_nan(top, __shfl_xor_sync(~0u, top, 1));
            top = max_nan(top, __shfl_xor_sync(~0u, top, 2));
            mn[mt][y] = top;
            moved |= top != m[mt][y];
          }
        if (__any_sync(~0u, moved)) {
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float a = mn[mt][y] == -CUDART_INF_F ? 1.f : ex2(m[mt][y] - mn[mt][y]);
              m[mt][y] = mn[mt][y];
              l[mt][y] *= a;
              if (x == 0) continue;  // nothing there yet
#pragma unroll
              for (int n = 0; n < C::NT; ++n) {
                o[mt][n][2 * y] *= a;
                o[mt][n][2 * y + 1] *= a;
              }
            }
        }
#pragma unroll
        for (int h = 0; h < C::NH; ++h) {
          const float inv = ex2(-lv[h]);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const float ref = lv[h] - (m[mt][y] == -CUDART_INF_F ? 0.f : m[mt][y]) + kPShift;
              float e[4];
#pragma unroll
              for (int q = 0; q < 4; ++q) e[q] = ex2(fmaf(f[mt][y][h], s[mt][2 * h + (q >> 1)][2 * y + (q & 1)], ref));
              l[mt][y] = fmaf((e[0] + e[1]) + (e[2] + e[3]), inv, l[mt][y]);
              pf[0][mt][h][y] = pack_h2(e[0], e[1]);
              pf[0][mt][h][2 + y] = pack_h2(e[2], e[3]);
              if (C::TERMS == 2) {
                pf[C::TERMS - 1][mt][h][y] = rest_h2(pf[0][mt][h][y], e[0], e[1]);
                pf[C::TERMS - 1][mt][h][2 + y] = rest_h2(pf[0][mt][h][2 + y], e[2], e[3]);
              }
            }
        }
        // The stage is filled again as soon as every lane's loads of it have come, and not before: nothing orders a load
        // before a later copy by TMA into its place but the load's own end (it may be held up behind stores of scores), and
        // the compiler may move products past the copy.  So the copy's addresses hang on a vote over a word of each load
        // of values (p.splits is 0 here); those of keys came before the scores that the votes above went by.
        uint32_t come = 0;
        auto refill = [&]() {
          const int y = x + C::DEPTH;
          if (y >= n_slices) return;
          ++filled;
          issue(y, stage, (y >> 5) == (x >> 5) ? id_now : id_nxt, __any_sync(~0u, come == 0x9e3779b9u) ? (uint32_t)p.splits : 0u);
        };
        // O += P V: lane t has keys 2t, 2t + 1, 2t + 8, 2t + 9 of each 16 as the B operand's rows, and
        // BLK / 8 neighbouring columns, one for each n-tile.
#pragma unroll
        for (int j = 0; j < C::NB; ++j)
#pragma unroll
          for (int h = 0; h < C::NH; ++h) {
            uint32_t vw[4][C::BLK / 32];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              // Key 16 h + 8 (q >> 1) + 2 t + (q & 1): its low three bits, which the swizzle uses, are the last two terms.
              const uint8_t *at = sv + j * (C::SK * C::BLK) + (16 * h + 8 * (q >> 1)) * C::BLK;
              if (C::BLK == 128) {
                const uint4 u = lds128(at + swz<C::BLK>(2 * t + (q & 1), g));
                vw[q][0] = u.x;
                vw[q][1] = u.y;
                vw[q][C::BLK / 32 - 2] = u.z;
                vw[q][C::BLK / 32 - 1] = u.w;
                come |= u.x;
              } else {
                const uint2 u = lds64(at + swz<C::BLK>(2 * t + (q & 1), g >> 1) + (g & 1) * 8);
                vw[q][0] = u.x;
                vw[q][1] = u.y;
                come |= u.x;
              }
            }
            if (j == C::NB - 1 && h == C::NH - 1) refill();
#pragma unroll
            for (int w = 0; w < C::BLK / 32; ++w)
#pragma unroll
              for (int z = 0; z < 2; ++z) {
                const uint32_t sel = z ? 0x7362 : 0x5140;
                uint32_t b0[2], b1[2];
                widen4<KIND>(__byte_perm(vw[0][w], vw[1][w], sel), b0[0], b0[1]);
                widen4<KIND>(__byte_perm(vw[2][w], vw[3][w], sel), b1[0], b1[1]);
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int q = 0; q < C::TERMS; ++q) mma_f16(o[mt][j * (C::BLK / 8) + 4 * w + 2 * z + e], pf[q][mt][h], b0[e], b1[e]);
              }
          }
      }
      __syncwarp();
      stage = stage + 1 == C::DEPTH ? 0 : stage + 1;
    }

    if (p.cluster || cur.u >= cur.u1) grid_launch_next();  // the join's blocks may take up their places

    // The run's end: each warp leaves its rows in its ring (nothing is in flight), four columns at a time,
    // the 16-byte groups permuted so that the lanes of a store meet different banks; then all threads add
    // the four warps' rows up.
    auto o_at = [](int r, int d) {  // float index of row r, column d (a multiple of 4)
      return r * D + ((d >> 2) ^ (4 * (r & 1) + ((d / (C::BLK / 4)) & 3))) * 4;
    };
    {
      float *my = reinterpret_cast<float *>(base + warp * (C::DEPTH * C::STAGE));
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int r = mt * 16 + 8 * y + g;
          float v = l[mt][y];
          v += __shfl_xor_sync(~0u, v, 1);
          v += __shfl_xor_sync(~0u, v, 2);
          if (t == 0) s_ml[warp * C::ROWS + r] = make_float2(m[mt][y] - kPShift, dead ? CUDART_NAN_F : v);
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int n = 0; n < C::NT; n += 4) {
              // n-tile n of a block: column (BLK / 8) (2 t + e) + n.
              const int j = n / (C::BLK / 8), d = j * C::BLK + (C::BLK / 8) * (2 * t + e) + n % (C::BLK / 8);
              *reinterpret_cast<float4 *>(my + o_at(r, d)) =
                  make_float4(o[mt][n][2 * y + e], o[mt][n + 1][2 * y + e], o[mt][n + 2][2 * y + e], o[mt][n + 3][2 * y + e]);
            }
        }
    }
    __syncwarp();
    if (s_large && !dead)  // (set by this warp or another: the warp's own keys decide)
      recount_rows<T, KIND>(p, run.hk * p.c.B + run.b, r0, run.range.len, {key0 + warp * C::SK, C::SK, kWarps * C::SK, key1}, s_ml + warp * C::ROWS, rows);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the ring's next fill comes by TMA
    __syncthreads();
    const bool one_of = p.cluster > 1, whole = !one_of && run.cnt == run.n, nans = s_any != 0, large = s_large != 0;
#pragma unroll 1
    for (int x = tid; x < rows * (D / 4); x += kThreads) {
      const int r = x / (D / 4), d = (x % (D / 4)) * 4;
      if (d >= p.c.D) continue;
      float2 ml[kWarps];
      float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        ml[w] = s_ml[w * C::ROWS + r];
        M = max_nan(M, ml[w].x);
      }
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (ml[w].x == -CUDART_INF_F) continue;
        const float f = ex2(ml[w].x - M);
        const float4 u = *reinterpret_cast<const float4 *>(base + w * (C::DEPTH * C::STAGE) + o_at(r, d) * 4);
        L += large ? rescaled(ml[w].y, ex2(0.5f * (ml[w].x - M))) : f * ml[w].y;
        v.x += f * u.x;
        v.y += f * u.y;
        v.z += f * u.z;
        v.w += f * u.w;
      }
      if (nans) {
        const uint32_t bits = s_nan[(r * D + d) / 32] >> (d % 32);
        if (bits & 1u) v.x = CUDART_NAN_F;
        if (bits & 2u) v.y = CUDART_NAN_F;
        if (bits & 4u) v.z = CUDART_NAN_F;
        if (bits & 8u) v.w = CUDART_NAN_F;
      }
      if (whole) {
        const RowEnd e = row_end(p, run.hk * p.G + (r0 + r) % p.G, M, L);
        if (d == 0) p.LSE[lse_at(p, run.b, run.hk, r0 + r)] = e.lse;
        put4(static_cast<T *>(p.O) + o_row(p, run.b, run.hk, r0 + r) + d, make_float4(v.x * e.scale, v.y * e.scale, v.z * e.scale, v.w * e.scale));
      } else if (one_of) {  // into warp 0's place, which this thread alone has read
        if (d == 0) s_cta[r] = make_float2(M, L);
        *reinterpret_cast<float4 *>(base + o_at(r, d) * 4) = v;
      } else {
        if (d == 0) p.ml_part[(size_t)run.slot * C::ROWS + r] = make_float2(M, L);
        *reinterpret_cast<float4 *>(p.o_part + ((size_t)run.slot * C::ROWS + r) * p.c.D + d) = v;
      }
    }
    if (one_of) {
      // The cluster's CTAs share out the item's outputs and add each other's parts up.
      cluster_sync();
#pragma unroll 1
      for (int x = rank * kThreads + tid; x < rows * (D / 4); x += p.cluster * kThreads) {
        const int r = x / (D / 4), d = (x % (D / 4)) * 4;
        if (d >= p.c.D) continue;
        const uint32_t ml_at = smem_u32(s_cta + r), v_at = smem_u32(base + o_at(r, d) * 4);
        float M = -CUDART_INF_F, L = 0.f;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = 0; k < p.cluster; ++k) {
          const float2 ml = dsmem_f2(ml_at, k);
          const float4 u = dsmem_f4(v_at, k);
          const float top = max_nan(M, ml.x);
          if (top == -CUDART_INF_F) continue;
          const float ha = ex2(0.5f * (M - top)), hf = ex2(0.5f * (ml.x - top)), a = ha * ha, f = hf * hf;
          M = top;
          L = rescaled(L, ha) + rescaled(ml.y, hf);
          v.x = v.x * a + f * u.x;
          v.y = v.y * a + f * u.y;
          v.z = v.z * a + f * u.z;
          v.w = v.w * a + f * u.w;
        }
        const RowEnd e = row_end(p, run.hk * p.G + (r0 + r) % p.G, M, L);
        if (d == 0) p.LSE[lse_at(p, run.b, run.hk, r0 + r)] = e.lse;
        if (M == -CUDART_INF_F) v = make_float4(0.f, 0.f, 0.f, 0.f);
        put4(static_cast<T *>(p.O) + o_row(p, run.b, run.hk, r0 + r) + d, make_float4(v.x * e.scale, v.y * e.scale, v.z * e.scale, v.w * e.scale));
      }
      cluster_sync();  // no CTA leaves while another reads its part
    }
    if (p.cluster) return;
    __syncthreads();  // the ring, s_ml and s_nan are free for the next run
    if (nans || large) {
      for (int x = tid; x < C::ROWS * D / 32; x += kThreads) s_nan[x] = 0u;
      if (tid == 0) s_any = s_large = 0;
      __syncthreads();
    }
  } while (cursor_next(p, &s_groups, cur, run));
}

template <typename T, int KIND, int D, int MT>
cudaError_t launch_t(const FwdParams &p, cudaStream_t st) {
  using C = Cfg<T, D, MT>;
  auto kernel = cache_fwd_mma_kernel<T, KIND, D, MT>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = raise_smem(kernel, done, C::SMEM);
  if (e != cudaSuccess) return e;
  CUtensorMap km, vm;
  const int rows = p.c.page < C::SK ? p.c.page : C::SK;
  if (!make_tmap_codes(&km, p.c.k, p.c.D, p.c.page, (long long)p.c.num_pages * p.c.Hkv, C::BLK, rows) ||
      !make_tmap_codes(&vm, p.c.v, p.c.D, p.c.page, (long long)p.c.num_pages * p.c.Hkv, C::BLK, rows))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.cluster ? p.NG * p.c.Hkv * p.cluster : p.max_ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.cluster;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.cluster > 1 ? 1 : 0;
  return counted(cudaLaunchKernelEx(&cfg, kernel, p, km, vm));
}

template <int KIND> cudaError_t launch_kind(const FwdParams &p, int dtype, cudaStream_t st) {
  const int D = mma_columns(p.c.D);
  if (dtype == kF32) {
    switch (D) {
      case 64: return launch_t<float, KIND, 64, 1>(p, st);
      case 128: return launch_t<float, KIND, 128, 1>(p, st);
      default: return launch_t<float, KIND, 256, 1>(p, st);
    }
  }
  const bool two = p.row_tile == 32;
  switch (D) {
    case 64: return two ? launch_t<__nv_bfloat16, KIND, 64, 2>(p, st) : launch_t<__nv_bfloat16, KIND, 64, 1>(p, st);
    case 128: return two ? launch_t<__nv_bfloat16, KIND, 128, 2>(p, st) : launch_t<__nv_bfloat16, KIND, 128, 1>(p, st);
    default: return launch_t<__nv_bfloat16, KIND, 256, 1>(p, st);
  }
}

}  // namespace
}  // namespace cache
}  // namespace attn
