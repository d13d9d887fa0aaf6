// cache_tc.cu -- attention over the 8-bit cache with tcgen05: bf16 queries, head dims up to 128 (compiled for 64
// and 128 columns, those past the head dim filled with zeros), many query rows per kv head (drafts of several
// tokens, chunks of a prompt, many heads to a kv head).
//
// m16n8k16 products end at some 300 TFLOP/s here; with many rows the tensor cores' own path does more (730 TFLOP/s
// for 2048 rows of 16111 keys at D = 128, 410 at D = 64).  One CTA computes one 128-row tile of one (sequence, kv
// head) over one share of its keys, in tiles of 128 keys:
//   warp 0        TMA: the tile's codes of K and V, page by page, and the scales of its 16-key groups into a
//                 small ring;
//   warp 1        MMA issuer: S_j = Q K_j^T into one of two TMEM buffers, O += P_{j-1} V_{j-1} with P in TMEM;
//   warps 2..9    softmax: a row is a TMEM lane, the two warps of a lane quarter split its keys (as in the
//                 dense forward); O is rescaled only when a row's reference grew by more than 2^4;
//   warps 10..13  converters: the queries once, scaled per row by a power of two into fp16, then every tile's
//                 codes widened to fp16 (exactly) into the 128-byte-swizzled operand layout.
// Scales never touch the operands: a key's scale multiplies its scores, a value's enters the exponent of the
// probabilities, as in the kernel for few rows (cache_work.cuh).  What bounds it now, of some
// 3500 clocks a tile: the softmax warps are busy for 2900 of them (the exponentials alone, 128 x 128 at 16 a
// clock, take 1024) and the converters for 2700; the two MMAs take 544 each.  Twice the converter warps, with
// registers moved to the softmax (640 threads), and converters for K and V apart were slower (258 and 270 us
// against 233): shared memory is what they share.  So was a form of 256 rows to a CTA, each of whose two groups of
// warps had 128 rows or every second tile, with scores in one buffer each: 176 us where this took 194 without a
// cap, but 405 against 342 with one, and 47 against 43 at 256 rows.  At 128 columns the softmax warps spill: 128 registers
// are what 448 threads leave, and 152 (e4m3) or 232 bytes a thread (int8) go to local memory.
#include <algorithm>

#include "cache_work.cuh"
#include "tc_common.cuh"

namespace attn {
namespace cache {
namespace {

using namespace attn::tc;

constexpr int kTcThreads = 448;
constexpr int kBM = 128, kBN = 128, kHC = kBN / 2;
// Growth of a row's reference (log2) that P may reach before O is rescaled, and what P is held times (log2): at most
// 2^15 in fp16, and normal down to 2^-25 of the row's largest.  (Rescaling from 2^8 on took the same time.)
constexpr float kLazy = 4.f, kPShift = 11.f;
constexpr float kZeroLog = kMinScaleExp - 1;
constexpr int kFailed = 0x7fffdead;  // a partner's row maximum that says that a wait gave up (no NaN that arithmetic gives)

// Scales of a tile's eight groups of 16 keys.
struct Info {
  float ks[8], lv[8];
  unsigned gone, zero;  // bit g: no page, or values that count as 0
};

template <int D_>
struct TcCfg {
  static constexpr int D = D_;
  static constexpr int TILE = kBN * D * 2;  // a K, V or Q tile in fp16
  static constexpr int CODES = kBN * D;     // a K or V tile as codes
  static constexpr int OFF_Q = 0, OFF_K = TILE, OFF_V = OFF_K + 2 * TILE, OFF_C = OFF_V + 2 * TILE;
  static constexpr int OFF_X = OFF_C + 2 * CODES;               // partner exchange [2 halves][3 slots][128] floats
  static constexpr int OFF_QM = OFF_X + 6 * kBM * 4;            // [128] what undoes a row's scaling
  static constexpr int OFF_NAN = OFF_QM + kBM * 4;              // a bit per output
  static constexpr int OFF_INFO = OFF_NAN + kBM * D / 8;
  static constexpr int OFF_BAR = OFF_INFO + 4 * (int)sizeof(Info);
  static constexpr int NBAR = 26;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  // (At least half an SM: two CTAs with all of its tensor memory each would only wait for one another.)
  static constexpr int SMEM = OFF_MISC + 64 + 1024 > 120 * 1024 ? OFF_MISC + 64 + 1024 : 120 * 1024;
  static constexpr int TM_O = 2 * kBN, TM_COLS = 512;
  static_assert(SMEM <= 227 * 1024 && OFF_BAR % 8 == 0 && OFF_INFO % 8 == 0, "shared memory");
};

// Instruction descriptor: fp16 operands (format 0), fp32 accumulators.
constexpr uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

template <int N>
__device__ __forceinline__ void reg_fence(uint32_t (&r)[N]) {
#pragma unroll
  for (int e = 0; e < N; ++e) asm volatile("" : "+r"(r[e]));
}

// TMEM column of the P pairs that the 16-key slice kk of the PV MMA reads: each half's P lies over the first
// half of its own score columns.
__device__ __forceinline__ constexpr uint32_t p_col(int kk) { return (uint32_t)(kk * 8 + (kk * 16 / kHC) * (kHC / 2)); }

// Barrier of the two softmax warps of lane quarter wq (ids 2..5).
__device__ __forceinline__ void pair_bar(int wq) {
  __syncwarp();
  asm volatile("bar.sync %0, 64;" ::"r"(2 + wq) : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap *m, uint32_t bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Four codes as two fp16 pairs, exactly (see cache_mma.cuh).
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

// Marks the outputs that a chunk's e4m3 NaNs belong to and makes them 0 (see cache_mma.cuh).
template <int D>
__device__ __noinline__ void mark_nans(const FwdParams &p, uint8_t *code, int pos, int d, int len, int r0, int rows, uint32_t *s_nan, int *s_any) {
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

// Chunk `ch` (16 bytes) of row `row` in a 128-row, 128-byte-swizzled block, as the MMA's descriptors have it.
__device__ __forceinline__ uint32_t sw128(int row, int ch) { return row * 128 + ((ch ^ (row & 7)) << 4); }
// The same where TMA put the codes of a tile: rows of D bytes.
template <int D> __device__ __forceinline__ uint32_t code_at(int row, int ch) {
  return D == 128 ? sw128(row, ch) : row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
}

template <int KIND, int D>
__global__ void __launch_bounds__(kTcThreads, 1)
cache_tc_kernel(const __grid_constant__ FwdParams p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
  using C = TcCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  float *xbuf = reinterpret_cast<float *>(smem + C::OFF_X), *s_qm = reinterpret_cast<float *>(smem + C::OFF_QM);
  uint32_t *s_nan = reinterpret_cast<uint32_t *>(smem + C::OFF_NAN);
  Info *info = reinterpret_cast<Info *>(smem + C::OFF_INFO);
  int *misc = reinterpret_cast<int *>(smem + C::OFF_MISC);  // 0: TMEM address, 1: any NaN marked, 2: any large scale

  // This CTA's tile and keys.
  const int item = blockIdx.x / p.splits, sp = blockIdx.x - item * p.splits;
  const int hk = item / p.NG, gr = item - hk * p.NG, b = p.RT == 1 ? gr : gr / p.RT, rt = gr - b * p.RT;
  const int r0 = rt * kBM, rows = min(kBM, p.R - r0);
  const Range range = group_range(p, b, rt);
  const int units = range_units(p, range), each = units / p.splits, extra = units - each * p.splits;
  const int n = each + (sp < extra);
  const int key0 = range.lo + ((sp * each + min(sp, extra)) << p.unit_shift), key1 = min(range.hi, key0 + (n << p.unit_shift));
  const int all_from = row_sees(p, range.len, query_of(p, r0 + rows - 1)).x;  // the keys that every row sees
  const int all_below = min(key1, row_sees(p, range.len, query_of(p, r0)).y);

  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto bar = [&](int i) { return bar0 + 8u * i; };
  const uint32_t q_full = bar(0), o_done = bar(1);
  auto c_full = [&](int kv) { return bar(2 + kv); };     // codes of K (0), V (1) have come
  auto c_empty = [&](int kv) { return bar(4 + kv); };
  auto k_full = [&](int x) { return bar(6 + x); };
  auto k_empty = [&](int x) { return bar(8 + x); };
  auto v_full = [&](int x) { return bar(10 + x); };
  auto v_empty = [&](int x) { return bar(12 + x); };
  auto s_full = [&](int x) { return bar(14 + x); };
  auto p_full = [&](int x) { return bar(16 + x); };
  auto i_full = [&](int x) { return bar(18 + x); };
  auto i_empty = [&](int x) { return bar(22 + x); };
  if (tid == 0) {
    mbar_init(q_full, 128);
    mbar_init(o_done, 1);
    for (int x = 0; x < 2; ++x) {
      mbar_init(c_full(x), 1);
      mbar_init(c_empty(x), 128);
      mbar_init(k_full(x), 128);
      mbar_init(k_empty(x), 1);
      mbar_init(v_full(x), 128);
      mbar_init(v_empty(x), 1);
      mbar_init(s_full(x), 1);
      mbar_init(p_full(x), 256);
    }
    for (int x = 0; x < 4; ++x) {
      mbar_init(i_full(x), 1);
      mbar_init(i_empty(x), 8);
    }
    fence_barrier_init();
    misc[1] = misc[2] = 0;
    if (sp == 0 && hk == 0 && rt == 0) {
      bool bad;
      seq_len(p.c, b, &bad);
      if (bad) set_status(p.c.status, kStatusBadPage);
    }
  }
  for (int x = tid; x < kBM * D / 32; x += kTcThreads) s_nan[x] = 0u;
  if (warp == 1) {
    tmem_alloc(smem_u32(misc), C::TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)misc[0];
  if (tid == 0 && (tmem & 0xFFFFu) + C::TM_COLS > 512) set_status(p.c.status, kStatusBadTmemAlloc);
  float m_ref = -CUDART_INF_F, l = 0.f;  // softmax: this row's reference (log2) and this half's sum
  bool ok = true;

  if (warp == 0) {
    // ------------------------------------------------------------ TMA and scales
    // Lane 8 i + g has group g of tile 4 batch + i; one batch ahead.
    if (lane == 0) {
      tma_prefetch_desc(&kmap);
      tma_prefetch_desc(&vmap);
    }
    const int grp = lane & 7, box = min(p.c.page, 64);
    int id = -1, id_nxt = -1;
    float ks = 0.f, vs = 0.f;
    auto load_id = [&](int batch) {
      const int pos = key0 + (batch * 4 + (lane >> 3)) * kBN + 16 * grp;
      return pos < key1 ? page_of(p.c, b, pos) : -1;
    };
    id_nxt = load_id(0);
    int asked[2] = {0, 0};  // tiles of K, of V
    for (int j = 0; ok && j < n; ++j) {
      const int sub = j & 3;
      if (sub == 0) {
        id = id_nxt;
        ks = vs = 0.f;
        if (id >= 0) {
          const size_t at = (size_t)id * p.c.Hkv + hk;
          ks = p.c.k_scale[at];
          vs = p.c.v_scale[at];
        }
        id_nxt = load_id((j >> 2) + 1);
      }
      const bool mine = (lane >> 3) == sub;
      const int pos = key0 + j * kBN + 16 * grp;
      const bool lead = mine && id >= 0 && (16 * grp) % box == 0;
      const unsigned bytes = __popc(__ballot_sync(~0u, lead)) * box * D;
      for (int kv = 0; kv < 2; ++kv) {
        if (j >= 1 && !mbar_wait_warp(c_empty(kv), (j - 1) & 1, p.c.status)) {
          ok = false;
          break;
        }
        if (lane == 0) mbar_arrive_expect_tx(c_full(kv), bytes);
        ++asked[kv];
        __syncwarp();
        if (lead)
          tma_load_3d(sbase + C::OFF_C + kv * C::CODES + grp * 16 * D, kv ? &vmap : &kmap, c_full(kv), 0, pos & (p.c.page - 1),
                      id * p.c.Hkv + hk);
        if (kv == 0) {  // the scales go out behind the keys' loads
          if (j >= 4 && !mbar_wait_warp(i_empty(sub), ((j >> 2) - 1) & 1, p.c.status)) {
            ok = false;
            break;
          }
          const bool zero = !(vs >= kMinScale);
          const unsigned gone = __ballot_sync(~0u, id < 0) >> (8 * sub), zeros = __ballot_sync(~0u, zero) >> (8 * sub);
          if (mine) {
            info[sub].ks[grp] = ks;
            const float lv = zero ? kZeroLog : log2f(vs);
            info[sub].lv[grp] = lv;
            if (lv > kFarTop) misc[2] = 1;
            if (grp == 0) {
              info[sub].gone = gone & 255u;
              info[sub].zero = zeros & 255u;
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(i_full(sub));
        }
      }
    }
    // A wait gave up: the copies in flight end in this CTA's memory, so they are waited for.
    for (int kv = 0; !ok && kv < 2; ++kv)
      if (asked[kv]) mbar_wait_warp(c_full(kv), (asked[kv] - 1) & 1, p.c.status);
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (n > 0) {
      constexpr uint32_t idS = idesc_f16(kBM, kBN, false), idO = idesc_f16(kBM, D, true);
      const uint64_t dq0 = sw128_desc(sbase + C::OFF_Q, 16, 1024);
      const uint64_t dk0 = sw128_desc(sbase + C::OFF_K, 16, 1024);
      const uint64_t dv0 = sw128_desc(sbase + C::OFF_V, kBN * 128, 1024);
      ok = mbar_wait_warp(q_full, 0, p.c.status);
      for (int j = 0; ok && j <= n; ++j) {
        if (j < n) {
          const int x = j & 1;
          if (!mbar_wait_warp(k_full(x), (j >> 1) & 1, p.c.status)) break;
          tc_fence_after();
          uint64_t qd = dq0, kd = desc_at(dk0, x * C::TILE);
#pragma unroll 1
          for (int c = 0; c < D / 64; ++c) {
#pragma unroll
            for (int k4 = 0; k4 < 4; ++k4) mma_ss_w(tmem + x * kBN, desc_at(qd, k4 * 32), desc_at(kd, k4 * 32), idS, (c | k4) != 0);
            qd = desc_at(qd, kBM * 128);
            kd = desc_at(kd, kBN * 128);
          }
          mma_commit_w(s_full(x));
          mma_commit_w(k_empty(x));
        }
        if (j >= 1) {
          const int jj = j - 1, x = jj & 1;
          if (!mbar_wait_warp(v_full(x), (jj >> 1) & 1, p.c.status)) break;
          if (!mbar_wait_warp(p_full(x), (jj >> 1) & 1, p.c.status)) break;
          tc_fence_after();
          const uint64_t dv = desc_at(dv0, x * C::TILE);
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            mma_ts_w(tmem + C::TM_O, tmem + x * kBN + p_col(kk), desc_at(dv, kk * (16 * 128)), idO, (jj > 0 || kk > 0) ? 1u : 0u);
          mma_commit_w(v_empty(x));
          mma_commit_w(o_done);
        }
      }
    }
  } else if (warp >= 10) {
    // ------------------------------------------------------------ converters
    const int t = tid - 320;
    if (n > 0) {  // query row t
      const int r = r0 + t, i = query_of(p, r), h = hk * p.G + (r - i * p.G);
      uint4 raw[D / 8];
      float amax = 0.f;
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        raw[c] = make_uint4(0, 0, 0, 0);
        if (t < rows && c * 8 < p.c.D)
          raw[c] = *reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) + b * p.q_sb + i * p.q_ss + h * p.q_sh + c * 8);
      }
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) amax = max_nan(amax, fabsf(__uint_as_float(w[e] << 16)), fabsf(__uint_as_float(w[e] & 0xffff0000u)));
      }
      // 2^x that brings the largest element into [2^14, 2^15); 1 for rows that are 0 or not finite.
      int x = 14 - ((int)(__float_as_uint(amax) >> 23) - 127);
      if (!(amax > 0.f) || !(amax <= 3.402823466e38f)) x = 0;
      x = x > 126 ? 126 : x;
      const float up = copysignf(__uint_as_float((unsigned)(x + 127) << 23), p.scale);
      s_qm[t] = __uint_as_float((unsigned)(127 - x) << 23) * fabsf(p.scale) * (p.cap > 0.f ? 2.f * kLog2e * p.inv_cap : kLog2e);
#pragma unroll
      for (int c = 0; c < D / 8; ++c) {
        uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack_h2(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xffff0000u) * up);
        *reinterpret_cast<uint4 *>(smem + C::OFF_Q + (c / 8) * (kBM * 128) + sw128(t, c % 8)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
      fence_async_smem();
      mbar_arrive(q_full);
    }
    for (int j = 0; ok && j < n; ++j) {
      const int x = j & 1, pos = key0 + j * kBN;
#pragma unroll 1
      for (int kv = 0; kv < 2; ++kv) {
        ok = mbar_wait_warp(c_full(kv), j & 1, p.c.status);
        if (ok && j >= 2) ok = mbar_wait_warp(kv ? v_empty(x) : k_empty(x), ((j >> 1) - 1) & 1, p.c.status);
        if (!ok) break;
        uint8_t *codes = smem + C::OFF_C + kv * C::CODES, *to = smem + (kv ? C::OFF_V : C::OFF_K) + x * C::TILE;
        unsigned hide = 0;
        bool partial = false;
        if (kv) {
          ok = mbar_wait_warp(i_full(j & 3), (j >> 2) & 1, p.c.status);
          if (!ok) break;
          hide = info[j & 3].gone | info[j & 3].zero;
          partial = hide || pos + kBN > all_below || pos < all_from;
        }
        constexpr int kPer = D / 16;  // chunks of 16 codes per row, and per thread
        const int c = t % kPer, row0 = t / kPer, step = 128 / kPer;
        uint4 u[kPer];
#pragma unroll
        for (int y = 0; y < kPer; ++y) u[y] = *reinterpret_cast<const uint4 *>(codes + code_at<D>(row0 + y * step, c));
        if (partial) {  // values only: a NaN is marked and becomes 0, and so does what no row sees
          auto hidden = [&](int row) { return pos + row >= key1 || ((hide >> (row >> 4)) & 1u); };
          if (KIND == ATTN_CACHE_E4M3) {
            unsigned any = 0;
#pragma unroll
            for (int y = 0; y < kPer; ++y)  // (a byte of 0x7f, and no other, carries into its top bit)
              any |= hidden(row0 + y * step) ? 0u
                                             : ((u[y].x & 0x7f7f7f7fu) + 0x01010101u) | ((u[y].y & 0x7f7f7f7fu) + 0x01010101u) |
                                                   ((u[y].z & 0x7f7f7f7fu) + 0x01010101u) | ((u[y].w & 0x7f7f7f7fu) + 0x01010101u);
            if (any & 0x80808080u) {
#pragma unroll 1
              for (int y = 0; y < kPer; ++y) {
                const int row = row0 + y * step;
                if (!hidden(row)) mark_nans<D>(p, codes + code_at<D>(row, c), pos + row, c * 16, range.len, r0, rows, s_nan, misc + 1);
              }
#pragma unroll
              for (int y = 0; y < kPer; ++y) u[y] = *reinterpret_cast<const uint4 *>(codes + code_at<D>(row0 + y * step, c));
            }
          }
#pragma unroll
          for (int y = 0; y < kPer; ++y)
            if (hidden(row0 + y * step)) u[y] = make_uint4(0, 0, 0, 0);
          fence_async_smem();  // (codes that mark_nans wrote, before the next load)
        }
        // The codes' place is given away only once they have come: a load may be held up longer than the arrival
        // and the next tile's copy take (by stores of scores in the same unit), and nothing orders it before a copy
        // by TMA.  So the barrier's address hangs on a word of each load (p.cluster is 0 here).
        uint32_t come = 0;
#pragma unroll
        for (int y = 0; y < kPer; ++y) come |= u[y].x;
        mbar_arrive(c_empty(kv) + (come & (uint32_t)p.cluster));
        // Chunks 2 (c % 4) and the next of block c / 4; the lanes of the second block store them the other way
        // round, so that eight lanes meet all banks.
        uint8_t *const blk = to + (c / 4) * (kBN * 128);
        const bool swap = (c & 4) != 0;
#pragma unroll
        for (int y = 0; y < kPer; ++y) {
          const uint32_t w0 = swap ? u[y].z : u[y].x, w1 = swap ? u[y].w : u[y].y, w2 = swap ? u[y].x : u[y].z, w3 = swap ? u[y].y : u[y].w;
          uint4 a, d;
          widen4<KIND>(w0, a.x, a.y);
          widen4<KIND>(w1, a.z, a.w);
          widen4<KIND>(w2, d.x, d.y);
          widen4<KIND>(w3, d.z, d.w);
          const int row = row0 + y * step, ch = 2 * (c % 4) + (swap ? 1 : 0);
          *reinterpret_cast<uint4 *>(blk + sw128(row, ch)) = a;
          *reinterpret_cast<uint4 *>(blk + sw128(row, ch ^ 1)) = d;
        }
        fence_async_smem();  // for the MMA
        mbar_arrive(kv ? v_full(x) : k_full(x));
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int wq = warp & 3, half = (warp - 2) >> 2, r = wq * 32 + lane;
    const bool active = wq * 32 < rows;  // warp-uniform
    const uint32_t lane_addr = tmem + ((uint32_t)(wq * 32) << 16);
    const int2 see = row_sees(p, range.len, query_of(p, r0 + min(r, rows - 1)));
    const int see_n = max(0, min(see.y, key1) - see.x);
    const float cap_log2 = p.cap * kLog2e;
    float q_mul = 0.f;
    if (n > 0) {
      ok = mbar_wait_warp(q_full, 0, p.c.status);
      q_mul = s_qm[r];
    }
    for (int j = 0; j < n; ++j) {
      const int pos = key0 + j * kBN, j0 = pos + half * kHC;
      bool got = mbar_wait_warp(i_full(j & 3), (j >> 2) & 1, p.c.status);
      float f[4], lv[4];
      unsigned gone = 0, odd = 0;
      if (got) {
        const Info &in = info[j & 3];
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          f[g] = q_mul * in.ks[half * 4 + g];
          lv[g] = in.lv[half * 4 + g];
        }
        gone = in.gone >> (half * 4);
        odd = in.gone | in.zero;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(i_empty(j & 3));
      got = got && mbar_wait_warp(s_full(j & 1), (j >> 1) & 1, p.c.status);
      tc_fence_after();
      if (!active) {  // rows that are not there: their lanes of P may hold anything
        if (!got) {
          ok = false;
          break;
        }
        tc_fence_before();
        mbar_arrive(p_full(j & 1));
        continue;
      }
      const uint32_t sa = lane_addr + (uint32_t)((j & 1) * kBN + half * kHC);
      uint32_t xr[kHC];
      float mx = -CUDART_INF_F;
      if (got) {
#pragma unroll
        for (int c = 0; c < kHC / 32; ++c) tmem_ld32(sa + c * 32, *reinterpret_cast<uint32_t(*)[32]>(xr + c * 32));
        tmem_wait_ld();
        reg_fence(xr);
        const bool partial = odd || pos + kBN > all_below || pos < all_from;
        if (partial || p.cap > 0.f) {  // form the logits; f is 1 from here on
#pragma unroll
          for (int e = 0; e < kHC; ++e) {
            float v = __uint_as_float(xr[e]) * f[e / 16];
            if (p.cap > 0.f) v = cap_log2 - __fdividef(2.f * cap_log2, 1.f + ex2_approx(v));
            if (partial && (((gone >> (e / 16)) & 1u) || (unsigned)(j0 + e - see.x) >= (unsigned)see_n)) v = -CUDART_INF_F;
            xr[e] = __float_as_uint(v);
          }
#pragma unroll
          for (int g = 0; g < 4; ++g) f[g] = 1.f;
        }
        if (p.scores && r < rows) {
          float *row = scores_row(p, b, hk, r0 + r) + j0;
#pragma unroll
          for (int e = 0; e < kHC; e += 4)
            if (j0 + e < p.Lpad)
              *reinterpret_cast<float4 *>(row + e) =
                  make_float4(f[e / 16] * __uint_as_float(xr[e]), f[e / 16] * __uint_as_float(xr[e + 1]),
                              f[e / 16] * __uint_as_float(xr[e + 2]), f[e / 16] * __uint_as_float(xr[e + 3]));
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float m = __uint_as_float(xr[16 * g]);
#pragma unroll
          for (int e = 1; e < 15; e += 2) m = max_nan(m, __uint_as_float(xr[16 * g + e]), __uint_as_float(xr[16 * g + e + 1]));
          m = max_nan(m, __uint_as_float(xr[16 * g + 15]));
          mx = max_nan(mx, fmaf(f[g], m, lv[g]));
        }
      }
      // The row's maximum over both halves; slot j & 1 is rewritten two tiles later, after the partner has
      // passed the next barrier.
      xbuf[(half * 3 + (j & 1)) * kBM + r] = got && ok ? mx : __int_as_float(kFailed);
      pair_bar(wq);
      const float other = xbuf[((1 - half) * 3 + (j & 1)) * kBM + r];
      if (!(got && ok) || __float_as_int(other) == kFailed) {
        ok = false;
        break;
      }
      const float m_new = max_nan(m_ref, max_nan(mx, other));
      float alpha = 1.f;
      if (m_ref == -CUDART_INF_F) {
        m_ref = m_new;  // O is all zeros, or not written yet
      } else if (m_new > m_ref + kLazy) {
        alpha = ex2_approx(m_ref - m_new);
        l *= alpha;
        m_ref = m_new;
      }
      const float mr = m_ref == -CUDART_INF_F ? 0.f : m_ref;
#pragma unroll
      for (int q = 0; q < 2; ++q) {  // (16 registers of P at a time)
        uint32_t pk[16];
#pragma unroll
        for (int g = 2 * q; g < 2 * q + 2; ++g) {
          const uint64_t f2 = f2_splat(f[g]), ref2 = f2_splat(lv[g] - mr + kPShift);
          uint64_t sum = 0;  // (two floats)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float p0, p1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(xr[16 * g + 2 * e]), __uint_as_float(xr[16 * g + 2 * e + 1])), f2, ref2), p0, p1);
            p0 = ex2_approx(p0);
            p1 = ex2_approx(p1);
            sum = f2_add(sum, f2_pack(p0, p1));
            pk[8 * (g - 2 * q) + e] = pack_h2(p0, p1);
          }
          float s0, s1;
          f2_unpack(sum, s0, s1);
          l = fmaf(s0 + s1, ex2_approx(-lv[g]), l);
        }
        __syncwarp();
        tmem_st16(sa + 16 * q, pk);
      }
      if (j >= 1) ok = mbar_wait_warp(o_done, (j - 1) & 1, p.c.status);
      if (j >= 1 && __any_sync(~0u, alpha != 1.f)) {
        tc_fence_after();
#pragma unroll 1
        for (int c = half * (D / 64); c < (half + 1) * (D / 64); ++c) {
          uint32_t o[32];
          tmem_ld32(lane_addr + C::TM_O + c * 32, o);
          tmem_wait_ld();
          reg_fence(o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          tmem_st32(lane_addr + C::TM_O + c * 32, o);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(p_full(j & 1));
      // (A wait on o_done that gave up reaches the partner in the next exchange.)
    }
    if (active && ok && n > 0) ok = mbar_wait_warp(o_done, (n - 1) & 1, p.c.status);
    tc_fence_after();
    // A scale so large that others may be too far below it (the records of all tiles were waited for): see
    // cache_work.cuh.  Each half counts 16 of the quarter's rows, and nothing for the others.
    const Keys keys = {key0, 512, 512, key1};
    if (active && n > 0 && misc[2] && __all_sync(~0u, ok) && far_apart(p, b, hk, keys)) {
      l = 0.f;
#pragma unroll 1
      for (int z = half * 16; z < half * 16 + 16 && wq * 32 + z < rows; ++z) {
        const float M = __shfl_sync(~0u, m_ref, z);
        const float sum = recount<__nv_bfloat16, KIND>(p, b, hk, r0 + wq * 32 + z, range.len, keys, M - kPShift);
        if (lane == z) l = sum;
      }
    }
    xbuf[(half * 3 + 2) * kBM + r] = ok ? l : CUDART_NAN_F;
  }

  __syncwarp();
  tc_fence_before();
  __syncthreads();  // the last marks of NaNs, and the halves' sums
  tc_fence_after();
  grid_launch_next();
  if (warp >= 2 && warp < 10) {
    const int wq = warp & 3, half = (warp - 2) >> 2, r = wq * 32 + lane;
    const float M = m_ref - kPShift;  // what O and the sum are relative to
    if (wq * 32 < rows) {
      const float L = xbuf[2 * kBM + r] + xbuf[5 * kBM + r];
      const uint32_t lane_addr = tmem + ((uint32_t)(wq * 32) << 16);
      const bool row_ok = r < rows, nans = misc[1] != 0, whole = p.splits == 1;
      const RowEnd e = row_end(p, hk * p.G + (r0 + min(r, rows - 1)) % p.G, M, L);
      const size_t part = (size_t)blockIdx.x * kBM + r;
      if (row_ok && half == 0) {
        if (whole) p.LSE[lse_at(p, b, hk, r0 + r)] = e.lse;
        else p.ml_part[part] = make_float2(M, L);
      }
      const bool none = n == 0 || M == -CUDART_INF_F;
#pragma unroll 1
      for (int c = half * (D / 64); c < (half + 1) * (D / 64); ++c) {
        uint32_t o[32];
        if (n > 0) {
          tmem_ld32(lane_addr + C::TM_O + c * 32, o);
          tmem_wait_ld();
          reg_fence(o);
        }
        const uint32_t bits = nans && row_ok ? s_nan[(r * D + c * 32) / 32] : 0u;
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          float v = none ? 0.f : __uint_as_float(o[x]);
          if ((bits >> x) & 1u) v = CUDART_NAN_F;
          o[x] = __float_as_uint(whole ? v * e.scale : v);
        }
        if (row_ok && whole) {
          uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.O) + o_row(p, b, hk, r0 + r) + c * 32);
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (c * 32 + 8 * x < p.c.D)
              dst[x] = make_uint4(pack_bf16(__uint_as_float(o[8 * x]), __uint_as_float(o[8 * x + 1])),
                                  pack_bf16(__uint_as_float(o[8 * x + 2]), __uint_as_float(o[8 * x + 3])),
                                  pack_bf16(__uint_as_float(o[8 * x + 4]), __uint_as_float(o[8 * x + 5])),
                                  pack_bf16(__uint_as_float(o[8 * x + 6]), __uint_as_float(o[8 * x + 7])));
        } else if (row_ok) {
          uint4 *dst = reinterpret_cast<uint4 *>(p.o_part + part * p.c.D + c * 32);
#pragma unroll
          for (int x = 0; x < 8; ++x)
            if (c * 32 + 4 * x < p.c.D) dst[x] = make_uint4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        }
        __syncwarp();  // together into the next load from TMEM
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TM_COLS);
  }
}

template <int KIND, int D> cudaError_t launch_t(const FwdParams &p, cudaStream_t st) {
  using C = TcCfg<D>;
  auto kernel = cache_tc_kernel<KIND, D>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = raise_smem(kernel, done, C::SMEM);
  if (e != cudaSuccess) return e;
  CUtensorMap km, vm;
  const int rows = std::min(p.c.page, 64);
  if (!make_tmap_codes(&km, p.c.k, p.c.D, p.c.page, (long long)p.c.num_pages * p.c.Hkv, D, rows) ||
      !make_tmap_codes(&vm, p.c.v, p.c.D, p.c.page, (long long)p.c.num_pages * p.c.Hkv, D, rows))
    return cudaErrorInvalidValue;
  kernel<<<(unsigned)(p.NG * p.c.Hkv * p.splits), kTcThreads, C::SMEM, st>>>(p, km, vm);
  return counted(cudaGetLastError());
}

}  // namespace

int tc_row_tile() { return kBM; }
int tc_unit_shift() { return 7; }

// When this kernel is taken instead of that of cache_mma.cuh.  Both measured (us, that one / this one; 4 query heads to each of
// 8 kv heads; ragged rows up to the keys given).
// D = 128, from 65 rows per kv head: 16 sequences of 8192 keys, 48 rows 106 / 90, 64 111 / 91 (with a cap 120 / 137), 96
// 159 / 97; 4 of 3000, 64 rows 22 / 29, 96 33 / 33; one of 16111, 64 rows 29 / 23 (cap 31 / 32), 96 39 / 24; one of 3000, 96
// 17 / 18.
// D = 64, where a tile's MMAs are half and its softmax is not: a batch from 65 rows on if the other kernel's tiles of
// 32 rows do not fit one wave of two CTAs per SM (8 kv heads x 16 sequences x 3 tiles do not), else from 513 on.  16 of
// 8192, 64 rows 65 / 79, 96 97 / 82, 128 125 / 86 (cap 145 / 135), 512 447 / 228; 16 of 1000, 64 17 / 27, 96 47 / 30; 64 of 1000,
// 96 126 / 54; 4 of 3000, 128 22 / 32, 256 37 / 52, 384 58 / 71, 512 71 / 56; 4 of 8192, 256 66 / 69, 512 128 / 84.  A single
// sequence from 257 rows on: 16111 keys, 128 rows 26 / 21 (cap 31 / 29), 256 48 / 32, 512 74 / 50; 3000, 128 13 / 16, 256 16 / 19, 384
// 23 / 22, 512 23 / 20.
// A head dim in between takes the time of the next larger one on either.
bool tc_supported_rows(int dtype, int D, int R, int B, int Hkv) {
  if (dtype != kBF16 || D > 128 || R <= 64) return false;
  if (D > 64) return true;
  return R > (B > 1 ? 512 : 256) || (B > 1 && (long long)B * Hkv * ((R + 31) / 32) > 2LL * device_sm_count());
}

// Shares of an item's keys, one CTA each, one CTA per SM, of at least four tiles.  One sequence: as many as end first,
// by a count of tiles (kStart: a CTA's start and end).  A batch, whose lengths the host does not know: enough for
// three waves, so that the block scheduler evens ragged rows out.  One row of 16111 keys (us, by the count / by three
// waves): 2048 rows 186 / 228, 256 41 / 72, 96 29 / 39.
int tc_splits(const FwdParams &p) {
  constexpr long long kStart = 6;
  const long long items = (long long)p.NG * p.c.Hkv, sms = device_sm_count();
  long long keys = (long long)p.c.max_pages << p.c.page_shift;
  if (p.window > 0) keys = std::min(keys, (long long)p.window + p.Sq);
  const long long tiles = std::max(1LL, (keys + kBN - 1) / kBN), most = (tiles + 3) / 4;
  if (p.c.B > 1) return (int)std::min(most, (3 * sms + items - 1) / items);
  long long best = 0, at = 1;
  for (long long s = 1; s <= most && (s == 1 || items * (s - 1) < 4 * sms); ++s) {
    const long long t = (items * s + sms - 1) / sms * ((tiles + s - 1) / s + kStart);
    if (s == 1 || t < best) {
      best = t;
      at = s;
    }
  }
  return (int)at;
}

cudaError_t launch_fwd_tc(const FwdParams &p, int kind, cudaStream_t st) {
  if (p.c.D <= 64) return kind == ATTN_CACHE_E4M3 ? launch_t<ATTN_CACHE_E4M3, 64>(p, st) : launch_t<ATTN_CACHE_INT8, 64>(p, st);
  return kind == ATTN_CACHE_E4M3 ? launch_t<ATTN_CACHE_E4M3, 128>(p, st) : launch_t<ATTN_CACHE_INT8, 128>(p, st);
}

}  // namespace cache
}  // namespace attn
