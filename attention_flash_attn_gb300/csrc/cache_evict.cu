// cache_evict.cu -- eviction by accumulated attention weight: which tokens stay, and their move
// to fresh pages.  Measured: the selection takes 16 us for 128 rows of up to 8192 weights and 33 us for 16 rows of
// up to 131072; the move 24 us for 128 x 2048 tokens and 27 us for 16 x 16384, D = 128 (134 MB, 5.6 and 5.0 TB/s).
#include <cooperative_groups.h>

#include "cache_common.cuh"

namespace attn {
namespace cache {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThr = 512, kSelWarps = kSelThr / 32;
constexpr int kBins = 2048, kGroup = kBins / 32;  // counts of a digit; each lane of a warp has a group of them
static_assert(kBins / kSelThr == 4 && kGroup == 64, "a group's counts are summed by 16 threads, four each");
constexpr int kMoveThr = 256;
constexpr int kSelSmemKeys = 49152;  // most weights that one CTA holds in shared memory (192 KB)

// Weights in an order of unsigned integers: larger weight, larger integer; -0 as +0, NaN largest.
__device__ __forceinline__ unsigned order_of(float w) {
  if (w != w) return 0xffffffffu;
  const unsigned u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ int warp_prefix(int x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, x, o);
    if (lane >= o) x += v;
  }
  return x;
}

// One cluster per (sequence, kv head); each of its CTAs has a contiguous part of the middle positions
// [first, n - recent), whose weights it reads once and keeps in shared memory
// (parts that do not fit are read again in every pass).  The K-th largest order T is found in three
// digits of 11, 11 and 10 bits: each CTA counts the next digit of its weights that share those found, and the
// cluster's counts are added up through distributed shared memory.  Then every position above T stays, and
// of those equal to T the lowest ones: each warp has a contiguous part, placed by prefix sums over the
// warps' and the CTAs' counts, so that the result is ascending.  Bound by latency: four cluster barriers and
// passes over shared memory.  Clusters of 16 instead of 8 took half as long again.
__global__ void __launch_bounds__(kSelThr) cache_select_kernel(const __grid_constant__ EvictParams p, int in_smem) {
  extern __shared__ __align__(16) float s_w[];
  __shared__ __align__(16) unsigned s_hist[2][kBins];  // (read in fours)
  __shared__ unsigned s_group[2][32];
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps], s_all[2], s_found[2];
  const cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), ranks = cluster.num_blocks();
  const int pair = blockIdx.x / ranks, b = pair / p.c.Hkv, h = pair - b * p.c.Hkv;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5, all_t = rank * kSelThr + t, step = ranks * kSelThr;
  bool bad;
  const int len = seq_len(p.c, b, &bad), n = min(len, p.keep);
  if (all_t == 0 && h == 0) {
    p.lengths_out[b] = n;
    if (bad) set_status(p.c.status, kStatusBadPage);
  }
  int *kept = p.kept + (size_t)pair * p.keep;
  float *w_out = p.weights_out + b * p.wo_sb + h * p.wo_sh;
  const float *w = p.weights + b * p.w_sb + h * p.w_sh;
  for (int i = n + all_t; i < p.keep; i += step) {
    kept[i] = -1;
    w_out[i] = 0.f;
  }
  if (len <= p.keep) {
    for (int i = all_t; i < n; i += step) {
      kept[i] = i;
      w_out[i] = w[i];
    }
    return;
  }
  const int lo = p.first, hi = len - p.recent, K = p.keep - p.first - p.recent;  // lo <= hi as len > keep
  for (int i = all_t; i < p.first; i += step) {
    kept[i] = i;
    w_out[i] = w[i];
  }
  for (int i = all_t; i < p.recent; i += step) {
    kept[p.keep - p.recent + i] = hi + i;
    w_out[p.keep - p.recent + i] = w[hi + i];
  }
  if (K == 0) return;
  const int part = (hi - lo + ranks - 1) / ranks;
  const int a0 = min(hi, lo + rank * part), cnt = min(hi, a0 + part) - a0;
  const float *wp = w + a0;
  if (in_smem) {
    // (Sixteen loads ahead of their stores: the compiler would not move them across.)
    for (int i0 = t; i0 < cnt; i0 += 16 * kSelThr) {
      float v[16];
#pragma unroll
      for (int x = 0; x < 16; ++x) v[x] = i0 + x * kSelThr < cnt ? wp[i0 + x * kSelThr] : 0.f;
#pragma unroll
      for (int x = 0; x < 16; ++x)
        if (i0 + x * kSelThr < cnt) s_w[i0 + x * kSelThr] = v[x];
    }
  }
  for (int i = t; i < kBins; i += kSelThr) s_hist[0][i] = 0;
  __syncthreads();
  auto weight = [&](int i) { return in_smem ? s_w[i] : wp[i]; };
  auto key = [&](int i) { return order_of(weight(i)); };
  unsigned prefix = 0;
  int want = K;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
    unsigned *hist = s_hist[pass & 1];
#pragma unroll 4
    for (int i = t; i < cnt; i += kSelThr) {
      const unsigned u = key(i);
      if (pass == 0 || (u >> (shift + bits)) == prefix) atomicAdd(&hist[(u >> shift) & ((1u << bits) - 1)], 1u);
    }
    __syncthreads();
    {
      const uint4 c = reinterpret_cast<const uint4 *>(hist)[t];
      unsigned sum = (c.x + c.y) + (c.z + c.w);
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) sum += __shfl_xor_sync(~0u, sum, o);
      if ((lane & 15) == 0) s_group[pass & 1][t >> 4] = sum;
    }
    cluster.sync();
    // The other buffer's counts were read, by every CTA, before that barrier.
    reinterpret_cast<uint4 *>(s_hist[(pass + 1) & 1])[t] = make_uint4(0, 0, 0, 0);
    if (warp == 0) {
      // The cluster's counts from the top: of the 32 groups, then of the 64 digits of the group where the sum
      // reaches `want`, two to a lane.  (All of a cluster's counts would be 64 KB through distributed shared memory.)
      int sum = 0;
      for (int r = 0; r < ranks; ++r) sum += (int)cluster.map_shared_rank(s_group[pass & 1], r)[31 - lane];
      int incl = warp_prefix(sum, lane);
      const int at = __ffs(__ballot_sync(~0u, incl >= want)) - 1, group = 31 - at;
      const int left = want - __shfl_sync(~0u, incl - sum, at);
      const int digit = group * kGroup + kGroup - 1 - 2 * lane;
      int c0 = 0, c1 = 0;
      for (int r = 0; r < ranks; ++r) {
        const unsigned *x = cluster.map_shared_rank(hist, r);
        c0 += (int)x[digit];
        c1 += (int)x[digit - 1];
      }
      incl = warp_prefix(c0 + c1, lane);
      const int before = incl - c0 - c1;
      if (before < left && left <= incl) {  // one lane
        const bool second = left > before + c0;
        s_found[0] = digit - (second ? 1 : 0);
        s_found[1] = left - before - (second ? c0 : 0);
      }
    }
    __syncthreads();
    prefix = (prefix << bits) | (unsigned)s_found[0];
    want = s_found[1];
  }
  const unsigned T = prefix;
  const int ties = want;  // positions equal to T that stay
  const int wpart = ((cnt + kSelWarps - 1) / kSelWarps + 127) & ~127;
  const int a = min(cnt, warp * wpart), z = min(cnt, a + wpart);
  // Four neighbouring positions per lane; those past the end count as nothing.
  auto four = [&](int i, float *v, unsigned *g, unsigned *e) {
    *g = *e = 0;
    if (in_smem && i + 4 <= z) {
      const float4 q = *reinterpret_cast<const float4 *>(s_w + i);
      v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x) v[x] = i + x < z ? weight(i + x) : 0.f;
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const unsigned u = order_of(v[x]);
      *g |= (u > T && i + x < z ? 1u : 0u) << x;
      *e |= (u == T && i + x < z ? 1u : 0u) << x;
    }
  };
  int gt = 0, eq = 0;
#pragma unroll 1
  for (int i = a + 4 * lane; i < z; i += 128) {
    float v[4];
    unsigned g, e;
    four(i, v, &g, &e);
    gt += __popc(g);
    eq += __popc(e);
  }
  gt = __reduce_add_sync(~0u, gt);
  eq = __reduce_add_sync(~0u, eq);
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  int g0 = 0, e0 = 0, gall = 0, eall = 0;  // above T, equal to T: in the warps before, and in this CTA
#pragma unroll
  for (int x = 0; x < kSelWarps; ++x) {
    if (x == warp) {
      g0 = gall;
      e0 = eall;
    }
    gall += s_gt[x];
    eall += s_eq[x];
  }
  if (t == 0) {
    s_all[0] = gall;
    s_all[1] = eall;
  }
  cluster.sync();
  for (int r = 0; r < rank; ++r) {
    const int *x = cluster.map_shared_rank(s_all, r);
    g0 += x[0];
    e0 += x[1];
  }
#pragma unroll 1
  for (int i0 = a; i0 < z; i0 += 128) {
    const int i = i0 + 4 * lane;
    float v[4];
    unsigned gm, em;
    four(i, v, &gm, &em);
    if (!__any_sync(~0u, gm | em)) continue;
    // Both counts of the lanes before, in one prefix sum (at most 128 each).
    const int both = __popc(gm) | (__popc(em) << 16), incl = warp_prefix(both, lane);
    int g = g0 + ((incl - both) & 0xffff), e = e0 + ((incl - both) >> 16);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const bool is_g = (gm >> x) & 1u, is_e = (em >> x) & 1u;
      if (is_g || (is_e && e < ties)) {
        const int at = p.first + g + min(e, ties);
        kept[at] = a0 + i + x;
        w_out[at] = v[x];
      }
      g += is_g;
      e += is_e;
    }
    const int all = __shfl_sync(~0u, incl, 31);
    g0 += all & 0xffff;
    e0 += all >> 16;
  }
  cluster.sync();  // no CTA leaves while another reads its counts
}

// Four codes as two fp16 pairs, exactly, and back: codes * ratio rounded to the nearest code, for a
// ratio that is a power of two in [2^-24, 2^15] (or 0) and results that do not exceed the largest code.
template <int KIND> __device__ __forceinline__ void widen4(unsigned w, __half2 &lo, __half2 &hi) {
  unsigned a, b;
  if (KIND == ATTN_CACHE_E4M3) {
    asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\tcvt.rn.f16x2.e4m3x2 %1, y;\n\t}" : "=r"(a), "=r"(b) : "r"(w));
    lo = *reinterpret_cast<__half2 *>(&a);
    hi = *reinterpret_cast<__half2 *>(&b);
  } else {  // code + 128 under the bits of 1024, less 1152
    const unsigned u = w ^ 0x80808080u;
    const __half2 bias = __half2half2(__ushort_as_half(0x6480));
    a = __byte_perm(u, 0x64646464u, 0x4140);
    b = __byte_perm(u, 0x64646464u, 0x4342);
    lo = __hsub2(*reinterpret_cast<__half2 *>(&a), bias);
    hi = __hsub2(*reinterpret_cast<__half2 *>(&b), bias);
  }
}
template <int KIND> __device__ __forceinline__ unsigned narrow4(__half2 lo, __half2 hi, __half2 ratio) {
  if (KIND == ATTN_CACHE_E4M3) {
    // Exact products where it matters: below 2^-10 the code is 0, and four bits from there down are fp16's.
    lo = __hmul2(lo, ratio);
    hi = __hmul2(hi, ratio);
    unsigned r;
    asm("{\n\t.reg .b16 x, y;\n\tcvt.rn.satfinite.e4m3x2.f16x2 x, %1;\n\tcvt.rn.satfinite.e4m3x2.f16x2 y, %2;\n\tmov.b32 %0, {x, y};\n\t}"
        : "=r"(r) : "r"(*reinterpret_cast<unsigned *>(&lo)), "r"(*reinterpret_cast<unsigned *>(&hi)));
    return r;
  }
  // One rounding, to an integer: 1.5 * 2^10 has a step of 1, and the low byte is the code.
  const __half2 magic = __half2half2(__ushort_as_half(0x6600));
  lo = __hfma2(lo, ratio, magic);
  hi = __hfma2(hi, ratio, magic);
  return __byte_perm(*reinterpret_cast<unsigned *>(&lo), *reinterpret_cast<unsigned *>(&hi), 0x6420);
}

// One block per (page of table_out, sequence, kv head): the K and V rows that go there, read once and held
// in registers (NP pieces of 16 codes per thread, for each), their largest magnitudes, their new scales, and
// their new codes.  The chain position -> page -> scales is walked once per row, into shared memory.  The
// work per code is kept in fp16 pairs (exact) where the scales are powers of two, as this library's are: in
// float it had taken longer than the memory.
template <int KIND, int NP>
__global__ void __launch_bounds__(kMoveThr) cache_move_kernel(const __grid_constant__ EvictParams p) {
  __shared__ float s_m[2][kMoveThr / 32], s_scale[2][128];
  __shared__ long long s_row[128];  // first code of each row, or -1
  grid_wait();
  const View &c = p.c;
  const int b = blockIdx.x / p.out_pages, nth = blockIdx.x - b * p.out_pages, h = blockIdx.y, t = threadIdx.x;
  const int i0 = nth << c.page_shift;
  const int out = p.table_out[b * p.table_out_stride + nth];
  const int pos = t < c.page && i0 + t < p.keep ? p.kept[((size_t)b * c.Hkv + h) * p.keep + i0 + t] : -1;
  const int rows = min(c.page, min(seq_len(c, b), p.keep) - i0);
  if (rows <= 0) return;
  if ((unsigned)out >= (unsigned)c.num_pages) {
    if (t == 0) set_status(c.status, kStatusBadPage);
    return;
  }
  if (t < rows) {
    const int page = page_of(c, b, pos);
    const size_t at = (size_t)max(page, 0) * c.Hkv + h;
    s_row[t] = page < 0 ? -1 : (long long)row_at(c, page, h, pos & (c.page - 1));
    s_scale[0][t] = page < 0 ? 0.f : c.k_scale[at];
    s_scale[1][t] = page < 0 ? 0.f : c.v_scale[at];
  }
  __syncthreads();
  const int per = c.D / 16, total = rows * per;
  uint4 w[2][NP];
  int row[NP];
#pragma unroll
  for (int x = 0; x < NP; ++x) {
    const int i = t + x * kMoveThr;
    w[0][x] = w[1][x] = make_uint4(0, 0, 0, 0);
    row[x] = i / per;
    if (i < total) {
      const long long at = s_row[row[x]];
      if (at >= 0) {
        const int d = (i - row[x] * per) * 16;
        w[0][x] = *reinterpret_cast<const uint4 *>(c.k + at + d);
        w[1][x] = *reinterpret_cast<const uint4 *>(c.v + at + d);
      }
    }
  }
  float amax[2] = {0.f, 0.f};
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int x = 0; x < NP; ++x) {
      if (t + x * kMoveThr >= total) continue;
      const unsigned u[4] = {w[kv][x].x, w[kv][x].y, w[kv][x].z, w[kv][x].w};
      __half2 m = __half2half2(__ushort_as_half(0));
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        __half2 lo, hi;
        widen4<KIND>(u[y], lo, hi);
        m = __hmax2(m, __hmax2(__habs2(lo), __habs2(hi)));  // (takes the other one where one is NaN)
      }
      amax[kv] = fmaxf(amax[kv], fmaxf(__low2float(m), __high2float(m)) * s_scale[kv][row[x]]);
    }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
    for (int o = 16; o; o >>= 1) amax[kv] = fmaxf(amax[kv], __shfl_xor_sync(~0u, amax[kv], o));
    if ((t & 31) == 0) s_m[kv][t >> 5] = amax[kv];
  }
  __syncthreads();
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
    for (int x = 0; x < kMoveThr / 32; ++x) amax[kv] = fmaxf(amax[kv], s_m[kv][x]);
    const float s = need_scale<KIND>(fminf(amax[kv], 3.402823466e38f)), inv = pow2_inverse(s);
    uint4 *dst = reinterpret_cast<uint4 *>((kv ? c.v : c.k) + row_at(c, out, h, 0));
#pragma unroll
    for (int x = 0; x < NP; ++x) {
      const int i = t + x * kMoveThr;
      if (i >= total) continue;
      const float f = s_scale[kv][row[x]], ratio = f * inv;
      unsigned u[4] = {w[kv][x].x, w[kv][x].y, w[kv][x].z, w[kv][x].w};
      if ((__float_as_uint(ratio) & 0x7fffffu) == 0u && ratio <= 32768.f) {
        const __half2 r2 = __float2half2_rn(ratio);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          __half2 lo, hi;
          widen4<KIND>(u[y], lo, hi);
          u[y] = narrow4<KIND>(lo, hi, r2);
        }
      } else {
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          float v[4];
          decode4<KIND>(u[y], v);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = v[e] * f * inv;  // the value (rounded to float), then an exact division
          u[y] = encode2<KIND>(v[0], v[1]) | (encode2<KIND>(v[2], v[3]) << 16);
        }
      }
      dst[i] = make_uint4(u[0], u[1], u[2], u[3]);
    }
    if (t == 0) (kv ? c.v_scale : c.k_scale)[(size_t)out * c.Hkv + h] = s;
  }
}

template <int KIND> cudaError_t launch_move(const EvictParams &p, cudaStream_t st) {
  const dim3 grid((unsigned)(p.c.B * p.out_pages), (unsigned)p.c.Hkv);
  const int pieces = (p.c.page * (p.c.D / 16) + kMoveThr - 1) / kMoveThr;  // at most 16: pages of 128 by 512
  if (pieces <= 1) return launch_dependent(cache_move_kernel<KIND, 1>, grid, kMoveThr, 0, st, p);
  if (pieces <= 2) return launch_dependent(cache_move_kernel<KIND, 2>, grid, kMoveThr, 0, st, p);
  if (pieces <= 4) return launch_dependent(cache_move_kernel<KIND, 4>, grid, kMoveThr, 0, st, p);
  if (pieces <= 8) return launch_dependent(cache_move_kernel<KIND, 8>, grid, kMoveThr, 0, st, p);
  return launch_dependent(cache_move_kernel<KIND, 16>, grid, kMoveThr, 0, st, p);
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int kind, cudaStream_t st) {
  // CTAs of a cluster: one for each 4096 positions of the table's width, up to the portable 8.
  const long long cap = (long long)p.c.max_pages << p.c.page_shift;
  int ranks = 1;
  while (ranks < 8 && ranks * 4096LL < cap) ranks *= 2;
  const long long part = (cap + ranks - 1) / ranks;
  const int in_smem = part <= kSelSmemKeys ? 1 : 0;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = raise_smem(cache_select_kernel, done, kSelSmemKeys * sizeof(unsigned));
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(p.c.B * p.c.Hkv * ranks));
  cfg.blockDim = dim3(kSelThr);
  cfg.dynamicSmemBytes = in_smem ? (size_t)part * sizeof(unsigned) : 0;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = ranks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if ((e = counted(cudaLaunchKernelEx(&cfg, cache_select_kernel, p, in_smem))) != cudaSuccess) return e;
  return kind == ATTN_CACHE_E4M3 ? launch_move<ATTN_CACHE_E4M3>(p, st) : launch_move<ATTN_CACHE_INT8>(p, st);
}

}  // namespace cache
}  // namespace attn
