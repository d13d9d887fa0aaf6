// cache_evict.cu -- eviction by accumulated attention weight: which tokens stay, and their move
// to fresh pages.
#include <cooperative_groups.h>

#include "cache_common.cuh"

namespace attn {
namespace cache {
namespace {

namespace cg = cooperative_groups;

constexpr int kSelThr = 512, kSelWarps = kSelThr / 32;
constexpr int kMoveThr = 256;
constexpr int kSelSmemKeys = 49152;  // most weights that one CTA holds in shared memory (192 KB)

// Weights in an order of unsigned integers: larger weight, larger integer; -0 as +0, NaN largest.
__device__ __forceinline__ unsigned order_of(float w) {
  if (w != w) return 0xffffffffu;
  const unsigned u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One cluster per (sequence, kv head); each of its CTAs has a contiguous part of the middle positions
// [first, n - recent), whose weights it reads once and keeps in shared memory in their integer order
// (parts that do not fit are read again in every pass).  The K-th largest order T is found byte by byte:
// each CTA counts the next byte of its weights that share the bytes found so far, and every CTA adds
// up the cluster's counts through distributed shared memory.  Then every position above T stays, and
// of those equal to T the lowest ones: each warp has a contiguous part, placed by prefix sums over the
// warps' and the CTAs' counts, so that the result is ascending.  Lanes that count the same byte add once
// (weights share few exponents).  Bound by latency: five cluster barriers and passes over shared memory.
__global__ void __launch_bounds__(kSelThr) cache_select_kernel(const __grid_constant__ EvictParams p, int in_smem) {
  extern __shared__ unsigned s_key[];
  __shared__ unsigned s_hist[2][256], s_sum[256];
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
  float *w_out = p.weights_out + (size_t)pair * p.keep;
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
#pragma unroll 4
    for (int i = t; i < cnt; i += kSelThr) s_key[i] = order_of(wp[i]);
  }
  for (int i = t; i < 512; i += kSelThr) s_hist[0][i] = 0;
  __syncthreads();
  auto key = [&](int i) { return in_smem ? s_key[i] : order_of(wp[i]); };
  unsigned prefix = 0;
  int want = K;
#pragma unroll 1
  for (int pass = 0; pass < 4; ++pass) {
    const int shift = 24 - 8 * pass;
    unsigned *hist = s_hist[pass & 1];
    for (int i0 = warp * 32; i0 < cnt; i0 += kSelThr) {
      const int i = i0 + lane;
      const unsigned u = i < cnt ? key(i) : 0u;
      const bool in = i < cnt && (pass == 0 || (u >> (shift + 8)) == prefix);
      const unsigned digit = (u >> shift) & 255u;
      const unsigned same = __match_any_sync(~0u, in ? digit : 256u);
      if (in && (same & ((1u << lane) - 1)) == 0) atomicAdd(&hist[digit], __popc(same));
    }
    cluster.sync();
    // (The other buffer's counts were read before that barrier.)
    for (int i = t; i < 256; i += kSelThr) {
      unsigned x = 0;
      for (int r = 0; r < ranks; ++r) x += cluster.map_shared_rank(hist, r)[i];
      s_sum[i] = x;
      s_hist[(pass + 1) & 1][i] = 0;
    }
    __syncthreads();
    if (warp == 0) {  // lane l has the digits 255 - 8 l and the seven below
      int c[8], sum = 0;
#pragma unroll
      for (int x = 0; x < 8; ++x) sum += c[x] = (int)s_sum[255 - 8 * lane - x];
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += v;
      }
      int left = want - (incl - sum);
      if (left > 0 && left <= sum) {
        int x = 0;
#pragma unroll
        for (; x < 7; ++x) {
          if (left <= c[x]) break;
          left -= c[x];
        }
        s_found[0] = 255 - 8 * lane - x;
        s_found[1] = left;
      }
    }
    __syncthreads();
    prefix = (prefix << 8) | (unsigned)s_found[0];
    want = s_found[1];
  }
  const unsigned T = prefix;
  const int ties = want;  // positions equal to T that stay
  const int wpart = ((cnt + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int a = min(cnt, warp * wpart), z = min(cnt, a + wpart);
  int gt = 0, eq = 0;
  for (int i = a + lane; i < z; i += 32) {
    const unsigned u = key(i);
    gt += u > T;
    eq += u == T;
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
  for (int i0 = a; i0 < z; i0 += 32) {
    const int i = i0 + lane;
    const unsigned u = i < z ? key(i) : 0u;
    const unsigned mg = __ballot_sync(~0u, i < z && u > T), me = __ballot_sync(~0u, i < z && u == T);
    const unsigned below = (1u << lane) - 1;
    const int e = e0 + __popc(me & below), g = g0 + __popc(mg & below);
    if (i < z && (u > T || (u == T && e < ties))) {
      const int at = p.first + g + min(e, ties);
      kept[at] = a0 + i;
      w_out[at] = wp[i];
    }
    g0 += __popc(mg);
    e0 += __popc(me);
  }
  cluster.sync();  // no CTA leaves while another reads its counts
}

// One block per (page of table_out, sequence, kv head, K or V): the rows that go there, read once and held
// in registers (NP pieces of 16 codes per thread), their largest magnitude, their new scale, and their
// new codes.  Bound by the gather of the rows; the chain position -> page -> scale is walked once per row,
// into shared memory.
template <int KIND, int NP>
__global__ void __launch_bounds__(kMoveThr) cache_move_kernel(const __grid_constant__ EvictParams p) {
  __shared__ float s_m[kMoveThr / 32], s_scale[128];
  __shared__ long long s_row[128];  // first code of each row, or -1
  grid_wait();
  const View &c = p.c;
  const int b = blockIdx.x / p.out_pages, nth = blockIdx.x - b * p.out_pages, h = blockIdx.y, t = threadIdx.x;
  const bool val = blockIdx.z == 1;
  const int n = min(seq_len(c, b), p.keep), i0 = nth << c.page_shift, rows = min(c.page, n - i0);
  if (rows <= 0) return;
  const int out = p.table_out[b * p.table_out_stride + nth];
  if ((unsigned)out >= (unsigned)c.num_pages) {
    if (t == 0) set_status(c.status, kStatusBadPage);
    return;
  }
  const uint8_t *codes = val ? c.v : c.k;
  float *scales = val ? c.v_scale : c.k_scale;
  if (t < rows) {
    const int pos = p.kept[((size_t)b * c.Hkv + h) * p.keep + i0 + t], page = page_of(c, b, pos);
    s_row[t] = page < 0 ? -1 : (long long)row_at(c, page, h, pos & (c.page - 1));
    s_scale[t] = page < 0 ? 0.f : scales[(size_t)page * c.Hkv + h];
  }
  __syncthreads();
  const int per = c.D / 16, total = rows * per;
  uint4 w[NP];
  float f[NP];
#pragma unroll
  for (int x = 0; x < NP; ++x) {
    const int i = t + x * kMoveThr;
    w[x] = make_uint4(0, 0, 0, 0);
    f[x] = 0.f;
    if (i < total) {
      const int r = i / per, d = (i - r * per) * 16;
      f[x] = s_scale[r];
      if (s_row[r] >= 0) w[x] = *reinterpret_cast<const uint4 *>(codes + s_row[r] + d);
    }
  }
  float amax = 0.f;
#pragma unroll
  for (int x = 0; x < NP; ++x) {
    const unsigned u[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      float v[4];
      decode4<KIND>(u[y], v);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float m = fabsf(v[e] * f[x]);
        if (m <= 3.402823466e38f) amax = fmaxf(amax, m);
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  if ((t & 31) == 0) s_m[t >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int x = 0; x < kMoveThr / 32; ++x) amax = fmaxf(amax, s_m[x]);
  const float s = need_scale<KIND>(amax), inv = pow2_inverse(s);
  uint4 *dst = reinterpret_cast<uint4 *>((val ? c.v : c.k) + row_at(c, out, h, 0));
#pragma unroll
  for (int x = 0; x < NP; ++x) {
    const int i = t + x * kMoveThr;
    if (i >= total) continue;
    unsigned u[4] = {w[x].x, w[x].y, w[x].z, w[x].w};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      float v[4];
      decode4<KIND>(u[y], v);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = v[e] * f[x] * inv;  // the value (rounded to float), then an exact division
      u[y] = encode2<KIND>(v[0], v[1]) | (encode2<KIND>(v[2], v[3]) << 16);
    }
    dst[i] = make_uint4(u[0], u[1], u[2], u[3]);
  }
  if (t == 0) scales[(size_t)out * c.Hkv + h] = s;
}

template <int KIND> cudaError_t launch_move(const EvictParams &p, cudaStream_t st) {
  const dim3 grid((unsigned)(p.c.B * p.out_pages), (unsigned)p.c.Hkv, 2);
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
