// cache_evict.cu -- eviction by accumulated attention weight: which tokens stay, and their move
// to fresh pages.
#include "cache_common.cuh"

namespace attn {
namespace cache {
namespace {

constexpr int kSelThr = 1024, kSelWarps = kSelThr / 32;
constexpr int kMoveThr = 256;

// Weights in an order of unsigned integers: larger weight, larger integer; -0 as +0, NaN largest.
__device__ __forceinline__ unsigned order_of(float w) {
  if (w != w) return 0xffffffffu;
  const unsigned u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// One block per (sequence, kv head).  Among the middle positions [first, n - recent) the K-th
// largest order T is found byte by byte (counts of each next byte among those that share the bytes
// found so far); then every position above T stays, and of those equal to T the lowest ones.  Each
// warp writes a contiguous part, placed by a prefix sum over the warps' counts, so that the
// result is ascending.  The weights stay in L2 over the passes.
__global__ void __launch_bounds__(kSelThr) cache_select_kernel(const __grid_constant__ EvictParams p) {
  __shared__ unsigned s_hist[256];
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
  __shared__ unsigned s_prefix;
  __shared__ int s_want;
  const int b = blockIdx.x / p.c.Hkv, h = blockIdx.x - b * p.c.Hkv;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  bool bad;
  const int len = seq_len(p.c, b, &bad), n = min(len, p.keep);
  if (t == 0 && h == 0) {
    p.lengths_out[b] = n;
    if (bad) set_status(p.c.status, kStatusBadPage);
  }
  int *kept = p.kept + (size_t)blockIdx.x * p.keep;
  float *w_out = p.weights_out + (size_t)blockIdx.x * p.keep;
  const float *w = p.weights + b * p.w_sb + h * p.w_sh;
  for (int i = n + t; i < p.keep; i += kSelThr) {
    kept[i] = -1;
    w_out[i] = 0.f;
  }
  if (len <= p.keep) {
    for (int i = t; i < n; i += kSelThr) {
      kept[i] = i;
      w_out[i] = w[i];
    }
    return;
  }
  const int lo = p.first, hi = len - p.recent, K = p.keep - p.first - p.recent;  // lo <= hi as len > keep
  for (int i = t; i < p.first; i += kSelThr) {
    kept[i] = i;
    w_out[i] = w[i];
  }
  for (int i = t; i < p.recent; i += kSelThr) {
    kept[p.keep - p.recent + i] = hi + i;
    w_out[p.keep - p.recent + i] = w[hi + i];
  }
  if (K == 0) return;
  if (t == 0) {
    s_prefix = 0;
    s_want = K;
  }
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int i = t; i < 256; i += kSelThr) s_hist[i] = 0;
    __syncthreads();
    const unsigned prefix = s_prefix;
    for (int i = lo + t; i < hi; i += kSelThr) {
      const unsigned u = order_of(w[i]);
      if (shift == 24 || (u >> (shift + 8)) == prefix) atomicAdd(&s_hist[(u >> shift) & 255u], 1u);
    }
    __syncthreads();
    if (t == 0) {
      int want = s_want, x = 255;
      while (x > 0 && (int)s_hist[x] < want) want -= (int)s_hist[x--];
      s_prefix = (prefix << 8) | (unsigned)x;
      s_want = want;
    }
    __syncthreads();
  }
  const unsigned T = s_prefix;
  const int ties = s_want;  // positions equal to T that stay
  const int part = ((hi - lo + kSelWarps - 1) / kSelWarps + 31) & ~31;
  const int a = min((long long)hi, lo + (long long)warp * part), z = min((long long)hi, a + (long long)part);
  int gt = 0, eq = 0;
  for (int i = a + lane; i < z; i += 32) {
    const unsigned u = order_of(w[i]);
    gt += u > T;
    eq += u == T;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    gt += __shfl_xor_sync(~0u, gt, o);
    eq += __shfl_xor_sync(~0u, eq, o);
  }
  if (lane == 0) {
    s_gt[warp] = gt;
    s_eq[warp] = eq;
  }
  __syncthreads();
  int g0 = 0, e0 = 0;  // above T, equal to T, in the parts before
  for (int x = 0; x < warp; ++x) {
    g0 += s_gt[x];
    e0 += s_eq[x];
  }
  for (int i0 = a; i0 < z; i0 += 32) {
    const int i = i0 + lane;
    const float wi = i < z ? w[i] : 0.f;
    const unsigned u = order_of(wi);
    const unsigned mg = __ballot_sync(~0u, i < z && u > T), me = __ballot_sync(~0u, i < z && u == T);
    const unsigned below = (1u << lane) - 1;
    const int e = e0 + __popc(me & below), g = g0 + __popc(mg & below);
    if (i < z && (u > T || (u == T && e < ties))) {
      const int at = p.first + g + min(e, ties);
      kept[at] = i;
      w_out[at] = wi;
    }
    g0 += __popc(mg);
    e0 += __popc(me);
  }
}

// One block per (page of table_out, sequence, kv head, K or V): the rows that go there, dequantised,
// their largest magnitude, their new scale, and their new codes.
template <int KIND>
__global__ void __launch_bounds__(kMoveThr) cache_move_kernel(const __grid_constant__ EvictParams p) {
  __shared__ float s_m[kMoveThr / 32];
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
  const int *kept = p.kept + ((size_t)b * c.Hkv + h) * p.keep + i0;
  const uint8_t *codes = val ? c.v : c.k;
  float *scales = val ? c.v_scale : c.k_scale;
  const int per = c.D / 8;
  auto load = [&](int x, float *v) {
    const int r = x / per, d = (x - r * per) * 8, pos = kept[r], page = page_of(c, b, pos);
    if (page < 0) {
#pragma unroll
      for (int y = 0; y < 8; ++y) v[y] = 0.f;
      return;
    }
    const float s = scales[(size_t)page * c.Hkv + h];
    const uint2 w = *reinterpret_cast<const uint2 *>(codes + row_at(c, page, h, pos & (c.page - 1)) + d);
    decode4<KIND>(w.x, v);
    decode4<KIND>(w.y, v + 4);
#pragma unroll
    for (int y = 0; y < 8; ++y) v[y] *= s;
  };
  float amax = 0.f;
  for (int x = t; x < rows * per; x += kMoveThr) {
    float v[8];
    load(x, v);
#pragma unroll
    for (int y = 0; y < 8; ++y)
      if (fabsf(v[y]) <= 3.402823466e38f) amax = fmaxf(amax, fabsf(v[y]));
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
  if ((t & 31) == 0) s_m[t >> 5] = amax;
  __syncthreads();
#pragma unroll
  for (int x = 0; x < kMoveThr / 32; ++x) amax = fmaxf(amax, s_m[x]);
  const float s = need_scale<KIND>(amax), inv = pow2_inverse(s);
  uint8_t *dst = (val ? c.v : c.k) + row_at(c, out, h, 0);
  for (int x = t; x < rows * per; x += kMoveThr) {
    float v[8];
    load(x, v);
    uint2 o;
    o.x = encode2<KIND>(v[0] * inv, v[1] * inv) | (encode2<KIND>(v[2] * inv, v[3] * inv) << 16);
    o.y = encode2<KIND>(v[4] * inv, v[5] * inv) | (encode2<KIND>(v[6] * inv, v[7] * inv) << 16);
    reinterpret_cast<uint2 *>(dst)[x] = o;
  }
  if (t == 0) scales[(size_t)out * c.Hkv + h] = s;
}

}  // namespace

cudaError_t launch_evict(const EvictParams &p, int kind, cudaStream_t st) {
  cache_select_kernel<<<(unsigned)(p.c.B * p.c.Hkv), kSelThr, 0, st>>>(p);
  cudaError_t e = counted(cudaGetLastError());
  if (e != cudaSuccess) return e;
  const dim3 grid((unsigned)(p.c.B * p.out_pages), (unsigned)p.c.Hkv, 2);
  if (kind == ATTN_CACHE_E4M3) cache_move_kernel<ATTN_CACHE_E4M3><<<grid, kMoveThr, 0, st>>>(p);
  else cache_move_kernel<ATTN_CACHE_INT8><<<grid, kMoveThr, 0, st>>>(p);
  return counted(cudaGetLastError());
}

}  // namespace cache
}  // namespace attn
