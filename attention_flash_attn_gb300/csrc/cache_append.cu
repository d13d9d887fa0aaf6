// cache_append.cu -- quantisation of new tokens into the paged 8-bit cache.
//
// One block per (sequence, page the new tokens touch, kv head, K or V).  The new rows' largest
// magnitude gives the scale they need, the least power of two; a page that holds earlier tokens
// keeps the larger of that and its present scale, and when it grows, the earlier codes are moved to
// it.  Bound by reading the new rows (2 or 4 bytes a value) and writing codes (1 byte).
#include "cache_common.cuh"

namespace attn {
namespace cache {
namespace {

constexpr int kThr = 256;

template <typename T> __device__ __forceinline__ void load8(const T *p, float *x);
template <> __device__ __forceinline__ void load8<float>(const float *p, float *x) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
template <> __device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16 *p, float *x) {
  const uint4 u = *reinterpret_cast<const uint4 *>(p);
  const unsigned w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

template <int KIND> __device__ __forceinline__ uint2 encode8(const float *x, float inv) {
  uint2 o;
  o.x = encode2<KIND>(x[0] * inv, x[1] * inv) | (encode2<KIND>(x[2] * inv, x[3] * inv) << 16);
  o.y = encode2<KIND>(x[4] * inv, x[5] * inv) | (encode2<KIND>(x[6] * inv, x[7] * inv) << 16);
  return o;
}

// Maximum over the block; every thread gets it.
__device__ __forceinline__ float block_max(float x) {
  __shared__ float s_m[kThr / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(~0u, x, o));
  if ((threadIdx.x & 31) == 0) s_m[threadIdx.x >> 5] = x;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThr / 32; ++w) x = fmaxf(x, s_m[w]);
  return x;
}

template <typename T, int KIND>
__global__ void __launch_bounds__(kThr) cache_append_kernel(const __grid_constant__ AppendParams p) {
  const View &c = p.c;
  const int b = blockIdx.x / p.span, nth = blockIdx.x - b * p.span, h = blockIdx.y, t = threadIdx.x;
  const bool val = blockIdx.z == 1;
  bool bad;
  const int len = seq_len(c, b, &bad);
  int cnt = p.counts ? p.counts[b] : p.S;
  cnt = cnt < 0 ? 0 : min(cnt, p.S);
  const long long cap = (long long)c.max_pages << c.page_shift;
  const int end = (int)(len + (long long)cnt > cap ? cap : len + (long long)cnt);  // positions [len, end) get a token
  if (nth == 0 && h == 0 && !val && t == 0) {
    if (p.lengths_out) p.lengths_out[b] = end;
    if (bad || end < len + (long long)cnt) set_status(c.status, kStatusBadPage);
  }
  const int slot_page = (len >> c.page_shift) + nth;     // column of the table
  const int first = max(len, slot_page << c.page_shift);  // the page's new positions: [first, last)
  const int last = min((long long)end, ((long long)slot_page + 1) << c.page_shift);
  if (first >= last) return;
  const int page = page_of(c, b, first);
  if (!val && p.weights)
    for (int x = first + t; x < last; x += kThr) p.weights[b * p.w_sb + h * p.w_sh + x] = 0.f;
  if (page < 0) return;
  const int D = c.D, per = D / 8, fresh = last - first, old = first & (c.page - 1);
  const T *src = static_cast<const T *>(val ? p.v : p.k) + b * (val ? p.v_sb : p.k_sb) + h * (val ? p.v_sh : p.k_sh);
  const long long ss = val ? p.v_ss : p.k_ss;
  uint8_t *dst = (val ? c.v : c.k) + row_at(c, page, h, 0);
  float *sc = (val ? c.v_scale : c.k_scale) + (size_t)page * c.Hkv + h;

  float amax = 0.f;
  bool odd = false;
  for (int x = t; x < fresh * per; x += kThr) {
    const int r = x / per, d = (x - r * per) * 8;
    float v[8];
    load8(src + (first - len + r) * ss + d, v);
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      const float a = fabsf(v[y]);
      if (a <= 3.402823466e38f) amax = fmaxf(amax, a);
      else odd = true;
    }
  }
  if (odd) set_status(c.status, kStatusNonFinite);
  const float was = *sc;
  amax = block_max(amax);  // (and every thread has read the old scale)
  float s = need_scale<KIND>(amax);
  if (old > 0 && was >= s) s = was;
  const float inv = 1.f / s;  // exact for the powers of two that this library writes
  for (int x = t; x < fresh * per; x += kThr) {
    const int r = x / per, d = (x - r * per) * 8;
    float v[8];
    load8(src + (first - len + r) * ss + d, v);
    *reinterpret_cast<uint2 *>(dst + (size_t)(old + r) * D + d) = encode8<KIND>(v, inv);
  }
  if (old > 0 && s != was) {
    const float f = was * inv;
    for (int x = t; x < old * per; x += kThr) {
      uint2 *at = reinterpret_cast<uint2 *>(dst) + x;
      const uint2 w = *at;
      float v[8];
      decode4<KIND>(w.x, v);
      decode4<KIND>(w.y, v + 4);
      *at = encode8<KIND>(v, f);
    }
  }
  if (t == 0) *sc = s;
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, int dtype, int kind, cudaStream_t st) {
  const dim3 grid((unsigned)(p.c.B * p.span), (unsigned)p.c.Hkv, 2);
  if (dtype == kF32) {
    if (kind == ATTN_CACHE_E4M3) cache_append_kernel<float, ATTN_CACHE_E4M3><<<grid, kThr, 0, st>>>(p);
    else cache_append_kernel<float, ATTN_CACHE_INT8><<<grid, kThr, 0, st>>>(p);
  } else {
    if (kind == ATTN_CACHE_E4M3) cache_append_kernel<__nv_bfloat16, ATTN_CACHE_E4M3><<<grid, kThr, 0, st>>>(p);
    else cache_append_kernel<__nv_bfloat16, ATTN_CACHE_INT8><<<grid, kThr, 0, st>>>(p);
  }
  return counted(cudaGetLastError());
}

}  // namespace cache
}  // namespace attn
