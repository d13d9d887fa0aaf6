// cache_append.cu -- quantisation of new tokens into the paged 8-bit cache.
//
// The new rows' largest magnitude gives the scale they need, the least power of two; a page that holds
// earlier tokens keeps the larger of that and its present scale, and when it grows, the earlier codes are
// moved to it.  Prompts: one block per (sequence, page the new tokens touch, kv head), which reads its rows
// of K and V once, into registers (what does not fit there it reads again, from L2): 27 us for 8 ragged
// prompts of up to 4096 tokens, 8 heads, D = 128, bf16, 132 MB at 4.9 TB/s.  One block for K and one for V
// each took 31.  Single tokens: one warp each, 4 us for 4 sequences, 5 for 192.  Prompts are bound by reading
// the new rows (2 or 4 bytes a value) and writing codes (1 byte); single tokens by the chain length -> page
// -> scale, three loads that wait for one another, and by the launch.
#include "cache_common.cuh"

namespace attn {
namespace cache {
namespace {

constexpr int kThr = 256;
constexpr int kHeld = 4;  // pieces of 8 values that a thread keeps between the two looks at them

// Eight values as they lie in memory, as floats, and their largest magnitude (NaN if one is NaN).
template <typename T> struct Raw;
template <> struct Raw<float> {
  uint4 a, b;
  __device__ __forceinline__ void zero() { a = b = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const float *p) {
    a = reinterpret_cast<const uint4 *>(p)[0];
    b = reinterpret_cast<const uint4 *>(p)[1];
  }
  __device__ __forceinline__ void get(float *x) const {
    const unsigned w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(w[i]);
  }
  __device__ __forceinline__ float amax() const {
    float x[8], m = 0.f;
    get(x);
#pragma unroll
    for (int i = 0; i < 8; i += 2) m = max_nan(m, fabsf(x[i]), fabsf(x[i + 1]));
    return m;
  }
};
template <> struct Raw<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void zero() { a = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void get(float *x) const {
    const unsigned w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ float amax() const {
    const unsigned w[4] = {a.x, a.y, a.z, a.w};
    __nv_bfloat162 m = __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[0]));
#pragma unroll
    for (int i = 1; i < 4; ++i) m = __hmax2_nan(m, __habs2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i])));
    return max_nan(__low2float(m), __high2float(m));
  }
};

// Codes of 8 values in units of 1 / inv.  FIT: they are known to be finite and within the largest code.
template <int KIND, bool FIT> __device__ __forceinline__ uint2 encode8(const float *x, float inv) {
  uint2 o;
  if (KIND == ATTN_CACHE_INT8 && FIT) {
    unsigned u[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(fmaf(x[i], inv, 12582912.f));  // rounded once, to an integer
    o.x = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
    o.y = __byte_perm(__byte_perm(u[4], u[5], 0x0040), __byte_perm(u[6], u[7], 0x0040), 0x5410);
  } else {
    o.x = encode2<KIND>(x[0] * inv, x[1] * inv) | (encode2<KIND>(x[2] * inv, x[3] * inv) << 16);
    o.y = encode2<KIND>(x[4] * inv, x[5] * inv) | (encode2<KIND>(x[6] * inv, x[7] * inv) << 16);
  }
  return o;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = max_nan(x, __shfl_xor_sync(~0u, x, o));
  return x;
}
// Two maxima over the block; every thread gets them.
__device__ __forceinline__ void block_max2(float *x) {
  __shared__ float2 s_m[kThr / 32];
  const float a = warp_max(x[0]), b = warp_max(x[1]);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_m[threadIdx.x >> 5] = make_float2(a, b);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kThr / 32; ++w) {
    x[0] = max_nan(x[0], s_m[w].x);
    x[1] = max_nan(x[1], s_m[w].y);
  }
}

// Where a sequence's new tokens go: positions [len, end).  Writes the new length and records what is
// out of place, once per sequence.
struct Span {
  int len, end;
};
__device__ __forceinline__ Span new_span(const AppendParams &p, int b, bool once) {
  bool bad;
  Span s;
  s.len = seq_len(p.c, b, &bad);
  int cnt = p.counts ? p.counts[b] : p.S;
  cnt = cnt < 0 ? 0 : min(cnt, p.S);
  const long long want = s.len + (long long)cnt, cap = (long long)p.c.max_pages << p.c.page_shift;
  s.end = (int)(want > cap ? cap : want);
  if (once) {
    if (p.lengths_out) p.lengths_out[b] = s.end;
    if (bad || s.end < want) set_status(p.c.status, kStatusBadPage);
  }
  return s;
}

constexpr float kMaxFloat = 3.402823466e38f;
// Largest finite magnitude of 8 values.
__device__ __forceinline__ float amax_finite(const float *v, float amax) {
#pragma unroll
  for (int y = 0; y < 8; ++y)
    if (fabsf(v[y]) <= kMaxFloat) amax = fmaxf(amax, fabsf(v[y]));
  return amax;
}

// Moves n16 pieces of 16 codes to a scale 1 / f times as large; called by `threads` threads.
template <int KIND> __device__ __forceinline__ void rescale(uint4 *at, int n16, float f, int t, int threads) {
#pragma unroll 4
  for (int x = t; x < n16; x += threads) {
    const uint4 w = at[x];
    unsigned u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      float v[4];
      decode4<KIND>(u[y], v);
      u[y] = encode2<KIND>(v[0] * f, v[1] * f) | (encode2<KIND>(v[2] * f, v[3] * f) << 16);
    }
    at[x] = make_uint4(u[0], u[1], u[2], u[3]);
  }
}

template <typename T, int KIND>
__global__ void __launch_bounds__(kThr) cache_append_kernel(const __grid_constant__ AppendParams p) {
  const View &c = p.c;
  const int b = blockIdx.x / p.span, nth = blockIdx.x - b * p.span, h = blockIdx.y, t = threadIdx.x;
  const Span sp = new_span(p, b, nth == 0 && h == 0 && t == 0);
  const int len = sp.len, col = (len >> c.page_shift) + nth;  // column of the table
  const int first = max(len, col << c.page_shift);            // the page's new positions: [first, last)
  const int last = min((long long)sp.end, ((long long)col + 1) << c.page_shift);
  if (first >= last) return;
  const int D = c.D, per = D / 8, total = (last - first) * per, old = first & (c.page - 1);
  const T *src[2] = {static_cast<const T *>(p.k) + b * p.k_sb + h * p.k_sh + (first - len) * p.k_ss,
                     static_cast<const T *>(p.v) + b * p.v_sb + h * p.v_sh + (first - len) * p.v_ss};
  const long long ss[2] = {p.k_ss, p.v_ss};
  // This thread's pieces of the rows, in order: t, t + kThr, ...; row and place in the row of the current one.
  const int row0 = t / per, piece0 = t - row0 * per, dr = kThr / per, dp = kThr - dr * per;
  int row = row0, piece = piece0;
  auto advance = [&]() {
    row += dr;
    piece += dp;
    if (piece >= per) {
      piece -= per;
      ++row;
    }
  };
  auto fetch = [&](int kv, Raw<T> &v) { v.load(src[kv] + row * ss[kv] + piece * 8); };
  Raw<T> held[2][kHeld];
#pragma unroll
  for (int x = 0; x < kHeld; ++x) {
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      held[kv][x].zero();
      if (t + x * kThr < total) fetch(kv, held[kv][x]);
    }
    advance();
  }
  const int rest_row = row, rest_piece = piece;
  const int page = page_of(c, b, first);
  if (p.weights)
    for (int x = first + t; x < last; x += kThr) p.weights[b * p.w_sb + h * p.w_sh + x] = 0.f;
  if (page < 0) return;
  const size_t sc = (size_t)page * c.Hkv + h, at = row_at(c, page, h, 0);
  const float was[2] = {c.k_scale[sc], c.v_scale[sc]};
  float amax[2] = {0.f, 0.f};
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
#pragma unroll
    for (int x = 0; x < kHeld; ++x) amax[kv] = max_nan(amax[kv], held[kv][x].amax());
    row = rest_row;
    piece = rest_piece;
#pragma unroll 1
    for (int i = t + kHeld * kThr; i < total; i += kThr) {  // pages of more than 8192 values
      Raw<T> v;
      fetch(kv, v);
      advance();
      amax[kv] = max_nan(amax[kv], v.amax());
    }
  }
  block_max2(amax);  // (and every thread has read the old scales)
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    const bool fit = amax[kv] <= kMaxFloat;
    if (!fit) {  // something is infinite or NaN: the scale goes by the rest
      if (t == 0) set_status(c.status, kStatusNonFinite);
      float m[2] = {0.f, 0.f};
      row = row0;
      piece = piece0;
#pragma unroll 1
      for (int i = t; i < total; i += kThr) {
        Raw<T> v;
        fetch(kv, v);
        advance();
        float x[8];
        v.get(x);
        m[0] = amax_finite(x, m[0]);
      }
      block_max2(m);
      amax[kv] = m[0];
    }
    float s = need_scale<KIND>(amax[kv]);
    if (old > 0 && was[kv] >= s) s = was[kv];
    const float inv = 1.f / s;  // exact for the powers of two that this library writes
    uint8_t *dst = (kv ? c.v : c.k) + at;
    uint2 *to = reinterpret_cast<uint2 *>(dst + (size_t)old * D);
    if (fit) {
#pragma unroll
      for (int x = 0; x < kHeld; ++x)
        if (t + x * kThr < total) {
          float v[8];
          held[kv][x].get(v);
          to[t + x * kThr] = encode8<KIND, true>(v, inv);
        }
    }
    if (!fit || total > kHeld * kThr) {
      row = fit ? rest_row : row0;
      piece = fit ? rest_piece : piece0;
#pragma unroll 1
      for (int i = t + (fit ? kHeld * kThr : 0); i < total; i += kThr) {
        Raw<T> v;
        fetch(kv, v);
        advance();
        float x[8];
        v.get(x);
        to[i] = encode8<KIND, false>(x, inv);
      }
    }
    if (old > 0 && s != was[kv]) rescale<KIND>(reinterpret_cast<uint4 *>(dst), old * (D / 16), was[kv] * inv, t, kThr);
    if (t == 0) (kv ? c.v_scale : c.k_scale)[sc] = s;
  }
}

// S = 1: warp w of the grid has (sequence, kv head, K or V).  The row is fetched before the chain that
// says where it goes.
template <typename T, int KIND>
__global__ void __launch_bounds__(128) cache_append_token_kernel(const __grid_constant__ AppendParams p) {
  const View &c = p.c;
  const int task = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int b = task / (2 * c.Hkv), h = (task >> 1) - b * c.Hkv;
  if (b >= c.B) return;
  const bool val = task & 1;
  const int D = c.D, per = D / 8;
  const T *src = static_cast<const T *>(val ? p.v : p.k) + b * (val ? p.v_sb : p.k_sb) + h * (val ? p.v_sh : p.k_sh);
  Raw<T> v[2];  // D <= 512: at most two pieces a lane
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    v[i].zero();
    if (lane + 32 * i < per) v[i].load(src + (lane + 32 * i) * 8);
  }
  const Span sp = new_span(p, b, h == 0 && !val && lane == 0);
  if (sp.end <= sp.len) return;
  const int page = page_of(c, b, sp.len), old = sp.len & (c.page - 1);
  if (!val && p.weights && lane == 0) p.weights[b * p.w_sb + h * p.w_sh + sp.len] = 0.f;
  if (page < 0) return;
  uint8_t *dst = (val ? c.v : c.k) + row_at(c, page, h, 0);
  float *sc = (val ? c.v_scale : c.k_scale) + (size_t)page * c.Hkv + h;
  const float was = *sc;
  float amax = warp_max(max_nan(v[0].amax(), v[1].amax()));
  float x[2][8];
  v[0].get(x[0]);
  v[1].get(x[1]);
  const bool fit = amax <= kMaxFloat;
  if (!fit) {
    if (lane == 0) set_status(c.status, kStatusNonFinite);
    amax = warp_max(amax_finite(x[1], amax_finite(x[0], 0.f)));
  }
  float s = need_scale<KIND>(amax);
  if (old > 0 && was >= s) s = was;
  const float inv = 1.f / s;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (lane + 32 * i < per)
      reinterpret_cast<uint2 *>(dst + (size_t)old * D)[lane + 32 * i] = fit ? encode8<KIND, true>(x[i], inv) : encode8<KIND, false>(x[i], inv);
  if (old > 0 && s != was) rescale<KIND>(reinterpret_cast<uint4 *>(dst), old * (D / 16), was * inv, lane, 32);
  if (lane == 0) *sc = s;
}

template <typename T, int KIND> cudaError_t launch_append_t(const AppendParams &p, cudaStream_t st) {
  if (p.S == 1) {
    const long long tasks = 2LL * p.c.B * p.c.Hkv;
    cache_append_token_kernel<T, KIND><<<(unsigned)((tasks + 3) / 4), 128, 0, st>>>(p);
  } else {
    cache_append_kernel<T, KIND><<<dim3((unsigned)(p.c.B * p.span), (unsigned)p.c.Hkv), kThr, 0, st>>>(p);
  }
  return counted(cudaGetLastError());
}

}  // namespace

cudaError_t launch_append(const AppendParams &p, int dtype, int kind, cudaStream_t st) {
  if (dtype == kF32)
    return kind == ATTN_CACHE_E4M3 ? launch_append_t<float, ATTN_CACHE_E4M3>(p, st) : launch_append_t<float, ATTN_CACHE_INT8>(p, st);
  return kind == ATTN_CACHE_E4M3 ? launch_append_t<__nv_bfloat16, ATTN_CACHE_E4M3>(p, st)
                                 : launch_append_t<__nv_bfloat16, ATTN_CACHE_INT8>(p, st);
}

}  // namespace cache
}  // namespace attn
