// cache_fwd.cu -- attention over the 8-bit cache on fp32 FFMA (head dims above 256), and the kernels that the
// other paths end in as well: the join of split items and the accumulation of attention weights.
#include "cache_work.cuh"

namespace attn {
namespace cache {
namespace {

constexpr int kWarps = kThreads / 32;
constexpr int kRows = 8;  // rows of a work item on this path

template <typename T> __device__ __forceinline__ float4 load4f(const T *p);
template <> __device__ __forceinline__ float4 load4f<float>(const float *p) { return *reinterpret_cast<const float4 *>(p); }
template <> __device__ __forceinline__ float4 load4f<__nv_bfloat16>(const __nv_bfloat16 *p) {
  const uint2 u = *reinterpret_cast<const uint2 *>(p);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
template <typename T> __device__ __forceinline__ void store4f(T *p, float4 x);
template <> __device__ __forceinline__ void store4f<float>(float *p, float4 x) { *reinterpret_cast<float4 *>(p) = x; }
template <> __device__ __forceinline__ void store4f<__nv_bfloat16>(__nv_bfloat16 *p, float4 x) {
  __nv_bfloat162 a = __floats2bfloat162_rn(x.x, x.y), b = __floats2bfloat162_rn(x.z, x.w);
  uint2 u;
  u.x = *reinterpret_cast<uint32_t *>(&a);
  u.y = *reinterpret_cast<uint32_t *>(&b);
  *reinterpret_cast<uint2 *>(p) = u;
}

__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x = max_nan(x, __shfl_xor_sync(~0u, x, o));
  return x;
}
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
  return x;
}

// Four warps; each takes every fourth slice of 32 keys of the CTA's run.  Scores: one key per
// lane, its codes read 16 at a time and multiplied with the rows' queries broadcast from shared
// memory.  Output: four columns per lane (of each 128), the slice's probabilities broadcast from
// shared memory.  NC: 128-column parts of D.  16 flops a byte (2 * 2 * 8 rows * D per 2 * D bytes) would let
// the fp32 pipes keep up with two thirds of the memory's rate, but each load of queries or probabilities
// feeds four products only: 0.5 TB/s at D = 512 (one row of 114,000 keys, 8 kv heads, 4 queries to each).
template <typename T, int KIND, int NC>
__global__ void __launch_bounds__(kThreads) cache_fwd_simt_kernel(const __grid_constant__ FwdParams p) {
  extern __shared__ __align__(16) float sm[];
  const int D = p.c.D;
  float *s_q = sm;                      // [kRows][D]
  float *s_o = s_q + kRows * D;         // [kRows][D]
  float *s_p = s_o + kRows * D;         // [kWarps][kRows][32]
  float2 *s_ml = reinterpret_cast<float2 *>(s_p + kWarps * kRows * 32);  // [kWarps][kRows]
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  float *my_p = s_p + warp * kRows * 32;

  grid_launch_next();  // (one wave of CTAs: the join's blocks take nobody's place)
  __shared__ Groups s_groups;
  Cursor cur;
  if (!cursor_begin(p, &s_groups, cur)) return;
  Run run;
  while (cursor_next(p, &s_groups, cur, run)) {
    const int r0 = run.rt * kRows, rows = min(kRows, p.R - r0);
    __syncthreads();  // the previous run has left shared memory
    for (int x = t; x < kRows * D / 4; x += kThreads) {
      const int r = x / (D / 4), d = (x - r * (D / 4)) * 4;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < rows) {
        const int i = query_of(p, r0 + r), h = run.hk * p.G + (r0 + r - i * p.G);
        v = load4f(static_cast<const T *>(p.q) + run.b * p.q_sb + i * p.q_ss + h * p.q_sh + d);
      }
      *reinterpret_cast<float4 *>(s_q + r * D + d) = v;
    }
    __syncthreads();

    float m[kRows], l[kRows], acc[kRows][NC][4];
    int2 see[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      m[r] = -CUDART_INF_F;
      l[r] = 0.f;
      see[r] = row_sees(p, run.range.len, query_of(p, r0 + r));
#pragma unroll
      for (int c = 0; c < NC; ++c)
#pragma unroll
        for (int x = 0; x < 4; ++x) acc[r][c][x] = 0.f;
    }
    const int key0 = run.range.lo + (run.off << p.unit_shift), key1 = min(run.range.hi, key0 + (run.cnt << p.unit_shift));
    for (int base = key0 + warp * 32; base < key1; base += kWarps * 32) {
      const int pos = base + lane;
      int page = -1;
      if (pos < key1) page = page_of(p.c, run.b, pos);
      const int slot = pos & (p.c.page - 1);
      float s[kRows];
#pragma unroll
      for (int r = 0; r < kRows; ++r) s[r] = 0.f;
      float ks = 0.f, lv = 0.f;
      bool zero = true;
      if (page >= 0) {
        ks = p.c.k_scale[(size_t)page * p.c.Hkv + run.hk] * p.scale;
        lv = scale_log2(p.c.v_scale[(size_t)page * p.c.Hkv + run.hk], &zero);
        const uint4 *krow = reinterpret_cast<const uint4 *>(p.c.k + row_at(p.c, page, run.hk, slot));
        for (int d = 0; d < D; d += 16) {
          const uint4 w = krow[d >> 4];
          const unsigned ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            float x[4];
            decode4<KIND>(ww[y], x);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
              const float4 q = *reinterpret_cast<const float4 *>(s_q + r * D + d + 4 * y);
              s[r] = fmaf(q.x, x[0], fmaf(q.y, x[1], fmaf(q.z, x[2], fmaf(q.w, x[3], s[r]))));
            }
          }
        }
      }
      bool all = true;
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const bool vis = page >= 0 && r < rows && within(see[r], pos);
        all = all && (vis || r >= rows);
        float u = s[r] * ks;
        if (p.cap > 0.f) u = p.cap * tanhf(u * p.inv_cap);
        const float t2 = vis ? u * kLog2e : -CUDART_INF_F;
        if (p.scores && r < rows) scores_row(p, run.b, run.hk, r0 + r)[pos] = t2;
        const float e = t2 + lv;
        const float mn = max_nan(m[r], warp_max(e));
        float pr = 0.f, half = 1.f, one = 0.f;
        if (mn != -CUDART_INF_F) {
          pr = vis ? exp2f(e - mn) : 0.f;
          one = vis ? exp2f(t2 - mn + kFarUp) : 0.f;  // (by an exponential of its own whatever the scale: see cache_work.cuh)
          half = exp2f(0.5f * (m[r] - mn));
        }
        const float alpha = half * half;
        m[r] = mn;
        l[r] = rescaled(l[r], half) + one * 0x1p-40f;
        if (alpha != 1.f) {
#pragma unroll
          for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int x = 0; x < 4; ++x) acc[r][c][x] *= alpha;
        }
        my_p[r * 32 + lane] = zero ? 0.f : pr;
      }
      // Keys that some row does not see: their values are skipped for that row, not multiplied
      // by 0 (a code may be NaN).
      const bool skip0 = !__all_sync(~0u, all && !zero);
      __syncwarp();
      const int nk = min(32, key1 - base);
      for (int kk = 0; kk < nk; ++kk) {
        const int pg = __shfl_sync(~0u, page, kk);
        if (pg < 0) continue;
        const uint8_t *vrow = p.c.v + row_at(p.c, pg, run.hk, (base + kk) & (p.c.page - 1));
#pragma unroll
        for (int c = 0; c < NC; ++c) {
          const int d = c * 128 + lane * 4;
          if (d < D) {
            float x[4];
            decode4<KIND>(*reinterpret_cast<const unsigned *>(vrow + d), x);
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
              const float pr = my_p[r * 32 + kk];
              if (skip0 && pr == 0.f) continue;
#pragma unroll
              for (int y = 0; y < 4; ++y) acc[r][c][y] = fmaf(pr, x[y], acc[r][c][y]);
            }
          }
        }
      }
      __syncwarp();
    }

    // The four warps' rows joined in shared memory.
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      const float lr = warp_sum(l[r]);
      if (lane == 0) s_ml[warp * kRows + r] = make_float2(m[r], lr);
    }
    __syncthreads();
    float f[kRows];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      float M = -CUDART_INF_F;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = max_nan(M, s_ml[w * kRows + r].x);
      f[r] = m[r] == -CUDART_INF_F ? 0.f : exp2f(m[r] - M);
    }
    for (int w = 0; w < kWarps; ++w) {
      if (warp == w) {
#pragma unroll
        for (int r = 0; r < kRows; ++r)
#pragma unroll
          for (int c = 0; c < NC; ++c) {
            const int d = c * 128 + lane * 4;
            if (d < D) {
              float4 *o = reinterpret_cast<float4 *>(s_o + r * D + d);
              float4 v = w ? *o : make_float4(0.f, 0.f, 0.f, 0.f);
              if (f[r] != 0.f) {
                v.x += f[r] * acc[r][c][0];
                v.y += f[r] * acc[r][c][1];
                v.z += f[r] * acc[r][c][2];
                v.w += f[r] * acc[r][c][3];
              }
              *o = v;
            }
          }
      }
      __syncthreads();
    }
    const bool whole = run.cnt == run.n;
    for (int r = warp; r < rows; r += kWarps) {
      float M = -CUDART_INF_F, L = 0.f;
      for (int w = 0; w < kWarps; ++w) M = max_nan(M, s_ml[w * kRows + r].x);
      for (int w = 0; w < kWarps; ++w) {
        const float2 ml = s_ml[w * kRows + r];
        if (ml.x != -CUDART_INF_F) L += rescaled(ml.y, exp2f(0.5f * (ml.x - M)));
      }
      float scale = 1.f;
      if (whole) {
        const RowEnd e = row_end(p, run.hk * p.G + (r0 + r) % p.G, M, L);
        scale = e.scale;
        if (lane == 0) p.LSE[lse_at(p, run.b, run.hk, r0 + r)] = e.lse;
      } else if (lane == 0) {
        p.ml_part[(size_t)run.slot * kRows + r] = make_float2(M, L);
      }
      for (int d = lane * 4; d < D; d += 128) {
        float4 v = *reinterpret_cast<float4 *>(s_o + r * D + d);
        if (whole) {
          if (M == -CUDART_INF_F) v = make_float4(0.f, 0.f, 0.f, 0.f);
          v.x *= scale; v.y *= scale; v.z *= scale; v.w *= scale;
          store4f(static_cast<T *>(p.O) + o_row(p, run.b, run.hk, r0 + r) + d, v);
        } else {
          *reinterpret_cast<float4 *>(p.o_part + ((size_t)run.slot * kRows + r) * D + d) = v;
        }
      }
    }
  }
}

// The rows of items that are split (or empty): the parts' outputs weighted by 2^(M_c - M), and the extra
// column added once.  Bound by latency (prefix -> M, l -> O').  Many items have few parts each: a warp
// per row (PER_ROW = 1 warp), four rows to a block; few items have many: a block per row, its warps
// taking every fourth part.
template <typename T, int PER_ROW>
__global__ void __launch_bounds__(kThreads) cache_join_kernel(const __grid_constant__ FwdParams p) {
  __shared__ float4 s_o[PER_ROW][PER_ROW > 1 ? 128 : 1];
  __shared__ float2 s_ml[PER_ROW];
  grid_wait();
  grid_launch_next();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, D = p.c.D;
  const int hk = blockIdx.x / p.NG, g = blockIdx.x - hk * p.NG, b = g / p.RT, rt = g - b * p.RT;
  const int sub = PER_ROW > 1 ? (int)blockIdx.y : (int)blockIdx.y * kWarps + warp, r = rt * p.row_tile + sub;
  if (sub >= p.row_tile || r >= p.R) return;
  // The parts c0 .. c1 of the item, and where the row's partial of part c lies.
  int c0 = 0, c1 = -1, second = 0;
  if (p.splits) {
    c1 = p.splits - 1;
  } else {
    const int first = p.prefix[g], n = p.prefix[g + 1] - first, Uh = p.prefix[p.NG], s = hk * Uh + first;
    const Shares sh(Uh * p.c.Hkv, p.max_ctas);
    if (n > 0) {
      c0 = sh.owner(s);
      c1 = sh.owner(s + n - 1);
      if (c0 == c1) return;  // one CTA had the whole item
      // The item is the second of the first CTA's two if it begins behind that CTA's first unit, and the
      // first of every later one's.
      second = s > sh.begin(c0) ? 1 : 0;
    }
  }
  auto part = [&](int c) {
    const size_t slot = p.splits ? (size_t)blockIdx.x * p.splits + c : (size_t)(2 * c + (c == c0 ? second : 0));
    return slot * p.row_tile + sub;
  };
  const int me = PER_ROW > 1 ? warp : 0;
  // Running maximum and sum over this warp's parts, four at a time, loads first.
  float M = -CUDART_INF_F, L = 0.f;
  float4 acc[4];  // 512 columns
#pragma unroll
  for (int x = 0; x < 4; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
  for (int c = c0 + me; c <= c1; c += 4 * PER_ROW) {
    float2 ml[4];
    size_t at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ci = c + i * PER_ROW;
      at[i] = part(min(ci, c1));
      ml[i] = ci <= c1 ? p.ml_part[at[i]] : make_float2(-CUDART_INF_F, 0.f);
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int d = x * 128 + lane * 4;
      if (x * 128 >= D) break;
      float4 v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = d < D ? *reinterpret_cast<const float4 *>(p.o_part + at[i] * D + d) : make_float4(0.f, 0.f, 0.f, 0.f);
      float top = M;
#pragma unroll
      for (int i = 0; i < 4; ++i) top = max_nan(top, ml[i].x);
      const float a = top == -CUDART_INF_F ? 1.f : exp2f(M - top);
      acc[x].x *= a; acc[x].y *= a; acc[x].z *= a; acc[x].w *= a;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (ml[i].x == -CUDART_INF_F) continue;
        const float f = exp2f(ml[i].x - top);
        acc[x].x += f * v[i].x; acc[x].y += f * v[i].y; acc[x].z += f * v[i].z; acc[x].w += f * v[i].w;
      }
    }
    float top = M;
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max_nan(top, ml[i].x);
    L = rescaled(L, top == -CUDART_INF_F ? 1.f : exp2f(0.5f * (M - top)));
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (ml[i].x != -CUDART_INF_F) L += rescaled(ml[i].y, exp2f(0.5f * (ml[i].x - top)));
    M = top;
  }
  if (PER_ROW > 1) {  // the warps' parts of the row
    if (lane == 0) s_ml[warp] = make_float2(M, L);
    __syncthreads();
    const float mine = M;
    L = 0.f;
#pragma unroll
    for (int w = 0; w < PER_ROW; ++w) M = max_nan(M, s_ml[w].x);
#pragma unroll
    for (int w = 0; w < PER_ROW; ++w)
      if (s_ml[w].x != -CUDART_INF_F) L += rescaled(s_ml[w].y, exp2f(0.5f * (s_ml[w].x - M)));
    const float f = mine == -CUDART_INF_F ? 0.f : exp2f(mine - M);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (x * 128 >= D) break;
      s_o[warp][PER_ROW > 1 ? x * 32 + lane : 0] = make_float4(f * acc[x].x, f * acc[x].y, f * acc[x].z, f * acc[x].w);
    }
    __syncthreads();
  }
  const RowEnd e = row_end(p, hk * p.G + r % p.G, M, L);
  const bool none = M == -CUDART_INF_F;
  T *out = static_cast<T *>(p.O) + o_row(p, b, hk, r);
  if (PER_ROW > 1 ? threadIdx.x == 0 : lane == 0) p.LSE[lse_at(p, b, hk, r)] = e.lse;
  auto put = [&](int d, float4 o) {
    if (none) o = make_float4(0.f, 0.f, 0.f, 0.f);
    o.x *= e.scale; o.y *= e.scale; o.z *= e.scale; o.w *= e.scale;
    store4f(out + d, o);
  };
  if (PER_ROW > 1) {
    const int d = threadIdx.x * 4;
    if (d < D) {
      float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < PER_ROW; ++w) {
        const float4 v = s_o[w][PER_ROW > 1 ? threadIdx.x : 0];
        o.x += v.x; o.y += v.y; o.z += v.z; o.w += v.w;
      }
      put(d, o);
    }
  } else {
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (x * 128 + lane * 4 < D) put(x * 128 + lane * 4, acc[x]);
  }
}

// weights_out = weights + sum over the rows of 2^(score - LSE): four keys per thread, the rows'
// scores read as the attention kernel stored them, four rows at a time (loads before sums: bound by
// the latency of each otherwise), summed in row order.  A block takes the queries that see any of its keys, which
// are neighbours; where there are none, nothing is read, and in place nothing is written either.
__global__ void __launch_bounds__(kThreads) cache_weights_kernel(const __grid_constant__ FwdParams p) {
  constexpr int kKeys = 4 * kThreads;
  const int b = blockIdx.x / p.c.Hkv, hk = blockIdx.x - b * p.c.Hkv;
  const int len = seq_len(p.c, b);
  const int k0 = blockIdx.y * kKeys, j0 = k0 + threadIdx.x * 4;
  const int q0 = len - p.Sq;  // position of query 0
  const int i0 = p.causal ? max(0, k0 - q0) : 0;                                        // the first query that sees one of the block's keys,
  const int i1 = p.window > 0 ? min(p.Sq, k0 + kKeys - 1 + p.window - q0) : p.Sq;       // and the first behind them
  const bool any = k0 < len && i0 < i1;
  const size_t at = (size_t)b * p.w_sb + (size_t)hk * p.w_sh + j0;
  float w[4] = {0.f, 0.f, 0.f, 0.f}, sum[4] = {0.f, 0.f, 0.f, 0.f};
  if (any || p.w_in != p.w_out) {
#pragma unroll
    for (int x = 0; x < 4; ++x)
      if (j0 + x < len) w[x] = p.w_in[at + x];
  }
  grid_wait();
  if (j0 >= len || (!any && p.w_in == p.w_out)) return;
  const int first = any ? i0 * p.G : 0, r1 = any ? i1 * p.G : 0;  // rows
  const float *row = scores_row(p, b, hk, first) + j0;
  const float *lse = p.LSE + ((size_t)b * p.Hq + hk * p.G) * p.Sq;
  int query = i0, head = 0;  // of row r0 + i
#pragma unroll 1
  for (int r0 = first; r0 < r1; r0 += 4, row += 4 * p.Lpad) {
    // Scores are stored for the keys that some row of the tile sees (a superset of what a row sees); the others, and
    // the last row's in place of those past it, are loaded too, unconditionally so that all loads go out at once (behind
    // conditions each waited for the one before: 86 sequences of 135 keys, 16 heads, 15 rows, 20 us for this pass
    // instead of 13), and not used.
    int2 see[4];
    float lse2[4];
    float4 s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lse2[i] = lse[(size_t)head * p.Sq + query];
      s[i] = *reinterpret_cast<const float4 *>(row + (min(r0 + i, r1 - 1) - r0) * p.Lpad);
      see[i] = row_sees(p, len, query);
      if (r0 + i >= r1) see[i] = make_int2(0, 0);
      if (r0 + i < r1 - 1 && ++head == p.G) {
        head = 0;
        ++query;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) lse2[i] *= kLog2e;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float t[4] = {s[i].x, s[i].y, s[i].z, s[i].w};
#pragma unroll
      for (int x = 0; x < 4; ++x)
        if (within(see[i], j0 + x)) sum[x] += t[x] == -CUDART_INF_F ? 0.f : exp2f(t[x] - lse2[i]);
    }
  }
#pragma unroll
  for (int x = 0; x < 4; ++x)
    if (j0 + x < len) p.w_out[at + x] = w[x] + sum[x];
}

template <typename T, int KIND>
cudaError_t launch_simt_t(const FwdParams &p, cudaStream_t st) {
  const int D = p.c.D;
  const size_t smem = (size_t)(2 * kRows * D + kWarps * kRows * 32) * 4 + kWarps * kRows * 8;
  auto go = [&](auto kernel) {
    kernel<<<p.max_ctas, kThreads, smem, st>>>(p);
    return counted(cudaGetLastError());
  };
  return D <= 384 ? go(cache_fwd_simt_kernel<T, KIND, 3>) : go(cache_fwd_simt_kernel<T, KIND, 4>);
}

}  // namespace

int simt_row_tile() { return kRows; }
int simt_unit_shift() { return 7; }  // four warps of 32 keys

cudaError_t launch_fwd_simt(const FwdParams &p, int dtype, int kind, cudaStream_t st) {
  if (dtype == kF32)
    return kind == ATTN_CACHE_E4M3 ? launch_simt_t<float, ATTN_CACHE_E4M3>(p, st) : launch_simt_t<float, ATTN_CACHE_INT8>(p, st);
  return kind == ATTN_CACHE_E4M3 ? launch_simt_t<__nv_bfloat16, ATTN_CACHE_E4M3>(p, st)
                                 : launch_simt_t<__nv_bfloat16, ATTN_CACHE_INT8>(p, st);
}

template <typename T> static cudaError_t launch_join_t(const FwdParams &p, cudaStream_t st) {
  const int rows = min(p.row_tile, p.R);
  const unsigned items = (unsigned)(p.NG * p.c.Hkv);
  // Parts per item are at most 1 + CTAs / items on average.
  if ((long long)items * 4 >= p.max_ctas || (p.splits && p.splits <= 4))
    return launch_dependent(cache_join_kernel<T, 1>, dim3(items, (rows + kWarps - 1) / kWarps), kThreads, 0, st, p);
  return launch_dependent(cache_join_kernel<T, kWarps>, dim3(items, rows), kThreads, 0, st, p);
}

cudaError_t launch_fwd_join(const FwdParams &p, int dtype, cudaStream_t st) {
  return dtype == kF32 ? launch_join_t<float>(p, st) : launch_join_t<__nv_bfloat16>(p, st);
}

cudaError_t launch_weights(const FwdParams &p, cudaStream_t st) {
  const long long cap = (long long)p.c.max_pages << p.c.page_shift;
  const dim3 grid((unsigned)(p.c.B * p.c.Hkv), (unsigned)((cap + 4 * kThreads - 1) / (4 * kThreads)));
  return launch_dependent(cache_weights_kernel, grid, kThreads, 0, st, p);
}

}  // namespace cache
}  // namespace attn
