// cache_work.cuh -- how attention over the cache is spread over the grid, and how a piece of work
// ends.  Work items are (kv head, sequence, row tile); an item's keys are cut into units (a slice for each warp),
// and the units of all items, in that order, are shared out evenly over the CTAs: one long
// sequence is split over the whole grid, many short ones are run several to a CTA, and ragged
// batches balance.  A CTA turns each run of units of one item into either the item's result, if
// it holds all of them, or a partial (exponent reference, sum, unnormalised output), which the
// join kernel combines.  A CTA has at most two partials: that of the item it begins in, and that
// of the item it ends in.
//
// Numbers.  With a value's scale 2^lv, a row keeps M >= max_j(t_j + lv_j) in base 2 and
//   O' = sum_j 2^(t_j + lv_j - M) code_j,      l = sum_j 2^(t_j + lv_j - M) 2^-lv_j,
// so the scale costs nothing per element of V and the 2^(..) fed to the MMA stay within (0, 1]
// whatever the pages' scales; O = O' / l and LSE = ln2 (M + log2 l).
// Beside a value scale 2^126 times as large, a key's 2^(t + lv - M) is 0 in float where its 2^(t - M) may be all of the
// sum (and its value nothing of the output), and M moves by more than float's exponents between terms of one size.
// Where the scales of a run's keys lie more than kFar apart, its rows' sums are therefore formed once more at its
// end, key by key, by exponentials of their own (recount); nearer ones lose 2^-46 of the sum for each key, or less.
// Parts are joined with their sums rescaled in two steps.
#pragma once

#include "cache_common.cuh"

namespace attn {
namespace cache {

constexpr int kThreads = 128;

// The units of a CTA, item by item.  Unit counts fit 31 bits (checked on the host).
struct Cursor {
  int Uh;         // units of one kv head
  int u0, u, u1;  // this CTA's units; u: the next one
  int hk, g;      // item of unit u
  int g_first;    // first unit of that item
};

// A run of units [off, off + cnt) of item (hk, b, rt), which has n of them.
struct Run {
  int hk, b, rt, off, cnt, n, slot;  // slot: where a partial goes
  Range range;
};

__device__ __forceinline__ Range range_of(const FwdParams &p, int g) {
  const int b = p.RT == 1 ? g : g / p.RT;
  return group_range(p, b, g - b * p.RT);
}

// The groups' ranges in shared memory, where they fit: few groups are the calls that take microseconds,
// and each would be read from memory and worked out again for every run.
struct Groups {
  int4 r[32];  // lo, hi, len, units
};
__device__ __forceinline__ bool few_groups(const FwdParams &p) { return p.NG <= 32; }

// False if this CTA has no units.  CTA 0 stores the prefix sums and records lengths outside the table.
// Called by all kThreads threads.  Few groups: every warp does it all, a group per lane, with no
// barrier; many: each thread has a contiguous part of them.
__device__ __forceinline__ bool cursor_begin(const FwdParams &p, Groups *few, Cursor &cur) {
  __shared__ int s_sum[kThreads / 32], s_at[2];
  const int t = threadIdx.x, lane = t & 31;
  int Uh = 0, excl, sum = 0, g0, per = 1;
  if (few_groups(p)) {
    g0 = lane;
    if (lane < p.NG) {
      const Range r = range_of(p, lane);
      sum = range_units(p, r);
      few->r[lane] = make_int4(r.lo, r.hi, r.len, sum);  // (every warp writes the same)
    }
  } else {
    per = (p.NG + kThreads - 1) / kThreads;
    g0 = min(p.NG, t * per);
#pragma unroll 1
    for (int g = g0; g < min(p.NG, g0 + per); ++g) sum += range_units(p, range_of(p, g));
  }
  int incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(~0u, incl, o);
    if (lane >= o) incl += v;
  }
  excl = incl - sum;
  if (few_groups(p)) {
    Uh = __shfl_sync(~0u, incl, 31);
    __syncwarp();
  } else {
    if (lane == 31) s_sum[t >> 5] = incl;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < (t >> 5)) excl += s_sum[w];
      Uh += s_sum[w];
    }
  }
  if (blockIdx.x == 0 && (t < 32 || !few_groups(p))) {
    int x = excl;
#pragma unroll 1
    for (int g = g0; g < min(p.NG, g0 + per); ++g) {
      p.prefix[g] = x;
      x += range_units(p, range_of(p, g));
    }
    if (t == 0) p.prefix[p.NG] = Uh;
#pragma unroll 1
    for (int b = t; b < p.c.B; b += few_groups(p) ? 32 : kThreads) {
      bool bad;
      seq_len(p.c, b, &bad);
      if (bad) set_status(p.c.status, kStatusBadPage);
    }
  }
  const Shares sh(Uh * p.c.Hkv, p.max_ctas);
  if (blockIdx.x >= sh.C) return false;
  cur.Uh = Uh;
  cur.u0 = cur.u = sh.begin(blockIdx.x);
  cur.u1 = sh.begin(blockIdx.x + 1);
  cur.hk = cur.u / Uh;
  const int r = cur.u - cur.hk * Uh;
  const bool here = excl <= r && r < excl + sum;
  if (few_groups(p)) {
    const int at = __ffs(__ballot_sync(~0u, here)) - 1;
    cur.g = at;
    cur.g_first = cur.hk * Uh + __shfl_sync(~0u, excl, at);
    return true;
  }
  if (here) {
    int x = excl, g = g0;
#pragma unroll 1
    for (;; ++g) {
      const int n = range_units(p, range_of(p, g));
      if (r < x + n) break;
      x += n;
    }
    s_at[0] = g;
    s_at[1] = x;
  }
  __syncthreads();
  cur.g = s_at[0];
  cur.g_first = cur.hk * Uh + s_at[1];
  return true;
}

// The next run of this CTA; false when there is none.  Uniform over the CTA.
__device__ __forceinline__ bool cursor_next(const FwdParams &p, const Groups *few, Cursor &cur, Run &run) {
  if (cur.u >= cur.u1) return false;
#pragma unroll 1
  for (;;) {
    if (few_groups(p)) {
      const int4 r = few->r[cur.g];
      run.range.lo = r.x;
      run.range.hi = r.y;
      run.range.len = r.z;
      run.n = r.w;
    } else {
      run.range = range_of(p, cur.g);
      run.n = range_units(p, run.range);
    }
    if (cur.u < cur.g_first + run.n) break;
    cur.g_first += run.n;
    if (++cur.g == p.NG) {
      cur.g = 0;
      ++cur.hk;
    }
  }
  run.b = p.RT == 1 ? cur.g : cur.g / p.RT;
  run.rt = cur.g - run.b * p.RT;
  run.hk = cur.hk;
  run.off = cur.u - cur.g_first;
  run.cnt = min(run.n - run.off, cur.u1 - cur.u);
  run.slot = 2 * blockIdx.x + (cur.g_first > cur.u0 ? 1 : 0);
  cur.u += run.cnt;
  return true;
}

// The keys [lo, hi) that query i of a sequence of `len` tokens sees.
__device__ __forceinline__ int2 row_sees(const FwdParams &p, int len, int i) {
  const int pos = len - p.Sq + i;
  return make_int2(p.window > 0 ? max(0, pos - p.window + 1) : 0, p.causal ? max(0, min(len, pos + 1)) : len);
}
__device__ __forceinline__ bool within(int2 see, int key) { return key >= see.x && key < see.y; }

// The logarithm (base 2) of a page's value scale; scales below 2^-60 count as 0.
__device__ __forceinline__ float scale_log2(float vs, bool *zero) {
  *zero = !(vs >= kMinScale);
  return log2f(*zero ? kMinScale : vs);
}

constexpr float kFar = 80.f;
constexpr float kFarTop = kMinScaleExp - 1 + kFar;  // with no lv above it (2^19), none lie further apart
constexpr float kFarUp = 40.f;  // what recounted terms are held times (log2): see recount

// l * 2^(2 h), in two steps (`half`: 2^h).
__device__ __forceinline__ float rescaled(float l, float half) { return l * half * half; }

// Elements x .. x + 3 of a row of queries.
__device__ __forceinline__ float4 query4(const float *q) { return *reinterpret_cast<const float4 *>(q); }
__device__ __forceinline__ float4 query4(const __nv_bfloat16 *q) {
  const uint2 u = *reinterpret_cast<const uint2 *>(q);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}

// The keys of a run that one warp has: `block` keys from `first` on, and from every `stride` keys further on, below `end`.
struct Keys {
  int first, block, stride, end;
};

// Whether the value scales of these keys lie more than kFar apart (log2).  Called by a warp.
static __device__ __noinline__ bool far_apart(const FwdParams &p, int b, int hk, Keys k) {
  float lo = CUDART_INF_F, hi = -CUDART_INF_F;
  const int lane = threadIdx.x & 31;
  for (int base = k.first; base < k.end; base += k.stride)
    for (int pos = base + 16 * lane; pos < min(k.end, base + k.block); pos += 512) {
      const int page = page_of(p.c, b, pos);
      if (page < 0) continue;
      bool zero;
      const float lv = scale_log2(p.c.v_scale[(size_t)page * p.c.Hkv + hk], &zero);
      lo = fminf(lo, lv);
      hi = fmaxf(hi, lv);
    }
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    lo = fminf(lo, __shfl_xor_sync(~0u, lo, o));
    hi = fmaxf(hi, __shfl_xor_sync(~0u, hi, o));
  }
  return hi - lo > kFar;
}

// The sum over these keys of row r's 2^(t - M), in fp32 throughout: a key to a lane, the query broadcast.  Called by a
// warp, every lane gets the sum.  t - M <= 15 - lv <= 76 (M may lie 15 below the largest t + lv) does not overflow with
// kFarUp; what underflows is 2^-44 of the sum or less for each key (the sum is 2^-122 or more, as the largest scale is 2^122).
template <typename T, int KIND>
__device__ __noinline__ float recount(const FwdParams &p, int b, int hk, int r, int len, Keys k, float M) {
  if (M == -CUDART_INF_F) return 0.f;
  const int lane = threadIdx.x & 31, i = query_of(p, r), h = hk * p.G + (r - i * p.G);
  const T *q = static_cast<const T *>(p.q) + b * p.q_sb + i * p.q_ss + h * p.q_sh;
  const int2 see = row_sees(p, len, i);
  float sum = 0.f;
  for (int base = k.first; base < k.end; base += k.stride)
    for (int pos = base + lane; pos < min(k.end, base + k.block); pos += 32) {
      const int page = within(see, pos) ? page_of(p.c, b, pos) : -1;
      if (page < 0) continue;
      const uint4 *row = reinterpret_cast<const uint4 *>(p.c.k + row_at(p.c, page, hk, pos & (p.c.page - 1)));
      float s = 0.f;
#pragma unroll 1
      for (int d = 0; d < p.c.D; d += 16) {
        const uint4 w = row[d / 16];
        const unsigned words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          float x[4];
          decode4<KIND>(words[y], x);
          const float4 v = query4(q + d + 4 * y);
          s = fmaf(v.x, x[0], fmaf(v.y, x[1], fmaf(v.z, x[2], fmaf(v.w, x[3], s))));
        }
      }
      s *= p.c.k_scale[(size_t)page * p.c.Hkv + hk] * p.scale;
      if (p.cap > 0.f) s = p.cap * tanhf(s * p.inv_cap);
      sum += exp2f(s * kLog2e - M + kFarUp);
    }
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  return sum * exp2f(-kFarUp);
}

// A row's final factors from its reference M and sum l: O = O' * scale.  The extra softmax column
// (sink or off-by-one) enters here, once.
struct RowEnd {
  float scale, lse;
};
__device__ __forceinline__ RowEnd row_end(const FwdParams &p, int h, float M, float l) {
  RowEnd e;
  float top = M;
  if (p.sink || p.off_by_one) {
    const float s2 = p.sink ? p.sink[h] * kLog2e : 0.f;
    top = max_nan(M, s2);
    l = (M == -CUDART_INF_F ? 0.f : l * exp2f(M - top)) + exp2f(s2 - top);
    if (s2 == -CUDART_INF_F && M == -CUDART_INF_F) l = 0.f;
  }
  if (top == -CUDART_INF_F) {
    e.scale = 0.f;
    e.lse = -CUDART_INF_F;
  } else {
    e.scale = (M == -CUDART_INF_F ? 0.f : exp2f(M - top)) / l;
    e.lse = kLn2 * (top + log2f(l));
  }
  return e;
}

// Where row r of an item lives in O (first element) and in LSE.
__device__ __forceinline__ size_t o_row(const FwdParams &p, int b, int hk, int r) {
  const int i = query_of(p, r), h = hk * p.G + (r - i * p.G);
  return (((size_t)b * p.Sq + i) * p.Hq + h) * p.c.D;
}
__device__ __forceinline__ size_t lse_at(const FwdParams &p, int b, int hk, int r) {
  const int i = query_of(p, r), h = hk * p.G + (r - i * p.G);
  return ((size_t)b * p.Hq + h) * p.Sq + i;
}
__device__ __forceinline__ float *scores_row(const FwdParams &p, int b, int hk, int r) {
  return p.scores + (((size_t)b * p.c.Hkv + hk) * p.R + r) * p.Lpad;
}

}  // namespace cache
}  // namespace attn
