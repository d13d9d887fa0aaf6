// cache_api.cu -- the C ABI declared in include/attn_cache_gb300.h: argument validation (fail
// closed: an invalid request never launches anything), workspace layout and launches.
#include <math.h>
#include <string.h>

#include <algorithm>

#include "cache_common.cuh"

namespace attn {
namespace cache {

namespace {

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool aligned16(const void *p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void *p) { return ((uintptr_t)p & 3u) == 0; }

int log2_of(int x) {
  int s = 0;
  while ((1 << s) < x) ++s;
  return s;
}

int validate(const attn_cache *c) {
  if (!c) return ATTN_ERR_INVALID;
  if (c->kind != ATTN_CACHE_E4M3 && c->kind != ATTN_CACHE_INT8) return ATTN_ERR_INVALID;
  if ((long long)c->num_pages * c->Hkv > INT_MAX) return ATTN_ERR_UNSUPPORTED;  // TMA coordinates
  if (c->num_pages < 1 || c->Hkv < 1 || c->Hkv > 65535 || c->D < 16) return ATTN_ERR_INVALID;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return ATTN_ERR_UNSUPPORTED;
  if (c->D % 16 != 0 || c->D > 512) return ATTN_ERR_UNSUPPORTED;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale || !c->status) return ATTN_ERR_INVALID;
  if (!aligned16(c->k) || !aligned16(c->v) || !aligned16(c->status)) return ATTN_ERR_INVALID;
  if (!aligned4(c->k_scale) || !aligned4(c->v_scale)) return ATTN_ERR_INVALID;
  return ATTN_OK;
}

int validate(const attn_cache *c, const attn_cache_seqs *s) {
  const int e = validate(c);
  if (e != ATTN_OK) return e;
  if (!s || s->B < 0 || s->max_pages < 0) return ATTN_ERR_INVALID;
  if ((long long)s->max_pages * c->page_size > (1LL << 24)) return ATTN_ERR_UNSUPPORTED;  // grids over positions
  if (s->B == 0) return ATTN_OK;
  if (!s->lengths || !aligned4(s->lengths)) return ATTN_ERR_INVALID;
  if (s->max_pages > 0 && (!s->table || !aligned4(s->table))) return ATTN_ERR_INVALID;
  if (s->table_stride < (s->B > 1 ? s->max_pages : 0)) return ATTN_ERR_INVALID;
  if ((long long)s->B * c->Hkv > INT_MAX / 16) return ATTN_ERR_UNSUPPORTED;  // grids (clusters of up to 16)
  return ATTN_OK;
}

View view(const attn_cache *c, const attn_cache_seqs *s) {
  View v;
  v.num_pages = c->num_pages;
  v.page = c->page_size;
  v.page_shift = log2_of(c->page_size);
  v.Hkv = c->Hkv;
  v.D = c->D;
  v.k = static_cast<uint8_t *>(c->k);
  v.v = static_cast<uint8_t *>(c->v);
  v.k_scale = c->k_scale;
  v.v_scale = c->v_scale;
  v.status = c->status;
  v.B = s->B;
  v.max_pages = s->max_pages;
  v.table = s->table;
  v.table_stride = s->table_stride;
  v.lengths = s->lengths;
  return v;
}

bool strides_ok(int dtype, std::initializer_list<int64_t> st) {
  const int64_t vec = dtype == ATTN_DTYPE_BF16 ? 8 : 4;  // elements per 16 bytes
  for (int64_t x : st)
    if (x < 0 || x % vec != 0) return false;
  return true;
}

// Rows of accumulated weights that a call writes, [B, Hkv, room], keep off one another.
bool rows_apart(const attn_cache *c, const attn_cache_seqs *s, int64_t sb, int64_t sh, int64_t room) {
  if (s->B <= 1) return c->Hkv <= 1 || sh >= room;
  if (c->Hkv <= 1) return sb >= room;
  const bool nested = sb >= sh;  // heads within sequences
  const int64_t in = nested ? sh : sb, out = nested ? sb : sh, count = nested ? c->Hkv : s->B;
  return in >= room && out >= (count - 1) * in + room;
}
int64_t table_room(const attn_cache *c, const attn_cache_seqs *s) { return (int64_t)s->max_pages * c->page_size; }

// The elements from the first to behind the last of such rows.
int64_t extent(const attn_cache *c, const attn_cache_seqs *s, int64_t sb, int64_t sh, int64_t room) {
  return (s->B - 1) * sb + (c->Hkv - 1) * sh + room;
}

int validate(const attn_cache *c, const attn_cache_seqs *s, const attn_cache_fwd_args *a) {
  const int e = validate(c, s);
  if (e != ATTN_OK) return e;
  if (!a || (a->dtype != ATTN_DTYPE_BF16 && a->dtype != ATTN_DTYPE_F32)) return ATTN_ERR_INVALID;
  if (a->Sq < 0 || a->Hq < 1 || a->Hq % c->Hkv != 0) return ATTN_ERR_INVALID;
  if (!isfinite(a->scale) || !isfinite(a->softcap) || a->softcap < 0.f) return ATTN_ERR_INVALID;
  if (a->softmax_type != ATTN_SOFTMAX_DEFAULT && a->softmax_type != ATTN_SOFTMAX_OFF_BY_ONE) return ATTN_ERR_INVALID;
  if (a->softmax_type == ATTN_SOFTMAX_OFF_BY_ONE && a->sink) return ATTN_ERR_INVALID;
  if ((a->weights == nullptr) != (a->weights_out == nullptr)) return ATTN_ERR_INVALID;
  if (!aligned4(a->weights) || !aligned4(a->weights_out) || !aligned4(a->sink)) return ATTN_ERR_INVALID;
  if (a->weights && (a->weights_stride_b < 0 || a->weights_stride_h < 0)) return ATTN_ERR_INVALID;
  if (s->B == 0 || a->Sq == 0) return ATTN_OK;
  if (a->weights && !rows_apart(c, s, a->weights_stride_b, a->weights_stride_h, table_room(c, s))) return ATTN_ERR_INVALID;
  if (!a->q || !aligned16(a->q)) return ATTN_ERR_INVALID;
  if (!strides_ok(a->dtype, {a->q_stride_b, a->q_stride_s, a->q_stride_h})) return ATTN_ERR_INVALID;
  const long long R = (long long)(a->Hq / c->Hkv) * a->Sq;
  // Positions of queries stay clear of 32 bits, the join's grid and the count of units
  // (64 keys, at the least, of a row tile of 8) within 31.
  if (a->Sq > (1 << 24) || R > INT_MAX / 2) return ATTN_ERR_UNSUPPORTED;
  const double units = (double)((R + 7) / 8) * s->B * c->Hkv * ((long long)s->max_pages * c->page_size / 64 + 1);
  if (units > INT_MAX) return ATTN_ERR_UNSUPPORTED;
  return ATTN_OK;
}

bool use_tc(const attn_cache *c, const attn_cache_seqs *s, const attn_cache_fwd_args *a) {
  return tc_supported_rows(a->dtype, c->D, (int)std::min((long long)INT_MAX, (long long)(a->Hq / c->Hkv) * a->Sq), s->B, c->Hkv);
}
bool use_mma(const attn_cache *c) { return mma_supported(c->D); }

struct FwdLayout {
  size_t prefix, o_part, ml_part, scores, total;
};

FwdParams fwd_params(const attn_cache *c, const attn_cache_seqs *s, const attn_cache_fwd_args *a, FwdLayout *L) {
  FwdParams p;
  memset(&p, 0, sizeof(p));
  p.c = view(c, s);
  p.Sq = a->Sq;
  p.Hq = a->Hq;
  p.G = a->Hq / c->Hkv;
  p.R = p.G * a->Sq;
  const bool tc = use_tc(c, s, a), mma = !tc && use_mma(c);
  p.row_tile = tc ? tc_row_tile() : mma ? mma_row_tile(a->dtype, c->D, p.R) : simt_row_tile();
  p.RT = (p.R + p.row_tile - 1) / p.row_tile;
  p.NG = s->B * p.RT;
  const long long cap = (long long)s->max_pages * c->page_size;
  p.unit_shift = tc ? tc_unit_shift() : mma ? mma_unit_shift(c->D) : simt_unit_shift();
  const long long most = std::max(1LL, (long long)p.NG * c->Hkv * ((cap >> p.unit_shift) + 1));
  p.max_ctas = (int)std::min(most, (mma ? mma_ctas_per_sm(c->D, p.row_tile) : 4LL) * device_sm_count());
  p.causal = a->causal ? 1 : 0;
  p.window = a->window > 0 ? std::min(a->window, 1 << 30) : 0;  // (no sequence is longer)
  p.cap = a->softcap;
  p.inv_cap = a->softcap > 0.f ? 1.f / a->softcap : 0.f;
  p.scale = a->scale;
  p.q = a->q;
  p.q_sb = a->q_stride_b;
  p.q_ss = a->q_stride_s;
  p.q_sh = a->q_stride_h;
  p.sink = a->sink;
  p.off_by_one = a->softmax_type == ATTN_SOFTMAX_OFF_BY_ONE ? 1 : 0;
  p.w_in = a->weights;
  p.w_out = a->weights_out;
  p.w_sb = a->weights_stride_b;
  p.w_sh = a->weights_stride_h;
  p.Lpad = (cap + 63) / 64 * 64;
  if (mma) p.cluster = mma_cluster(p);
  if (tc) p.splits = tc_splits(p);
  size_t off = 0;
  L->prefix = L->o_part = L->ml_part = 0;
  if (p.splits) {
    const size_t parts = p.splits > 1 ? (size_t)p.NG * c->Hkv * p.splits : 0;
    L->o_part = off; off += align_up(parts * p.row_tile * c->D * sizeof(float));
    L->ml_part = off; off += align_up(parts * p.row_tile * sizeof(float2));
  } else if (!p.cluster) {
    L->prefix = off; off += align_up(((size_t)p.NG + 1) * sizeof(int));
    L->o_part = off; off += align_up((size_t)2 * p.max_ctas * p.row_tile * c->D * sizeof(float));
    L->ml_part = off; off += align_up((size_t)2 * p.max_ctas * p.row_tile * sizeof(float2));
  }
  L->scores = off;
  if (a->weights) off += align_up((size_t)s->B * c->Hkv * p.R * p.Lpad * sizeof(float));
  L->total = std::max(off, kAlign);
  return p;
}

bool nothing(const attn_cache_seqs *s, const attn_cache_fwd_args *a) { return s->B == 0 || a->Sq == 0; }
int cuda_status(cudaError_t e) { return e == cudaSuccess ? ATTN_OK : ATTN_ERR_CUDA; }

}  // namespace
}  // namespace cache
}  // namespace attn

using namespace attn;
using namespace attn::cache;

extern "C" {

int attn_cache_append(const attn_cache *c, const attn_cache_seqs *s, const attn_cache_append_args *a,
                      attn_stream_t stream) {
  const int e = validate(c, s);
  if (e != ATTN_OK) return e;
  if (!a || (a->dtype != ATTN_DTYPE_BF16 && a->dtype != ATTN_DTYPE_F32) || a->S < 0) return ATTN_ERR_INVALID;
  if (s->B == 0) return ATTN_OK;
  if (!aligned4(a->counts) || !aligned4(a->lengths_out) || !aligned4(a->weights)) return ATTN_ERR_INVALID;
  if (a->lengths_out && a->lengths_out == s->lengths) return ATTN_ERR_INVALID;
  if (a->weights && (a->weights_stride_b < 0 || a->weights_stride_h < 0)) return ATTN_ERR_INVALID;
  if (a->weights && !rows_apart(c, s, a->weights_stride_b, a->weights_stride_h, table_room(c, s))) return ATTN_ERR_INVALID;
  if (a->S > 0) {
    if (!a->k || !a->v || !aligned16(a->k) || !aligned16(a->v)) return ATTN_ERR_INVALID;
    if (!strides_ok(a->dtype, {a->k_stride_b, a->k_stride_s, a->k_stride_h, a->v_stride_b, a->v_stride_s, a->v_stride_h}))
      return ATTN_ERR_INVALID;
  }
  AppendParams p;
  memset(&p, 0, sizeof(p));
  p.c = view(c, s);
  p.S = a->S;
  const long long span = std::max(1LL, ((long long)a->S + c->page_size - 2) / c->page_size + 1);
  p.span = (int)std::min(span, (long long)std::max(1, s->max_pages));
  if ((long long)p.span * s->B > INT_MAX) return ATTN_ERR_UNSUPPORTED;
  p.k = a->k; p.k_sb = a->k_stride_b; p.k_ss = a->k_stride_s; p.k_sh = a->k_stride_h;
  p.v = a->v; p.v_sb = a->v_stride_b; p.v_ss = a->v_stride_s; p.v_sh = a->v_stride_h;
  p.counts = a->counts;
  p.lengths_out = a->lengths_out;
  p.weights = a->weights;
  p.w_sb = a->weights_stride_b;
  p.w_sh = a->weights_stride_h;
  return cuda_status(launch_append(p, a->dtype, c->kind, reinterpret_cast<cudaStream_t>(stream)));
}

size_t attn_cache_fwd_workspace_size(const attn_cache *c, const attn_cache_seqs *s, const attn_cache_fwd_args *a) {
  if (validate(c, s, a) != ATTN_OK) return 0;
  if (nothing(s, a)) return kAlign;
  FwdLayout L;
  fwd_params(c, s, a, &L);
  return L.total;
}

const char *attn_cache_path_name(const attn_cache *c, const attn_cache_seqs *s, const attn_cache_fwd_args *a) {
  if (validate(c, s, a) != ATTN_OK) return "";
  return use_tc(c, s, a) ? "tc" : use_mma(c) ? "mma" : "simt";
}

int attn_cache_fwd(const attn_cache *c, const attn_cache_seqs *s, const attn_cache_fwd_args *a, void *O,
                   float *LSE, void *ws, size_t ws_bytes, attn_stream_t stream) {
  const int v = validate(c, s, a);
  if (v != ATTN_OK) return v;
  if (nothing(s, a)) return ATTN_OK;
  if (!O || !LSE || !aligned16(O) || !aligned4(LSE)) return ATTN_ERR_INVALID;
  FwdLayout L;
  FwdParams p = fwd_params(c, s, a, &L);
  if (!ws || ws_bytes < L.total || ((uintptr_t)ws % kAlign) != 0) return ATTN_ERR_WORKSPACE;
  char *w = static_cast<char *>(ws);
  p.prefix = reinterpret_cast<int *>(w + L.prefix);
  p.o_part = reinterpret_cast<float *>(w + L.o_part);
  p.ml_part = reinterpret_cast<float2 *>(w + L.ml_part);
  p.scores = a->weights ? reinterpret_cast<float *>(w + L.scores) : nullptr;
  p.O = O;
  p.LSE = LSE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = p.splits ? launch_fwd_tc(p, c->kind, st) : use_mma(c) ? launch_fwd_mma(p, a->dtype, c->kind, st) : launch_fwd_simt(p, a->dtype, c->kind, st);
  if (e == cudaSuccess && !p.cluster && p.splits != 1) e = launch_fwd_join(p, a->dtype, st);
  if (e == cudaSuccess && a->weights && s->max_pages > 0) e = launch_weights(p, st);
  return cuda_status(e);
}

int attn_cache_evict(const attn_cache *c, const attn_cache_seqs *s, const attn_cache_evict_args *a,
                     attn_stream_t stream) {
  const int e = validate(c, s);
  if (e != ATTN_OK) return e;
  if (!a || a->keep < 1 || a->first < 0 || a->recent < 0 || (long long)a->first + a->recent > a->keep) return ATTN_ERR_INVALID;
  if (a->keep > (1 << 30)) return ATTN_ERR_UNSUPPORTED;
  if (s->B == 0) return ATTN_OK;
  if (!a->weights || !a->table_out || !a->kept || !a->lengths_out || !a->weights_out) return ATTN_ERR_INVALID;
  if (!aligned4(a->weights) || !aligned4(a->table_out) || !aligned4(a->kept) || !aligned4(a->lengths_out) ||
      !aligned4(a->weights_out))
    return ATTN_ERR_INVALID;
  if (a->weights_stride_b < 0 || a->weights_stride_h < 0 || a->lengths_out == s->lengths) return ATTN_ERR_INVALID;
  const bool dense = a->weights_out_stride_b == 0 && a->weights_out_stride_h == 0;
  const int64_t wo_sh = dense ? a->keep : a->weights_out_stride_h, wo_sb = dense ? (int64_t)c->Hkv * a->keep : a->weights_out_stride_b;
  if (wo_sb < 0 || wo_sh < 0 || !rows_apart(c, s, wo_sb, wo_sh, a->keep)) return ATTN_ERR_INVALID;
  // The selection reads weights while it writes those that stay.
  const float *w0 = a->weights, *w1 = w0 + extent(c, s, a->weights_stride_b, a->weights_stride_h, table_room(c, s));
  const float *o0 = a->weights_out, *o1 = o0 + extent(c, s, wo_sb, wo_sh, a->keep);
  const bool in_place = w0 == o0 && wo_sb == a->weights_stride_b && wo_sh == a->weights_stride_h && a->keep >= table_room(c, s);
  if (w0 < o1 && o0 < w1 && !in_place) return ATTN_ERR_INVALID;  // (in place nothing moves where nothing can be evicted)
  EvictParams p;
  memset(&p, 0, sizeof(p));
  p.c = view(c, s);
  p.keep = a->keep;
  p.first = a->first;
  p.recent = a->recent;
  p.out_pages = (a->keep + c->page_size - 1) / c->page_size;
  if (a->table_out_stride < (s->B > 1 ? p.out_pages : 0)) return ATTN_ERR_INVALID;
  if ((long long)p.out_pages * s->B > INT_MAX) return ATTN_ERR_UNSUPPORTED;
  p.weights = a->weights;
  p.w_sb = a->weights_stride_b;
  p.w_sh = a->weights_stride_h;
  p.table_out = a->table_out;
  p.table_out_stride = a->table_out_stride;
  p.kept = a->kept;
  p.lengths_out = a->lengths_out;
  p.weights_out = a->weights_out;
  p.wo_sb = wo_sb;
  p.wo_sh = wo_sh;
  return cuda_status(launch_evict(p, c->kind, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
