// Host layer of the serving entry points around the paged cache: argument validation and
// dispatch.  No allocation, no synchronisation, no state.
#include <cmath>

#include "kvq_internal.cuh"

using namespace kvq;

namespace {

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool valid_dtype(int dt) { return dt == KVQ_F32 || dt == KVQ_F16 || dt == KVQ_BF16; }
int64_t dtype_bytes(int dt) { return dt == KVQ_F32 ? 4 : 2; }
kvq_status launched(cudaError_t e) { return e == cudaSuccess ? KVQ_OK : KVQ_ERR_CUDA; }

// A device array of int32 that must be there.
bool ints(const void* p) { return p && aligned(p, 4); }

// Two arrays of n int32 that share a place.
bool overlap(const int32_t* p, const int32_t* q, int64_t n) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return (a < b ? b - a : a - b) < (uintptr_t)n * 4;
}

kvq_status rope_args(const kvq_rope* r, int D, RopeArgs* out) {
  out->table = nullptr;
  out->n_pos = 0;
  out->rot = out->inter = 0;
  if (!r) return KVQ_OK;
  if (!r->table || !aligned(r->table, 16) || r->n_pos < 1 || r->n_pos > ((int64_t)1 << 31)) return KVQ_ERR_INVALID;
  if (r->rot_dim < 16 || r->rot_dim % 16 || r->rot_dim > D) return KVQ_ERR_INVALID;
  if (r->interleaved != 0 && r->interleaved != 1) return KVQ_ERR_INVALID;
  out->table = r->table;
  out->n_pos = r->n_pos;
  out->rot = r->rot_dim;
  out->inter = r->interleaved;
  return KVQ_OK;
}

// Row strides of [row][head][D] rows.
bool row_strides(int64_t st, int64_t sh, int64_t eb) {
  return st >= 0 && sh >= 0 && (st * eb) % 16 == 0 && (sh * eb) % 16 == 0;
}

// The paged format these entry points take (q heads per KV head apart).
bool paged_format(const kvq_format* f) {
  return f->head_dim == 128 && f->group_tokens == 128 && f->k_scheme == KVQ_ASYM && f->k_bits == 4 &&
         f->v_scheme == KVQ_ASYM && f->v_bits == 2 && f->rope == 0;
}

constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr size_t kMaxTiles = (size_t)4 << 30;   // expanded pages that a workspace is sized for

// Checks shared by the calls over a paged cache, and its device-side numbers.
kvq_status paged_batch(const kvq_format* f, const kvq_paged_cache* pc, const int32_t* cu, int64_t n_rows,
                       int64_t max_rows, const int32_t* t_quant, const int32_t* t_res, int32_t* d_status, Layout* L,
                       PagedBatch* b) {
  const kvq_status s = paged_layout(f, pc, L);
  if (s != KVQ_OK) return s;
  if (!paged_format(f)) return KVQ_ERR_UNSUPPORTED;
  if (n_rows < 0 || n_rows > kMaxRows || max_rows < 0 || max_rows > n_rows) return KVQ_ERR_INVALID;
  if (!ints(cu) || !ints(t_quant) || !ints(t_res) || !aligned(d_status, 4)) return KVQ_ERR_INVALID;
  if (pc->max_blocks >= (1 << 24)) return KVQ_ERR_UNSUPPORTED;
  if (L->Hkv > 32767 || pc->num_seqs > 65535) return KVQ_ERR_UNSUPPORTED;
  if (L->n_sink && (!pc->sink_k || !pc->sink_v || !aligned(pc->sink_k, 16) || !aligned(pc->sink_v, 16)))
    return KVQ_ERR_INVALID;
  if (L->res_cap && (!pc->res_k || !pc->res_v || !aligned(pc->res_k, 16) || !aligned(pc->res_v, 16)))
    return KVQ_ERR_INVALID;
  b->cu = cu;
  b->t_quant = t_quant;
  b->t_res = t_res;
  b->table = pc->block_table;
  b->num_seqs = pc->num_seqs;
  b->max_blocks = pc->max_blocks;
  b->num_blocks = L->B;
  b->n_sink = L->n_sink;
  b->res_cap = L->res_cap;
  b->n_rows = n_rows;
  b->max_rows = max_rows;
  return KVQ_OK;
}

}  // namespace

extern "C" {

kvq_status kvq_rope_table(const kvq_rope_spec* p, int64_t pos0, int64_t n_pos, float* table, void* stream) {
  if (!p || p->rot_dim < 16 || p->rot_dim > 256 || p->rot_dim % 16) return KVQ_ERR_INVALID;
  if (p->scaling < KVQ_ROPE_PLAIN || p->scaling > KVQ_ROPE_RAMP) return KVQ_ERR_INVALID;
  if (!(p->base > 1.0) || !std::isfinite(p->base) || !(p->amplitude > 0.0) || !std::isfinite(p->amplitude))
    return KVQ_ERR_INVALID;
  const bool scaled = p->scaling != KVQ_ROPE_PLAIN;
  const bool bounded = p->scaling == KVQ_ROPE_BANDS || p->scaling == KVQ_ROPE_RAMP;
  if (scaled && (!(p->factor > 0.0) || !std::isfinite(p->factor))) return KVQ_ERR_INVALID;
  if (bounded && (!(p->original_len > 0.0) || !std::isfinite(p->original_len) || !(p->low > 0.0) ||
                  !(p->high > p->low) || !std::isfinite(p->high)))
    return KVQ_ERR_INVALID;
  if (pos0 < 0 || n_pos < 0 || pos0 > ((int64_t)1 << 31) || n_pos > ((int64_t)1 << 31) - pos0)
    return KVQ_ERR_INVALID;
  if (n_pos == 0) return KVQ_OK;
  if (!table || !aligned(table, 16)) return KVQ_ERR_INVALID;
  const int R = p->rot_dim, half = R / 2;
  const double two_pi = 6.283185307179586476925286766559;
  double a = 0.0, z = 0.0;
  if (p->scaling == KVQ_ROPE_RAMP) {
    auto turns_at = [&](double b) { return R * std::log(p->original_len / (two_pi * b)) / (2.0 * std::log(p->base)); };
    a = std::fmax(std::floor(turns_at(p->high)), 0.0);
    z = std::fmin(std::ceil(turns_at(p->low)), R - 1.0);
  }
  double f[128];
  for (int i = 0; i < half; ++i) {
    const double w = std::pow(p->base, -2.0 * i / R);
    double g;
    switch (p->scaling) {
      case KVQ_ROPE_LINEAR: f[i] = w / p->factor; break;
      case KVQ_ROPE_BANDS:
        g = std::fmin(std::fmax((p->original_len * w / two_pi - p->low) / (p->high - p->low), 0.0), 1.0);
        f[i] = (1.0 - g) * w / p->factor + g * w;
        break;
      case KVQ_ROPE_RAMP:
        g = std::fmin(std::fmax((i - a) / std::fmax(z - a, 0.001), 0.0), 1.0);
        f[i] = (1.0 - g) * w + g * w / p->factor;
        break;
      default: f[i] = w;
    }
    if (!std::isfinite(f[i])) return KVQ_ERR_INVALID;   // a base or factor beyond what double carries
  }
  return launched(launch_rope_table(f, half, p->amplitude, pos0, n_pos, table, reinterpret_cast<cudaStream_t>(stream)));
}

kvq_status kvq_norm_rope(int32_t D, int32_t dtype, int64_t n, const kvq_head_rows* q, const kvq_head_rows* k,
                         float eps, float offset, const kvq_rope* rope, const int32_t* positions, int32_t* d_status,
                         void* stream) {
  if (D < 16 || D > 256 || D % 16 || !valid_dtype(dtype) || n < 0 || n > kMaxRows || !q) return KVQ_ERR_INVALID;
  RopeArgs r;
  const kvq_status s = rope_args(rope, D, &r);
  if (s != KVQ_OK) return s;
  if ((positions && !aligned(positions, 4)) || !aligned(d_status, 4)) return KVQ_ERR_INVALID;
  const int64_t eb = dtype_bytes(dtype);
  HeadRows side[2] = {};
  int64_t heads = 0;
  const kvq_head_rows* in[2] = {q, k};
  for (int w = 0; w < 2; ++w) {
    if (!in[w]) continue;
    const kvq_head_rows& x = *in[w];
    if (x.heads < 1 || x.heads > 65536 || !row_strides(x.x_stride_t, x.x_stride_h, eb) ||
        !row_strides(x.y_stride_t, x.y_stride_h, eb))
      return KVQ_ERR_INVALID;
    if (n && (!x.x || !x.y || !aligned(x.x, 16) || !aligned(x.y, 16))) return KVQ_ERR_INVALID;
    if (x.weight && (!aligned(x.weight, 16) || !(eps >= 0.0f) || !std::isfinite(eps) || !std::isfinite(offset)))
      return KVQ_ERR_INVALID;
    // in place means the same rows; rows of the output must not run into one another
    if (x.x == x.y && (x.x_stride_t != x.y_stride_t || x.x_stride_h != x.y_stride_h)) return KVQ_ERR_INVALID;
    if ((n > 1 && x.y_stride_t < D) || (x.heads > 1 && x.y_stride_h < D)) return KVQ_ERR_INVALID;
    side[w] = HeadRows{x.x, x.y, x.x_stride_t, x.x_stride_h, x.y_stride_t, x.y_stride_h, x.heads, x.weight};
    heads += x.heads;
  }
  if (n * heads > ((int64_t)1 << 31)) return KVQ_ERR_UNSUPPORTED;
  if (n == 0) return KVQ_OK;
  return launched(launch_norm_rope(D, dtype, n, side[0], side[1], eps, offset, r, positions, d_status,
                                   reinterpret_cast<cudaStream_t>(stream)));
}

kvq_status kvq_append_paged(const kvq_format* f, const kvq_paged_cache* pc, const int32_t* cu, int64_t n_rows,
                            int64_t max_new, const int32_t* t_quant, const int32_t* t_res, const void* k_src,
                            int64_t k_st, int64_t k_sh, const void* v_src, int64_t v_st, int64_t v_sh,
                            const kvq_rope* rope, const int32_t* positions, int32_t* tq_out, int32_t* tr_out,
                            int32_t* d_status, void* stream) {
  AppendArgs a;
  kvq_status s = paged_batch(f, pc, cu, n_rows, max_new, t_quant, t_res, d_status, &a.L, &a.b);
  if (s != KVQ_OK) return s;
  if (a.L.res_cap < 128 || a.L.res_cap % 128) return KVQ_ERR_UNSUPPORTED;
  s = rope_args(rope, a.L.D, &a.rope);
  if (s != KVQ_OK) return s;
  if (positions && !aligned(positions, 4)) return KVQ_ERR_INVALID;
  if (!ints(tq_out) || !ints(tr_out)) return KVQ_ERR_INVALID;
  // other CTAs still read the lengths when the first ones write theirs
  const int64_t seqs = pc->num_seqs;
  if (overlap(tq_out, tr_out, seqs) || overlap(tq_out, t_quant, seqs) || overlap(tq_out, t_res, seqs) ||
      overlap(tr_out, t_quant, seqs) || overlap(tr_out, t_res, seqs))
    return KVQ_ERR_INVALID;
  const int64_t eb = dtype_bytes(a.L.src_dtype);
  if (!row_strides(k_st, k_sh, eb) || !row_strides(v_st, v_sh, eb)) return KVQ_ERR_INVALID;
  if (n_rows && (!k_src || !v_src || !aligned(k_src, 16) || !aligned(v_src, 16))) return KVQ_ERR_INVALID;
  a.src[0] = k_src;
  a.src[1] = v_src;
  a.st[0] = k_st;
  a.st[1] = v_st;
  a.sh[0] = k_sh;
  a.sh[1] = v_sh;
  a.positions = positions;
  a.t_quant_out = tq_out;
  a.t_res_out = tr_out;
  a.sink[0] = pc->sink_k;
  a.sink[1] = pc->sink_v;
  a.res[0] = pc->res_k;
  a.res[1] = pc->res_v;
  a.status = d_status;
  return launched(launch_append_paged(a, reinterpret_cast<cudaStream_t>(stream)));
}

kvq_status kvq_read_paged(const kvq_format* f, const kvq_paged_cache* pc, const int32_t* cu, int64_t n_rows,
                          int64_t max_rows, const int32_t* first, const int32_t* t_quant, const int32_t* t_res,
                          void* k_out, void* v_out, int32_t out_dtype, int32_t* d_status, void* stream) {
  ReadArgs a;
  const kvq_status s = paged_batch(f, pc, cu, n_rows, max_rows, t_quant, t_res, d_status, &a.L, &a.b);
  if (s != KVQ_OK) return s;
  if (!ints(first) || !valid_dtype(out_dtype) || !aligned(k_out, 16) || !aligned(v_out, 16)) return KVQ_ERR_INVALID;
  if (n_rows == 0) return KVQ_OK;
  if (!k_out && !v_out) return KVQ_ERR_INVALID;
  a.first = first;
  a.out[0] = k_out;
  a.out[1] = v_out;
  a.out_dtype = out_dtype;
  a.sink[0] = pc->sink_k;
  a.sink[1] = pc->sink_v;
  a.res[0] = pc->res_k;
  a.res[1] = pc->res_v;
  a.status = d_status;
  return launched(launch_read_paged(a, reinterpret_cast<cudaStream_t>(stream)));
}

static kvq_status attn_sizes(const kvq_format* f, int32_t num_seqs, int32_t Hq, int32_t Hkv, int64_t n_rows,
                             int64_t max_new, int64_t max_tq, int32_t max_tr) {
  const kvq_status s = kvq_format_check(f);
  if (s != KVQ_OK) return s;
  if (num_seqs < 1 || Hkv < 1 || Hq < 1 || Hq % Hkv) return KVQ_ERR_INVALID;
  if (n_rows < 0 || n_rows > kMaxRows || max_new < 0 || max_new > n_rows) return KVQ_ERR_INVALID;
  if (max_tq < 0 || max_tr < 0 || max_tr > f->residual_cap) return KVQ_ERR_INVALID;
  if (!paged_format(f) || Hq / Hkv > 16 || Hkv > 32767 || num_seqs > 65535 || n_rows * Hq >= (int64_t)1 << 31 ||
      max_tq >= (int64_t)1 << 30)
    return KVQ_ERR_UNSUPPORTED;
  return KVQ_OK;
}

size_t kvq_attention_paged_workspace_bytes(const kvq_format* f, int32_t num_seqs, int32_t Hq, int32_t Hkv,
                                           int64_t n_rows, int64_t max_new, int64_t max_tq, int32_t max_tr) {
  if (attn_sizes(f, num_seqs, Hq, Hkv, n_rows, max_new, max_tq, max_tr) != KVQ_OK) return 0;
  size_t n = attn_paged_workspace_upto(Hq / Hkv, max_new);
  if (attn_wide_pays(num_seqs, Hq / Hkv, n_rows)) {
    const size_t tiles = attn_wide_tiles(num_seqs, Hkv, max_tq, max_tr, f->n_sink);
    if (tiles <= kMaxTiles) n += tiles;
  }
  return n;
}

kvq_status kvq_attention_paged(const kvq_format* f, const kvq_paged_cache* pc, const int32_t* cu, int64_t n_rows,
                               int64_t max_new, const int32_t* t_quant, const int32_t* t_res, int64_t max_tq,
                               int32_t max_tr, const void* q, int32_t q_dtype, int32_t Hq, float scale,
                               int32_t causal, void* out, int32_t out_dtype, float* lse, void* ws, size_t ws_bytes,
                               int32_t* d_status, void* stream) {
  AttnArgs a;
  kvq_status s = paged_batch(f, pc, cu, n_rows, max_new, t_quant, t_res, d_status, &a.L, &a.b);
  if (s != KVQ_OK) return s;
  s = attn_sizes(f, pc->num_seqs, Hq, a.L.Hkv, n_rows, max_new, max_tq, max_tr);
  if (s != KVQ_OK) return s;
  if (max_tq > (int64_t)pc->max_blocks * 128) return KVQ_ERR_INVALID;
  if (!valid_dtype(q_dtype) || !valid_dtype(out_dtype) || !(scale > 0.0f) || !std::isfinite(scale))
    return KVQ_ERR_INVALID;
  if (causal != 0 && causal != 1) return KVQ_ERR_INVALID;
  if (!aligned(lse, 4)) return KVQ_ERR_INVALID;
  if (n_rows && (!q || !out || !aligned(q, 16) || !aligned(out, 16))) return KVQ_ERR_INVALID;
  if (!ws || !aligned(ws, 16)) return KVQ_ERR_INVALID;
  if (ws_bytes < attn_paged_workspace(Hq / a.L.Hkv, max_new)) return KVQ_ERR_WORKSPACE;
  if (n_rows == 0 || max_new == 0) return KVQ_OK;
  a.max_t_quant = max_tq;
  a.max_t_res = max_tr;
  a.q = q;
  a.q_dtype = q_dtype;
  a.Hq = Hq;
  a.G = Hq / a.L.Hkv;
  a.qscale = scale * 1.4426950408889634f;
  a.causal = causal;
  a.out = out;
  a.out_dtype = out_dtype;
  a.lse = lse;
  a.ws = ws;
  a.ws_bytes = ws_bytes;
  a.sink[0] = pc->sink_k;
  a.sink[1] = pc->sink_v;
  a.res[0] = pc->res_k;
  a.res[1] = pc->res_v;
  a.status = d_status;
  return launched(launch_attn_paged(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
