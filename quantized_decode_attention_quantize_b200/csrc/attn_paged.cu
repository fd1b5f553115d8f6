// Attention of several new tokens per sequence over the paged cache (D = 128, groups of 128
// tokens, 4-bit per-channel keys, 2-bit per-token values, raw sink and window rows).
//
// One warp per (query row, query head): lane l holds channels 4 l .. 4 l + 3, walks the
// visible tokens one by one with an online softmax in the log2 domain, all in fp32.
#include "kvq_internal.cuh"
#include "wht.cuh"

namespace kvq {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

struct AttnSeq {
  int64_t row0;
  int n, tq, tr;
  bool ok;
};

__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int s) {
  const PagedBatch& b = a.b;
  AttnSeq q;
  const int64_t lo = b.cu[s], hi = b.cu[s + 1];
  q.tq = b.t_quant[s];
  q.tr = b.t_res[s];
  q.row0 = lo;
  q.ok = lo >= 0 && hi >= lo && hi <= b.n_rows && hi - lo <= b.max_rows && q.tq >= 0 && q.tq <= a.max_t_quant &&
         q.tr <= a.max_t_res && q.tr >= -b.n_sink && (q.tr >= 0 || q.tq == 0);
  q.n = q.ok ? (int)(hi - lo) : 0;
  return q;
}

__device__ __forceinline__ void quad(const void* base, int64_t i, int dtype, float (&x)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = load_elem(base, i + j, dtype);
}

__device__ __forceinline__ int raw_flags(float x) {
  return !isfinite(x) ? KVQ_DEV_NONFINITE : fabsf(x) > 65504.0f ? KVQ_DEV_RANGE : 0;
}

__global__ void __launch_bounds__(128) attn_paged_kernel(const __grid_constant__ AttnArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const PagedBatch& b = a.b;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int s = blockIdx.y, ns = b.n_sink;
  const AttnSeq q = attn_seq(a, s);
  if (!q.ok) {
    if (threadIdx.x == 0 && blockIdx.x == 0) flag(a.status, KVQ_DEV_BOUNDS);
    return;
  }
  int flags = 0;
  for (int64_t w = (int64_t)blockIdx.x * 4 + warp; w < (int64_t)q.n * a.Hq; w += (int64_t)gridDim.x * 4) {
    const int i = (int)(w / a.Hq), hq = (int)(w % a.Hq), h = hq / a.G;
    const int64_t qrow = (q.row0 + i) * a.Hq + hq;
    float qv[4], qr[4], o[4] = {0, 0, 0, 0};
    quad(a.q, qrow * 128 + 4 * lane, a.q_dtype, qv);
    bool bad = false;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bad |= !isfinite(qv[j]);
      qr[j] = qv[j];
    }
    if (bad) flags |= KVQ_DEV_NONFINITE;
    if (a.L.k_rotate) {
      wht128_quad_unscaled(qr, lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) qr[j] *= a.L.rot_scale;
    }
    const int64_t L = (int64_t)ns + q.tq + q.tr;
    const int64_t seen = a.causal ? max((int64_t)0, L - q.n + i + 1) : L;   // visible tokens
    float m = -INFINITY, l = 0.0f;
    auto step = [&](float d, const float (&v)[4]) {
#pragma unroll
      for (int e = 16; e > 0; e >>= 1) d += __shfl_xor_sync(0xffffffffu, d, e);
      d *= a.qscale;
      const float mn = fmaxf(m, d), c = exp2f(m - mn), p = exp2f(d - mn);
      m = mn;
      l = l * c + p;
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = fmaf(p, v[j], o[j] * c);
    };
    const int64_t slab = (int64_t)s * a.L.Hkv + h;
    auto raw = [&](const void* kb, const void* vb, int64_t rows, int64_t cap) {
      for (int64_t r = 0; r < rows; ++r) {
        const int64_t e = (slab * cap + r) * 128 + 4 * lane;
        float k[4], v[4];
        quad(kb, e, a.L.src_dtype, k);
        quad(vb, e, a.L.src_dtype, v);
#pragma unroll
        for (int j = 0; j < 4; ++j) {   // what the format cannot hold counts as 0
          flags |= raw_flags(k[j]) | raw_flags(v[j]);
          if (raw_flags(k[j])) k[j] = 0.0f;
          if (raw_flags(v[j])) v[j] = 0.0f;
        }
        step(qv[0] * k[0] + qv[1] * k[1] + qv[2] * k[2] + qv[3] * k[3], v);
      }
    };
    raw(a.sink[0], a.sink[1], min(seen, (int64_t)ns), ns);
    const int packed = (int)min(max(seen - ns, (int64_t)0), (int64_t)q.tq);
    for (int g = 0; 128 * g < packed; ++g) {
      int blk = b.table[(int64_t)s * b.max_blocks + g];
      if (blk < 0 || blk >= b.num_blocks) {
        flags |= KVQ_DEV_BOUNDS;
        blk = 0;
      }
      const int64_t ps = (int64_t)blk * a.L.Hkv + h;
      const uint8_t* kc = reinterpret_cast<const uint8_t*>(a.L.side[0].codes) + ps * a.L.side[0].code_slab_bytes;
      const uint8_t* vc = reinterpret_cast<const uint8_t*>(a.L.side[1].codes) + ps * a.L.side[1].code_slab_bytes;
      float ks[4], kz[4];
      quad(a.L.side[0].scale, ps * 128 + 4 * lane, KVQ_F16, ks);
      quad(a.L.side[0].zero, ps * 128 + 4 * lane, KVQ_F16, kz);
      const int rows = min(128, packed - 128 * g);
      for (int r = 0; r < rows; ++r) {
        const uint32_t kw = reinterpret_cast<const uint16_t*>(kc + r * 64)[lane];
        // pair layout: channels 8 w .. of token 2u in the low half of word w, of 2u + 1 in the high
        const uint32_t vw = reinterpret_cast<const uint8_t*>(vc)[(r >> 1) * 64 + (lane >> 1) * 4 + 2 * (r & 1) + (lane & 1)];
        const float vs = load_elem(a.L.side[1].scale, ps * 128 + r, KVQ_F16);
        const float vz = load_elem(a.L.side[1].zero, ps * 128 + r, KVQ_F16);
        float d = 0.0f, v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          d = fmaf(qr[j], fmaf((float)((kw >> (4 * j)) & 15u), ks[j], kz[j]), d);
          v[j] = fmaf((float)((vw >> (2 * j)) & 3u), vs, vz);
        }
        step(d, v);
      }
    }
    raw(a.res[0], a.res[1], min(max(seen - ns - q.tq, (int64_t)0), (int64_t)max(q.tr, 0)), b.res_cap);
#pragma unroll
    for (int j = 0; j < 4; ++j) store_elem(a.out, qrow * 128 + 4 * lane + j, a.out_dtype, l > 0.0f ? o[j] / l : 0.0f);
    if (a.lse && lane == 0) a.lse[qrow] = l > 0.0f ? kLn2 * (m + log2f(l)) : -INFINITY;
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (flags && lane == 0) flag(a.status, flags);
}

}  // namespace

size_t attn_paged_workspace(int num_seqs, int Hq, int Hkv, int64_t n_rows, int64_t max_new, int64_t max_t_quant,
                            int max_t_res, int n_sink) {
  return 16;
}

cudaError_t launch_attn_paged(const AttnArgs& a, cudaStream_t s) {
  const int64_t want = (a.b.max_rows * a.Hq + 3) / 4;
  return launch_pdl(attn_paged_kernel, dim3((unsigned)(want < 4096 ? want : 4096), a.b.num_seqs), dim3(128), 0, s, a);
}

}  // namespace kvq
