// Rotary positions: the cos / sin table, and the norm of query and key heads with their
// rotation in one pass.
#include <cmath>

#include "rope.cuh"

namespace kvq {
namespace {

// ---- table -----------------------------------------------------------------------------
// Row p: a cos(p f_i), i < R/2, then a sin(p f_i), in double, rounded once to fp32.  A thread takes one pair
// over kSteps consecutive positions: the first angle and the step by sincos, the others by turning
// (four fused operations), which adds at most kSteps 2^-52 to the 2^-25 of the rounding.  Bound by the
// stores (4 R bytes a position).  131072 positions of 128: 15.3 us (4.4 TB/s stored), 71.8 with a sincos for each
// entry.
struct TableArgs {
  double freq[128];
  int half;
  double amplitude;
  int64_t pos0, n_pos;
  float* table;
};
constexpr int kSteps = 16;

__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ TableArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t p0 = i / a.half * kSteps;
  if (p0 >= a.n_pos) return;
  const int c = (int)(i % a.half);
  double s, k, ds, dk;
  sincos((double)(a.pos0 + p0) * a.freq[c], &s, &k);
  sincos(a.freq[c], &ds, &dk);
  float* row = a.table + p0 * 2 * a.half + c;
  const int n = (int)min((int64_t)kSteps, a.n_pos - p0);
  for (int j = 0; j < n; ++j) {
    row[0] = (float)(a.amplitude * k);
    row[a.half] = (float)(a.amplitude * s);
    row += 2 * a.half;
    const double t = fma(k, dk, -(s * ds));
    s = fma(s, dk, k * ds);
    k = t;
  }
}

// ---- norm and rotation -----------------------------------------------------------------
// LPR lanes (8, 16 or 32) hold one head row, an octet each; the mean square meets over them
// by shuffles, and the half-layout partner octet comes from its lane.  Bound by the rows read and written and
// the waits on those loads; two heads to a group and four CTAs per SM keep enough of them in flight.
struct NormArgs {
  HeadRows side[2];
  int D, dtype;
  int64_t n_tokens;
  float eps, offset, inv_d;
  RopeArgs rope;
  const int32_t* positions;
  int32_t* status;
};

// kHeads heads of one token and side per group of lanes: all their loads are issued first, and the token's
// cosines and sines are read once for them.
constexpr int kHeads = 2;

template <int LPR, int DT>
__global__ void __launch_bounds__(256, 4) norm_rope_kernel(const __grid_constant__ NormArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int cq = (a.side[0].heads + kHeads - 1) / kHeads, chunks = cq + (a.side[1].heads + kHeads - 1) / kHeads;
  const unsigned item = blockIdx.x * (256 / LPR) + threadIdx.x / LPR;   // the host keeps rows below 2^31
  const int o = threadIdx.x % LPR;
  const int64_t t = item / (unsigned)chunks;
  const int chunk = (int)(item - (unsigned)t * chunks), which = chunk >= cq;
  const HeadRows& S = a.side[which];
  const int h0 = (which ? chunk - cq : chunk) * kHeads;
  const bool live = t < a.n_tokens && 8 * o < a.D;
  const int n = live ? min(kHeads, S.heads - h0) : 0;
  float x[kHeads][8];
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[k][j] = 0.0f;
    if (k < n) load8(S.x, t * S.xt + (h0 + k) * S.xh + 8 * o, DT, x[k]);
  }
  const bool turns = a.rope.table && live && 8 * o < a.rope.rot;
  bool turned = turns;
  OctetTurn turn;
  if (turns) {
    const int64_t pos = a.positions ? a.positions[t] : t;
    if (pos < 0 || pos >= a.rope.n_pos) {
      flag(a.status, KVQ_DEV_BOUNDS);
      turned = false;
    } else {
      rope_load(a.rope, pos, o, turn);
    }
  }
  float w[8];
  if (S.weight) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 0.0f;
    if (live) load8(S.weight, 8 * o, DT, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] += a.offset;
  }
  const int po = rope_partner(a.rope, o);
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kHeads; ++k) {
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[k][j], x[k][j], ss);
    if (!(ss <= 3.402823466e38f)) {   // a NaN or Inf among them, or squares that overflow
#pragma unroll
      for (int j = 0; j < 8; ++j) bad |= !isfinite(x[k][j]);
    }
#pragma unroll
    for (int m = 1; m < LPR; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    if (S.weight) {   // alike over the lanes of a row; rows of one warp may differ
      float eps = a.eps, r = fmaf(ss, a.inv_d, eps);
      // Squares outside fp32's range: the row is taken 2^70 times smaller or 2^100 times larger (below 2^-41 all of
      // it then, up to 2^59 and down to the smallest subnormal's 2^-49), eps by the square of that.
      const bool big = !(ss <= 0x1p126f), small = r < 0x1p-90f;
      if (big || small) {
        const float by = big ? 0x1p-70f : 0x1p100f;
        eps *= by;
        eps *= by;
        ss = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          x[k][j] *= by;
          ss = fmaf(x[k][j], x[k][j], ss);
        }
        const unsigned row = LPR == 32 ? 0xffffffffu : ((1u << (LPR & 31)) - 1u) << (threadIdx.x & 31 & ~(LPR - 1));
#pragma unroll
        for (int m = 1; m < LPR; m <<= 1) ss += __shfl_xor_sync(row, ss, m);
        r = fmaf(ss, a.inv_d, eps);
      }
      r = rsqrtf(r);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[k][j] = x[k][j] * w[j] * r;
    }
    if (a.rope.table) {
      float p[8];
      if (!a.rope.inter) {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = __shfl_sync(0xffffffffu, x[k][j], po, LPR);
      }
      if (turned) rope_turn(a.rope, o, turn, x[k], p);
    }
    if (k < n) store8(S.y, t * S.yt + (h0 + k) * S.yh + 8 * o, DT, x[k]);
  }
  if (bad) flag(a.status, KVQ_DEV_NONFINITE);
}

template <int LPR>
cudaError_t launch_norm_rope_t(const NormArgs& a, cudaStream_t s) {
  const int chunks = (a.side[0].heads + kHeads - 1) / kHeads + (a.side[1].heads + kHeads - 1) / kHeads;
  const int64_t items = a.n_tokens * chunks;
  const unsigned grid = (unsigned)((items + 256 / LPR - 1) / (256 / LPR));
  auto kern = a.dtype == KVQ_F32   ? norm_rope_kernel<LPR, KVQ_F32>
              : a.dtype == KVQ_F16 ? norm_rope_kernel<LPR, KVQ_F16>
                                   : norm_rope_kernel<LPR, KVQ_BF16>;
  return launch_pdl(kern, dim3(grid), dim3(256), 0, s, a);
}

}  // namespace

cudaError_t launch_rope_table(const double* freq, int half, double amplitude, int64_t pos0, int64_t n_pos,
                              float* table, cudaStream_t s) {
  TableArgs a;
  for (int i = 0; i < 128; ++i) a.freq[i] = i < half ? freq[i] : 0.0;
  a.half = half;
  a.amplitude = amplitude;
  a.pos0 = pos0;
  a.n_pos = n_pos;
  a.table = table;
  const int64_t threads = (n_pos + kSteps - 1) / kSteps * half;
  return launch_pdl(rope_table_kernel, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, s, a);
}

cudaError_t launch_norm_rope(int D, int dtype, int64_t n_tokens, const HeadRows& q, const HeadRows& k, float eps,
                             float weight_offset, const RopeArgs& rope, const int32_t* positions, int32_t* d_status,
                             cudaStream_t s) {
  NormArgs a;
  a.side[0] = q;
  a.side[1] = k;
  a.D = D;
  a.dtype = dtype;
  a.n_tokens = n_tokens;
  a.eps = eps;
  a.offset = weight_offset;
  a.inv_d = 1.0f / (float)D;
  a.rope = rope;
  a.positions = positions;
  a.status = d_status;
  return D <= 64 ? launch_norm_rope_t<8>(a, s) : D <= 128 ? launch_norm_rope_t<16>(a, s) : launch_norm_rope_t<32>(a, s);
}

}  // namespace kvq
