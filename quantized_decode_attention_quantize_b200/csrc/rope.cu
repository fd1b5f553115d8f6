// Rotary positions: the cos / sin table, and the norm of query and key heads with their
// rotation in one pass.
#include <cmath>

#include "rope.cuh"

namespace kvq {
namespace {

// ---- table -----------------------------------------------------------------------------
// Row p: a cos(p f_i), i < R/2, then a sin(p f_i), in double, rounded once to fp32.
struct TableArgs {
  double freq[128];
  int half;
  double amplitude;
  int64_t pos0, n_pos;
  float* table;
};

__global__ void __launch_bounds__(256) rope_table_kernel(const __grid_constant__ TableArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= a.n_pos * a.half) return;
  const int64_t p = i / a.half;
  const int c = (int)(i % a.half);
  double s, k;
  sincos((double)(a.pos0 + p) * a.freq[c], &s, &k);
  float* row = a.table + p * 2 * a.half;
  row[c] = (float)(a.amplitude * k);
  row[a.half + c] = (float)(a.amplitude * s);
}

// ---- norm and rotation -----------------------------------------------------------------
// LPR lanes (8, 16 or 32) hold one head row, an octet each; the mean square meets over them
// by shuffles, and the half-layout partner octet comes from its lane.
struct NormArgs {
  HeadRows side[2];
  int D, dtype;
  int64_t n_tokens;
  float eps, offset;
  RopeArgs rope;
  const int32_t* positions;
  int32_t* status;
};

template <int LPR>
__global__ void __launch_bounds__(256) norm_rope_kernel(NormArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int heads = a.side[0].heads + a.side[1].heads;
  const int64_t row = (int64_t)blockIdx.x * (256 / LPR) + threadIdx.x / LPR;
  const int o = threadIdx.x % LPR;
  const bool live = row < a.n_tokens * heads && 8 * o < a.D;
  const int64_t t = live ? row / heads : 0;
  int h = live ? (int)(row % heads) : 0;
  const int which = h >= a.side[0].heads;
  const HeadRows& S = a.side[which];
  if (which) h -= a.side[0].heads;
  float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (live) load8(S.x, t * S.xt + h * S.xh + 8 * o, a.dtype, x);
  float fin = 0.0f, ss = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    fin = fmaf(x[j], 0.0f, fin);
    ss = fmaf(x[j], x[j], ss);
  }
  if (live && !(fin == 0.0f)) flag(a.status, KVQ_DEV_NONFINITE);
#pragma unroll
  for (int m = 1; m < LPR; m <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
  if (S.weight && live) {
    const float r = 1.0f / sqrtf(ss / (float)a.D + a.eps);
    float w[8];
    load8(S.weight, 8 * o, a.dtype, w);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = x[j] * r * (a.offset + w[j]);
  }
  if (a.rope.table) {
    const int po = rope_partner(a.rope, o);
    float p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) p[j] = __shfl_sync(0xffffffffu, x[j], po, LPR);
    if (live && 8 * o < a.rope.rot) {
      const int64_t pos = a.positions ? a.positions[t] : t;
      if (pos < 0 || pos >= a.rope.n_pos) {
        flag(a.status, KVQ_DEV_BOUNDS);
      } else {
        OctetTurn turn;
        rope_load(a.rope, pos, o, turn);
        rope_turn(a.rope, o, turn, x, p);
      }
    }
  }
  if (live) store8(S.y, t * S.yt + h * S.yh + 8 * o, a.dtype, x);
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
  return launch_pdl(rope_table_kernel, dim3((unsigned)((n_pos * half + 255) / 256)), dim3(256), 0, s, a);
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
  a.rope = rope;
  a.positions = positions;
  a.status = d_status;
  const int64_t rows = n_tokens * (q.heads + k.heads);
  const int lpr = D <= 64 ? 8 : D <= 128 ? 16 : 32;
  const unsigned grid = (unsigned)((rows + 256 / lpr - 1) / (256 / lpr));
  auto kern = lpr == 8 ? norm_rope_kernel<8> : lpr == 16 ? norm_rope_kernel<16> : norm_rope_kernel<32>;
  return launch_pdl(kern, dim3(grid), dim3(256), 0, s, a);
}

}  // namespace kvq
