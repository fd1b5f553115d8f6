// The ragged append of new tokens to a paged cache (rotation and packing on the way) and
// the read-back of cached tokens.  D = 128, groups of 128 tokens, 4-bit per-channel keys and
// 2-bit per-token values.
//
// Both run on a flat grid of units, the pieces of work of all sequences end to end: a CTA
// finds the sequence of its unit from the ragged batch's own numbers, so a batch of one long
// and many short sequences costs no empty CTAs beyond the bound's slack.
#include "paged_batch.cuh"
#include "rope.cuh"
#include "wht.cuh"

namespace kvq {
namespace {

constexpr int kThreads = 256;

// One sequence of an append as its device-side numbers give it.
struct AppendSeq {
  int64_t row0;       // its first new row
  int n, tq, tr;      // new tokens, packed and window tokens before the call
  int to_sink;        // new tokens that go to the sink
  int old;            // window rows in use (tr >= 0)
  int total;          // window rows and new tokens behind the sink
  int groups;         // whole groups packed by this call
  int units;          // CTAs of each (kv head, keys | values)
  bool ok;
};

__device__ __forceinline__ AppendSeq append_seq(const PagedBatch& b, int s) {
  AppendSeq q;
  const int64_t lo = b.cu[s], hi = b.cu[s + 1];
  q.tq = b.t_quant[s];
  q.tr = b.t_res[s];
  q.row0 = lo;
  q.ok = lo >= 0 && hi >= lo && hi <= b.n_rows && hi - lo <= b.max_rows && q.tq >= 0 && q.tq % 128 == 0 &&
         q.tr <= b.res_cap && q.tr >= -b.n_sink && (q.tr >= 0 || q.tq == 0);
  q.n = q.ok ? (int)(hi - lo) : 0;
  q.to_sink = q.tr < 0 ? min(q.n, -q.tr) : 0;
  q.old = max(q.tr, 0);
  // a sink that stays short of full leaves nothing behind it
  q.total = q.ok ? q.old + q.n - q.to_sink : 0;
  q.groups = q.n > 0 && q.total >= b.res_cap ? q.total / 128 : 0;
  if ((int64_t)q.tq / 128 + q.groups > b.max_blocks) {
    q.ok = false;
    q.n = q.to_sink = q.groups = 0;
    q.total = q.old;
  }
  // without a flush: the groups of window rows that receive new tokens (one at least, which
  // also writes the lengths and the sink)
  q.units = q.groups > 0 ? q.groups : q.total > q.old ? (q.total - 1) / 128 - q.old / 128 + 1 : 1;
  return q;
}

// An octet of a row as its source type holds it (fp32: eight words, else four).
template <int DT>
struct Octet {
  uint32_t w[DT == KVQ_F32 ? 8 : 4];
};
template <int DT>
__device__ __forceinline__ Octet<DT> octet_load(const void* base, int64_t i) {
  Octet<DT> x;
  const uint4* p = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(base) + i * (DT == KVQ_F32 ? 4 : 2));
#pragma unroll
  for (int k = 0; k < (DT == KVQ_F32 ? 2 : 1); ++k) {
    const uint4 v = p[k];
    x.w[4 * k] = v.x; x.w[4 * k + 1] = v.y; x.w[4 * k + 2] = v.z; x.w[4 * k + 3] = v.w;
  }
  return x;
}
template <int DT>
__device__ __forceinline__ void octet_store(void* base, int64_t i, const Octet<DT>& x) {
  uint4* p = reinterpret_cast<uint4*>(reinterpret_cast<char*>(base) + i * (DT == KVQ_F32 ? 4 : 2));
#pragma unroll
  for (int k = 0; k < (DT == KVQ_F32 ? 2 : 1); ++k) p[k] = make_uint4(x.w[4 * k], x.w[4 * k + 1], x.w[4 * k + 2], x.w[4 * k + 3]);
}
template <int DT>
__device__ __forceinline__ void octet_get(const Octet<DT>& x, float (&f)[8]) {
  if constexpr (DT == KVQ_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(x.w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == KVQ_F16) {
        f[2 * j] = half_bits_to_float((uint16_t)(x.w[j] & 0xffffu));
        f[2 * j + 1] = half_bits_to_float((uint16_t)(x.w[j] >> 16));
      } else {
        f[2 * j] = __uint_as_float(x.w[j] << 16);
        f[2 * j + 1] = __uint_as_float(x.w[j] & 0xffff0000u);
      }
    }
  }
}
template <int DT>
__device__ __forceinline__ Octet<DT> octet_put(const float (&f)[8]) {   // rounded to the type
  Octet<DT> x;
  if constexpr (DT == KVQ_F32) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x.w[j] = __float_as_uint(f[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) x.w[j] = pack2(f[2 * j], f[2 * j + 1], DT);
  }
  return x;
}

// Codes of eight values, BITS each, packed from the low end: rint_even(fl(fl(x - z) / s)) as pack8 finds it (the
// product with fl(1 / s) decides unless it lies within 2^-12 of a half-integer).  0 <= x - z and s is rounded
// up, so the quotient stays within half a step of 0 .. 2^BITS - 1 and needs no clamp; where x, s or z is
// not finite it is NaN (or 0), and the code 0 as pack8's.  q + 1.5 * 2^23 holds the integer in its low bits; the
// sums of these words, less the constants, are the packed codes, so no word may hold anything else.
template <int BITS>
__device__ __forceinline__ uint32_t pack_codes(const float (&x)[8], const float (&s)[8], const float (&rs)[8],
                                               const float (&z)[8]) {
  const float big = 12582912.0f;
  float q[8], t[8];
  bool near = false;   // or NaN
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    q[j] = __fmul_rn(__fsub_rn(x[j], z[j]), rs[j]);
    t[j] = __fadd_rn(q[j], big);
    near |= !(fabsf(__fsub_rn(q[j], __fsub_rn(t[j], big))) <= 0.5f - 0x1p-12f);
  }
  if (near) {
#pragma unroll
    for (int j = 0; j < 8; ++j)   // NaN becomes code 0
      t[j] = fmaxf(__fadd_rn(__fdiv_rn(__fsub_rn(x[j], z[j]), s[j]), big), big);
  }
  uint32_t w = 0, less = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    w += __float_as_uint(t[j]) << (BITS * j);
    less += 0x4B400000u << (BITS * j);
  }
  return w - less;
}

// Whether an octet holds a NaN or Inf (0 times it is NaN), two 16-bit numbers at a time.
template <int DT>
__device__ __forceinline__ bool octet_bad(const Octet<DT>& x) {
  if constexpr (DT == KVQ_F32) {
    float fin = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) fin = fmaf(__uint_as_float(x.w[j]), 0.0f, fin);
    return !(fin == 0.0f);
  } else {
    uint32_t fin = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if constexpr (DT == KVQ_F16) asm("fma.rn.f16x2 %0, %1, %2, %0;" : "+r"(fin) : "r"(x.w[j]), "r"(0));
      else asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(fin) : "r"(x.w[j]), "r"(0));
    }
    return (fin & 0x7fff7fffu) != 0;
  }
}

// Octet o of N rows, those with fresh[k] being new tokens (row `row[k]` of the source, at position pos[k]),
// when they are keys turned and rounded, and checked as they are stored.  The 16 lanes of a row call together: the
// half-layout partner comes from its lane.  A NaN or Inf stays one when it is turned, so the check of what is
// stored finds it as well as numbers that the turn, up to sqrt 2 in magnitude, takes beyond the type; then the
// octets it came from tell the two apart.
template <int DT, int N>
__device__ __forceinline__ void turn_rows(const AppendArgs& a, int which, int o, const int64_t (&row)[N],
                                          const int64_t (&pos)[N], const bool (&fresh)[N], Octet<DT> (&x)[N], int& flags) {
  const bool turns = which == KVQ_KEYS && a.rope.table;
  const int po = rope_partner(a.rope, o);
#pragma unroll
  for (int k = 0; k < N; ++k) {
    Octet<DT> y = x[k];
    if (turns && !a.rope.inter) {
#pragma unroll
      for (int j = 0; j < (DT == KVQ_F32 ? 8 : 4); ++j) y.w[j] = __shfl_sync(0xffffffffu, x[k].w[j], po, 16);
    }
    if (!fresh[k]) continue;
    int64_t at = -1;
    bool turned = turns && 8 * o < a.rope.rot;
    if (turned) {
      at = a.positions ? a.positions[row[k]] : pos[k];
      if (at < 0 || at >= a.rope.n_pos) {
        flags |= KVQ_DEV_BOUNDS;
        turned = false;
      }
    }
    if (!turned) {
      if (octet_bad<DT>(x[k])) flags |= KVQ_DEV_NONFINITE;
      continue;
    }
    float f[8], p[8];
    octet_get<DT>(x[k], f);
    octet_get<DT>(y, p);
    OctetTurn t;
    rope_load(a.rope, at, o, t);
    rope_turn(a.rope, o, t, f, p);
    const Octet<DT> r = octet_put<DT>(f);
    if (octet_bad<DT>(r)) flags |= octet_bad<DT>(x[k]) || octet_bad<DT>(y) ? KVQ_DEV_NONFINITE : KVQ_DEV_RANGE;
    x[k] = r;
  }
}

// Grid (units, kv head x {keys, values}).  Thread (r, o): octet o = t % 16 of rows
// 2 (r + 16 j), 2 (r + 16 j) + 1, j = 0 .. 3, of the unit's 128 rows, in registers (as the source type holds
// them; a rotating format's keys in fp32) from the load to the codes.  Keys: a channel's min and max meet over
// the two row slices of a warp, then over the 8 warps in shared memory; values: a token's over its 16
// lanes.  The rows of a value pair sit in one thread, which owns the pair's word.
// Rows kept as loaded leave three CTAs per SM (80 registers) where fp32 registers left one: a batch of prompts,
// 30k tokens of 8 heads in bf16, 310 us with one CTA, 129 with two, 117 with three (1.2 TB/s of rows in and
// codes out; bound by instruction fetch, the chain of dependent loads and barriers of a unit, and its
// arithmetic).  fp32 rows and transformed keys need 178 to 192 registers and have one CTA: 227 and 254 us against 135
// of bf16 in the same run with its caches flushed.
template <int DT, bool ROT>
__global__ void __launch_bounds__(kThreads, DT == KVQ_F32 || ROT ? 1 : 3)
    append_paged_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ float pmin[8][128], pmax[8][128];
  __shared__ float sf[128], zf[128], rf[128];
  griddep_wait();
  griddep_launch_dependents();
  const PagedBatch& b = a.b;
  const int h = blockIdx.y >> 1, which = blockIdx.y & 1;
  int s, unit;
  if (a.direct) {   // one unit each: no search
    s = blockIdx.x;
    unit = 0;
  } else if (!find_unit(b.num_seqs, blockIdx.x, [&](int i) { return append_seq(b, i).units; }, &s, &unit)) {
    return;
  }
  AppendSeq q = append_seq(b, s);
  int flags = q.ok ? 0 : KVQ_DEV_BOUNDS;
  // every block the sequence needs is checked by each of its CTAs: all of it or nothing
  bool missing = false;
  for (int j = threadIdx.x; j < q.groups; j += kThreads) {
    const int blk = b.table[(int64_t)s * b.max_blocks + q.tq / 128 + j];
    missing |= blk < 0 || blk >= b.num_blocks;
  }
  if (__syncthreads_or(missing)) {
    flags = KVQ_DEV_BOUNDS;
    q.ok = false;
  }
  if (unit == 0 && blockIdx.y == 0 && threadIdx.x == 0) {
    a.t_quant_out[s] = q.tq + (q.ok ? 128 * q.groups : 0);
    a.t_res_out[s] = !q.ok ? q.tr : q.groups ? q.total - 128 * q.groups : q.tr + q.n;
  }
  if (!q.ok || q.n == 0) {
    if (flags && threadIdx.x == 0) flag(a.status, flags);
    return;
  }
  const int ns = b.n_sink;
  const int o = threadIdx.x & 15, rs = threadIdx.x >> 4, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t pos0 = (int64_t)ns + q.tq + q.tr;                 // position of the first new token
  // a few tokens for the window alone: the sequence's first CTA copies them for all heads, the others are
  // done (64 sequences, one token each, 8 heads: 18.4 us with a CTA per head and side)
  if (a.direct && q.groups == 0 && q.tr >= 0 && q.n * a.L.Hkv <= 64) {
    if (blockIdx.y) return;
#pragma unroll
    for (int side = 0; side < 2; ++side)
      for (int i0 = 0; i0 < q.n * a.L.Hkv; i0 += 16) {
        const int i = i0 + rs, r = i / a.L.Hkv, hh = i - r * a.L.Hkv;
        const bool fresh[1] = {i < q.n * a.L.Hkv};
        const int64_t row[1] = {q.row0 + r}, pos[1] = {pos0 + r};
        Octet<DT> x[1] = {};
        if (fresh[0]) x[0] = octet_load<DT>(a.src[side], row[0] * a.st[side] + hh * a.sh[side] + 8 * o);
        turn_rows<DT, 1>(a, side, o, row, pos, fresh, x, flags);
        if (fresh[0])
          octet_store<DT>(a.res[side], (((int64_t)s * a.L.Hkv + hh) * b.res_cap + q.tr + r) * 128 + 8 * o, x[0]);
      }
    flags = __reduce_or_sync(0xffffffffu, flags);
    if (flags && lane == 0) flag(a.status, flags);
    return;
  }
  const int64_t slab = (int64_t)s * a.L.Hkv + h;
  char* res = reinterpret_cast<char*>(a.res[which]) + slab * b.res_cap * 128 * a.L.raw_bytes;
  // row r of (window rows, then new tokens behind the sink)
  const int64_t new0 = q.row0 + q.to_sink - q.old;                // + r: the new row of r >= old
  const int64_t npos = pos0 + q.to_sink - q.old;                  // + r: its position
  // new rows [lo, hi) (counted from source row `from` at position `at`) to rows from `to` on of a raw array, four
  // of this thread's in flight
  auto copy_rows = [&](int64_t from, int64_t at, int lo, int hi, char* dst, int to) {
    for (int r0 = lo; r0 < hi; r0 += 64) {
      Octet<DT> x[4] = {};
      int64_t row[4], pos[4];
      bool fresh[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int r = r0 + rs + 16 * k;
        fresh[k] = r < hi;
        row[k] = from + r;
        pos[k] = at + r;
        if (fresh[k]) x[k] = octet_load<DT>(a.src[which], row[k] * a.st[which] + h * a.sh[which] + 8 * o);
      }
      turn_rows<DT, 4>(a, which, o, row, pos, fresh, x, flags);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (fresh[k]) octet_store<DT>(dst, (int64_t)(to + r0 - lo + rs + 16 * k) * 128 + 8 * o, x[k]);
    }
  };
  if (q.groups > 0) {
    Octet<DT> raw[8];
    {
      int64_t row[8], pos[8];
      bool fresh[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = 128 * unit + 2 * (rs + 16 * (k >> 1)) + (k & 1);
        fresh[k] = r >= q.old;
        row[k] = new0 + r;
        pos[k] = npos + r;
        raw[k] = fresh[k] ? octet_load<DT>(a.src[which], row[k] * a.st[which] + h * a.sh[which] + 8 * o)
                          : octet_load<DT>(res, (int64_t)r * 128 + 8 * o);
      }
      turn_rows<DT, 8>(a, which, o, row, pos, fresh, raw, flags);
    }
    const int blk = b.table[(int64_t)s * b.max_blocks + q.tq / 128 + unit];
    const Side& S = a.L.side[which];
    const int64_t ps = (int64_t)blk * a.L.Hkv + h;
    uint8_t* codes = reinterpret_cast<uint8_t*>(S.codes) + ps * S.code_slab_bytes;
    __half* scale = reinterpret_cast<__half*>(S.scale) + ps * 128;
    __half* zero = reinterpret_cast<__half*>(S.zero) + ps * 128;
    if (which == KVQ_KEYS) {
      float wide[ROT ? 8 : 1][8];
      if constexpr (ROT) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          octet_get<DT>(raw[k], wide[k]);
          wht128_octet_unscaled(wide[k], lane);
#pragma unroll
          for (int j = 0; j < 8; ++j) wide[k][j] = __fmul_rn(wide[k][j], a.L.rot_scale);
        }
      }
      auto value = [&](int k, float (&x)[8]) {
        if constexpr (ROT) {
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = wide[k][j];
        } else {
          octet_get<DT>(raw[k], x);
        }
      };
      float mn[8], mx[8];
      value(0, mn);
#pragma unroll
      for (int j = 0; j < 8; ++j) mx[j] = mn[j];
#pragma unroll
      for (int k = 1; k < 8; ++k) {
        float x[8];
        value(k, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          mn[j] = fminf(mn[j], x[j]);
          mx[j] = fmaxf(mx[j], x[j]);
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        mn[j] = fminf(mn[j], __shfl_xor_sync(0xffffffffu, mn[j], 16));
        mx[j] = fmaxf(mx[j], __shfl_xor_sync(0xffffffffu, mx[j], 16));
        if (lane < 16) {
          pmin[warp][8 * o + j] = mn[j];
          pmax[warp][8 * o + j] = mx[j];
        }
      }
      __syncthreads();
      if (threadIdx.x < 128) {
        const int c = threadIdx.x;
        float m0 = pmin[0][c], m1 = pmax[0][c];
#pragma unroll
        for (int k = 1; k < 8; ++k) {
          m0 = fminf(m0, pmin[k][c]);
          m1 = fmaxf(m1, pmax[k][c]);
        }
        __half sh, zh;
        if (!asym_params(m0, m1, 4, &sh, &zh)) flags |= KVQ_DEV_RANGE;
        scale[c] = sh;
        zero[c] = zh;
        sf[c] = __half2float(sh);
        zf[c] = __half2float(zh);
        rf[c] = __frcp_rn(sf[c]);
      }
      __syncthreads();
      float s8[8], z8[8], r8[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        s8[j] = sf[8 * o + j];
        z8[j] = zf[8 * o + j];
        r8[j] = rf[8 * o + j];
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int r = 2 * (rs + 16 * (k >> 1)) + (k & 1);
        float x[8];
        value(k, x);
        *reinterpret_cast<uint32_t*>(codes + r * 64 + 4 * o) = pack_codes<4>(x, s8, r8, z8);
      }
    } else {
      uint32_t half_word = 0;
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float x[8];
        octet_get<DT>(raw[k], x);
        float mn = x[0], mx = x[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) {
          mn = fminf(mn, x[j]);
          mx = fmaxf(mx, x[j]);
        }
#pragma unroll
        for (int m = 1; m < 16; m <<= 1) {
          mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, m));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
        }
        __half sh, zh;
        if (!asym_params(mn, mx, 2, &sh, &zh)) flags |= KVQ_DEV_RANGE;
        const int u = rs + 16 * (k >> 1), r = 2 * u + (k & 1);
        if (o == 0) {
          scale[r] = sh;
          zero[r] = zh;
        }
        float s8[8], z8[8], r8[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          s8[j] = __half2float(sh);
          z8[j] = __half2float(zh);
          r8[j] = __frcp_rn(s8[j]);
        }
        const uint32_t w = pack_codes<2>(x, s8, r8, z8) & 0xffffu;
        if ((k & 1) == 0) half_word = w;
        else reinterpret_cast<uint32_t*>(codes)[u * 16 + o] = half_word | (w << 16);
      }
    }
  }
  if (unit == 0) {
    // the sink's share of the new tokens
    if (q.to_sink > 0)
      copy_rows(q.row0, pos0, 0, q.to_sink, reinterpret_cast<char*>(a.sink[which]) + slab * ns * 128 * a.L.raw_bytes,
                ns + q.tr);
    // rows behind the packed groups start the window anew; every thread has read its window
    // rows of group 0 (the only ones that overlap rows below 128) before the barrier
    if (q.groups > 0) {
      __syncthreads();
      copy_rows(new0, npos, 128 * q.groups, q.total, res, 0);
    }
  }
  if (q.groups == 0) {
    const int lo = max(q.old, (q.old / 128 + unit) * 128), hi = min(q.total, (q.old / 128 + unit + 1) * 128);
    copy_rows(new0, npos, lo, hi, res, lo);
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (flags && lane == 0) flag(a.status, flags);
}

// ---- read-back -------------------------------------------------------------------------
// A sequence's rows as pieces: one of the sink, one per touched group of packed tokens, one
// of the window.
struct ReadSeq {
  int64_t row0, p0, p1;     // first row; positions [p0, p1)
  int tq, tr, g0, ng;       // first touched group and their number
  bool ok;
};

__device__ __forceinline__ ReadSeq read_seq(const ReadArgs& a, int s) {
  const PagedBatch& b = a.b;
  ReadSeq q;
  const int64_t lo = b.cu[s], hi = b.cu[s + 1];
  q.tq = b.t_quant[s];
  q.tr = b.t_res[s];
  q.row0 = lo;
  q.p0 = a.first[s];
  q.p1 = q.p0 + (hi - lo);
  q.ok = lo >= 0 && hi >= lo && hi <= b.n_rows && hi - lo <= b.max_rows && q.tq >= 0 && q.tr <= b.res_cap &&
         q.tr >= -b.n_sink && (q.tr >= 0 || q.tq == 0) && (q.tq + 127ll) / 128 <= b.max_blocks && q.p0 >= 0 &&
         (hi == lo || q.p1 <= (int64_t)b.n_sink + q.tq + q.tr);
  if (!q.ok) q.p1 = q.p0;
  const int64_t lo_t = max(q.p0 - b.n_sink, (int64_t)0), hi_t = min(q.p1 - b.n_sink, (int64_t)q.tq);
  q.g0 = (int)(lo_t / 128);
  q.ng = hi_t > lo_t ? (int)((hi_t - 1) / 128) - q.g0 + 1 : 0;
  return q;
}

// Grid (units, kv head x {keys, values}); thread (r, o): octet o of rows r + 16 j (keys) or pairs r + 16 j
// (values).  Bound by the rows written; four CTAs per SM cover the dependent loads (table, page, codes).
template <int OD>
__global__ void __launch_bounds__(kThreads, 4) read_paged_kernel(const __grid_constant__ ReadArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const PagedBatch& b = a.b;
  const int h = blockIdx.y >> 1, which = blockIdx.y & 1;
  if (a.out[which] == nullptr) return;
  int s, unit;
  if (a.direct) {   // four pieces each at most: no search
    s = blockIdx.x >> 2;
    unit = blockIdx.x & 3;
  } else if (!find_unit(b.num_seqs, blockIdx.x, [&](int i) { return read_seq(a, i).ng + 2; }, &s, &unit)) {
    return;
  }
  const ReadSeq q = read_seq(a, s);
  if (unit > q.ng + 1) return;
  if (!q.ok) {
    if (unit == 0 && h == 0 && threadIdx.x == 0) flag(a.status, KVQ_DEV_BOUNDS);   // either side may be the only one
    return;
  }
  const int o = threadIdx.x & 15, rs = threadIdx.x >> 4, lane = threadIdx.x & 31;
  const int dt = a.L.src_dtype, ns = b.n_sink;
  const int64_t slab = (int64_t)s * a.L.Hkv + h;
  // output element of position p, octet o
  auto at = [&](int64_t p) { return ((q.row0 + p - q.p0) * a.L.Hkv + h) * 128 + 8 * o; };
  if (unit >= q.ng) {   // raw rows: the sink, then the window
    const bool win = unit > q.ng;
    const char* src = reinterpret_cast<const char*>(win ? a.res[which] : a.sink[which]) +
                      slab * (win ? b.res_cap : ns) * 128 * a.L.raw_bytes;
    const int64_t base = win ? (int64_t)ns + q.tq : 0;
    const int64_t lo = max(q.p0, base), hi = win ? q.p1 : min(q.p1, (int64_t)ns);
#pragma unroll 4
    for (int64_t p = lo + rs; p < hi; p += 16) {
      float x[8];
      load8(src, (p - base) * 128 + 8 * o, dt, x);
      store8(a.out[which], at(p), OD, x);
    }
    return;
  }
  const int gi = q.g0 + unit;
  const int blk = b.table[(int64_t)s * b.max_blocks + gi];
  if (blk < 0 || blk >= b.num_blocks) {
    if (threadIdx.x == 0) flag(a.status, KVQ_DEV_BOUNDS);
    return;
  }
  const int64_t base = (int64_t)ns + 128ll * gi;     // position of the group's first token
  const int lo = (int)max(q.p0 - base, (int64_t)0), hi = (int)min(min(q.p1 - base, (int64_t)ns + q.tq - base), (int64_t)128);
  const Side& S = a.L.side[which];
  const int64_t ps = (int64_t)blk * a.L.Hkv + h;
  const uint8_t* codes = reinterpret_cast<const uint8_t*>(S.codes) + ps * S.code_slab_bytes;
  const __half* scale = reinterpret_cast<const __half*>(S.scale) + ps * 128;
  const __half* zero = reinterpret_cast<const __half*>(S.zero) + ps * 128;
  // all of the thread's words of the group first, then the rows
  if (which == KVQ_KEYS) {
    float s8[8], z8[8];
    load8(scale, 8 * o, KVQ_F16, s8);
    load8(zero, 8 * o, KVQ_F16, z8);
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) w[k] = reinterpret_cast<const uint32_t*>(codes)[(rs + 16 * k) * 16 + o];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int r = rs + 16 * k;
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(__fmul_rn((float)((w[k] >> (4 * j)) & 15u), s8[j]), z8[j]);
      if (a.L.k_rotate) {
        wht128_octet_unscaled(x, lane);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fmul_rn(x[j], a.L.rot_scale);
      }
      if (r >= lo && r < hi) store8(a.out[which], at(base + r), OD, x);
    }
  } else {
    uint32_t w[4], sz[4][2];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = rs + 16 * k;
      w[k] = reinterpret_cast<const uint32_t*>(codes)[u * 16 + o];
      sz[k][0] = reinterpret_cast<const uint32_t*>(scale)[u];
      sz[k][1] = reinterpret_cast<const uint32_t*>(zero)[u];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = 2 * (rs + 16 * k) + e;
        const float sv = half_bits_to_float((uint16_t)(sz[k][0] >> (16 * e))), zv = half_bits_to_float((uint16_t)(sz[k][1] >> (16 * e)));
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(__fmul_rn((float)((w[k] >> (16 * e + 2 * j)) & 3u), sv), zv);
        if (r >= lo && r < hi) store8(a.out[which], at(base + r), OD, x);
      }
  }
}

}  // namespace

cudaError_t launch_append_paged(const AppendArgs& args, cudaStream_t s) {
  // units of a sequence: at most floor((res_cap + n) / 128), one at least; exactly one each for short
  // appends to a window of one group, which then need no search for their sequence
  const int64_t units = (int64_t)args.b.num_seqs * (args.b.res_cap / 128) + args.b.n_rows / 128;
  AppendArgs a = args;
  a.direct = a.b.res_cap == 128 && a.b.max_rows < 128;
  const dim3 grid(a.direct ? a.b.num_seqs : (unsigned)units, 2 * a.L.Hkv);
  const bool rot = a.L.k_rotate;
  auto kern = a.L.src_dtype == KVQ_F32   ? (rot ? append_paged_kernel<KVQ_F32, true> : append_paged_kernel<KVQ_F32, false>)
              : a.L.src_dtype == KVQ_F16 ? (rot ? append_paged_kernel<KVQ_F16, true> : append_paged_kernel<KVQ_F16, false>)
                                         : (rot ? append_paged_kernel<KVQ_BF16, true> : append_paged_kernel<KVQ_BF16, false>);
  return launch_pdl(kern, grid, dim3(kThreads), 0, s, a);
}

cudaError_t launch_read_paged(const ReadArgs& args, cudaStream_t s) {
  // touched groups of n rows: at most (n + 254) / 128; the sink and the window two more
  ReadArgs a = args;
  a.direct = a.b.max_rows <= 129;
  const int64_t units = 4ll * a.b.num_seqs + (a.direct ? 0 : a.b.n_rows / 128);
  auto kern = a.out_dtype == KVQ_F32   ? read_paged_kernel<KVQ_F32>
              : a.out_dtype == KVQ_F16 ? read_paged_kernel<KVQ_F16>
                                       : read_paged_kernel<KVQ_BF16>;
  return launch_pdl(kern, dim3((unsigned)units, 2 * a.L.Hkv), dim3(kThreads), 0, s, a);
}

}  // namespace kvq
