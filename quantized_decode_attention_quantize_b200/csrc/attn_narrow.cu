// Attention of a few new tokens per sequence (drafts to verify, single tokens): blocks of up to 16 query
// rows, each run of KV tiles on one warp with its own copies, so that no warp waits for another.
//
// Mathematics.  Scores are products with tokens as M and query rows as N (m16n8k16, two of them for 16
// rows), values with channels as M and query rows as N:
//   A[t][d] = c[t][d] 2^-24 f_d   (a 4-bit code masked into the low bits of an fp16 number, f_d = 1 or 16),
//   B[d][r] = fp16(q[r][d] s[d] / (f_d n))  per group,   score = 2^24 n (A B) + sum_d (q z + 8 (q s - f_d n B)),
//   A[d][t] = c[t][d] exactly (masked into 2^k + c, less 2^k),   B[t][r] = fp16(p s 2^7),
//   O[d][r] = 2^-7 (A B) + sum_t p z.
// A lane's four words of a key row are the A fragments of eight k-steps (channels go to k in the order that the
// masks give, for B alike), and word g and g + 8 of a value pair are rows g and g + 8 of the eight channel tiles
// (tile c: channels 8 g + c and 64 + 8 g + c).  The probabilities go from one product to the other by an 8x8
// transpose in registers.  The running maximum follows score + log2 s, which keeps B inside fp16 for any
// scale; it moves only when exceeded by more than 8.  Queries are scaled to [4, 8) by a power of two of their
// row, and n is 1 but for groups with a key scale above 8188 (65504 / 8), where 8 times the scale would leave fp16:
// there n = 16, which serves up to fp16's largest scale.  A smaller range of the queries would serve all
// groups, but costs small scales their last bits: q s / 16 is subnormal below 2^-14.
//
// What bounds it: the expansion and the softmax on CUDA cores, 476 warp instructions and 1.5 us per 16 tokens, at
// two warps per scheduler (255 registers), which use 42 % of the issue slots; the packed bytes pass once per 16
// rows.  4 tokens and fewer x 8 sequences over 32768 and fewer, 8 x 4 heads: 99 us with the merge.
#include "attn_paged.cuh"

namespace kvq {
namespace {

using namespace attn;

constexpr int kWarps = 8;
constexpr int kStage = 8192 + 4096 + 4 * 256;   // a group: codes, then key and value scales and zero-points
constexpr int kKMeta = 8192 + 4096, kVMeta = kKMeta + 512;
constexpr int kStages = 2;
struct Small {
  alignas(8) uint64_t in[kWarps][kStages];
  int stop;
};
constexpr size_t kSmem = (size_t)kWarps * kStages * kStage + sizeof(Small);

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t h2mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
constexpr uint32_t kSixteenth2 = 0x2C002C00u;
__device__ __forceinline__ uint32_t at_most_8188(uint32_t s) {   // all ones in such halves
  return __hle2_mask(*reinterpret_cast<const __half2*>(&s), __half2half2(__ushort_as_half(0x6FFF)));
}
__device__ __forceinline__ float2 h2f(uint32_t a) { return __half22float2(*reinterpret_cast<const __half2*>(&a)); }

// The orthonormal transform of a row of which this lane (t of four) holds channels 32 t .. + 31.
__device__ __forceinline__ void wht_quarter(float (&x)[32], int lane, float scale) {
#pragma unroll
  for (int h = 1; h < 32; h <<= 1)
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (!(j & h)) {
        const float u = x[j], v = x[j + h];
        x[j] = u + v;
        x[j + h] = u - v;
      }
#pragma unroll
  for (int m = 1; m < 4; m <<= 1)
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float o = __shfl_xor_sync(0xffffffffu, x[j], m);
      x[j] = (lane & m ? o - x[j] : x[j] + o) * (m == 2 ? scale : 1.0f);
    }
}

// 32 channels from element i on.
__device__ __forceinline__ void load32(const void* p, int64_t i, int dtype, bool there, float (&x)[32]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    if (there) load8(p, i + 8 * k, dtype, y);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[8 * k + j] = y[j];
  }
}
// As fp16 pairs in the order of the masks: octet k gives (0, 4), (1, 5), (2, 6), (3, 7).
__device__ __forceinline__ uint32_t octet_pair(const float (&x)[32], int k, int j, float f) {
  return pack_f16(x[8 * k + j] * f, x[8 * k + j + 4] * f);
}

// A warp's state for its block: lane (g, t) = (lane / 4, lane % 4) holds queries 2 t, 2 t + 1, 8 + 2 t, 9 + 2 t of the
// scalars (alike over g, but l and zp, which are sums over the lane's own tokens).
struct State {
  float o[8][2][4];     // channel tile, row tile: (8 g + c, q), (8 g + c, q + 1), (64 + 8 g + c, q), ...
  float m[4], l[4], zp[4];
};

// 16 tokens: raw scores acc[row tile][4] (tokens g, g, g + 8, g + 8; queries 2 t, 2 t + 1), score = acc * mul[q] + add[q];
// scale, log2 scale and zero-point of tokens g and g + 8; cols[q]: tokens of these 16 that q sees.  Leaves the
// weights as B fragments.
__device__ __forceinline__ void weigh(State& st, const float (&acc)[2][4], const float (&mul)[4], const float (&add)[4],
                                      const float (&s)[2], const float (&ls)[2], const float (&z)[2], const int (&cols)[4],
                                      bool edge, int g, uint32_t (&b)[2][2]) {
  float x[2][4];   // [row tile][acc order]
  bool over = false;
#pragma unroll
  for (int n = 0; n < 2; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int q = 2 * n + (e & 1);
      x[n][e] = fmaf(acc[n][e], mul[q], add[q]);
      if (edge && g + 8 * (e >> 1) >= cols[q]) x[n][e] = -INFINITY;
      over |= x[n][e] + ls[e >> 1] > st.m[q] + kLazy;
    }
  if (__any_sync(0xffffffffu, over)) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int n = q >> 1, e = q & 1;
      float top = fmaxf(x[n][e] + ls[0], x[n][e + 2] + ls[1]);
#pragma unroll
      for (int k = 4; k < 32; k <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
      if (top > st.m[q] + kLazy) {
        const float f = exp2_approx(st.m[q] - top);
        st.m[q] = top;
        st.l[q] *= f;
        st.zp[q] *= f;
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          st.o[c][n][e] *= f;
          st.o[c][n][e + 2] *= f;
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    float w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int q = 2 * n + (e & 1);
      const float p = exp2_approx(x[n][e] - (st.m[q] == -INFINITY ? 0.0f : st.m[q]));
      st.l[q] += p;
      st.zp[q] = fmaf(p, z[e >> 1], st.zp[q]);
      w[e] = p * (s[e >> 1] * 128.0f);
    }
    b[n][0] = transpose8(pack_f16(w[0], w[1]));
    b[n][1] = transpose8(pack_f16(w[2], w[3]));
  }
}

template <uint32_t MASK, uint32_t MAGIC>
__device__ __forceinline__ uint32_t code_only(uint32_t w) { return h2sub((w & MASK) | MAGIC, MAGIC); }
// Channel tile c's A fragment from words g and g + 8 of two token pairs.
template <uint32_t MASK, uint32_t MAGIC>
__device__ __forceinline__ void value_tile(State& st, int c, const uint32_t (&w)[4], const uint32_t (&b)[2][2]) {
  const uint32_t a0 = code_only<MASK, MAGIC>(w[0]), a1 = code_only<MASK, MAGIC>(w[1]);
  const uint32_t a2 = code_only<MASK, MAGIC>(w[2]), a3 = code_only<MASK, MAGIC>(w[3]);
  mma16816(st.o[c][0], a0, a1, a2, a3, b[0][0], b[0][1]);
  mma16816(st.o[c][1], a0, a1, a2, a3, b[1][0], b[1][1]);
}

// A group's metadata, four channels and four tokens a lane: what gives numbers beyond fp16 is flagged, and key
// channels with an infinity or NaN are set to zero where they lie (value tokens are as they are read).  With
// a scale above 8188 all key scales are divided by n = 16 there; true then.
__device__ __forceinline__ bool check_group(uint8_t* in, int lane, int valid, int& flags) {
  uint2* ks = reinterpret_cast<uint2*>(in + kKMeta) + lane;
  uint2* kz = reinterpret_cast<uint2*>(in + kKMeta + 256) + lane;
  const uint2 vs = reinterpret_cast<const uint2*>(in + kVMeta)[lane], vz = reinterpret_cast<const uint2*>(in + kVMeta + 256)[lane];
  uint2 s = *ks, z = *kz;
  const int left = valid - 4 * lane;
  const uint32_t k = finite2(h2fma(kFifteen2, s.x, z.x)) & finite2(h2fma(kFifteen2, s.y, z.y));
  const uint32_t v = (finite2(h2fma(kThree2, vs.x, vz.x)) | (left >= 2 ? 0u : left == 1 ? 0xffff0000u : 0xffffffffu)) &
                     (finite2(h2fma(kThree2, vs.y, vz.y)) | (left >= 4 ? 0u : left == 3 ? 0xffff0000u : 0xffffffffu));
  const uint32_t small = at_most_8188(s.x) & at_most_8188(s.y);
  if (!__any_sync(0xffffffffu, (k & v & small) != 0xffffffffu)) return false;
  if ((k & v) != 0xffffffffu) flags |= KVQ_DEV_RANGE;
  const uint32_t mx = finite2(s.x) & finite2(z.x), my = finite2(s.y) & finite2(z.y);
  s = make_uint2(s.x & mx, s.y & my);
  z = make_uint2(z.x & mx, z.y & my);
  const bool big = __any_sync(0xffffffffu, (at_most_8188(s.x) & at_most_8188(s.y)) != 0xffffffffu);
  if (big) s = make_uint2(h2mul(s.x, kSixteenth2), h2mul(s.y, kSixteenth2));
  *ks = s;
  *kz = z;
  fence_async_smem();   // before the next group's copies into this stage
  __syncwarp();
  return big;
}

__global__ void __launch_bounds__(32 * kWarps, 1) attn_narrow_kernel(const __grid_constant__ AttnArgs a,
                                                                     const __grid_constant__ Work work) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Small* sm = reinterpret_cast<Small*>(smem + kWarps * kStages * kStage);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kWarps * kStages; ++i) mbar_init(smem_u32(&sm->in[i / kStages][i % kStages]), 1);
    sm->stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  uint8_t* const stages = smem + warp * kStages * kStage;
  int flags = 0, issued = 0, taken = 0;   // groups of this warp
  AttnSeq q0 = {};
  int64_t w0 = 0;
  const Cut cut = find_cut(a, work.runs, lane, &q0, &w0);
  const int run = blockIdx.x * kWarps + warp;
  if (run == 0 && lane == 0) *work.cut = cut;
  if (run < cut.runs && cut.units > 0) {
    int64_t unit, left = run_start(cut, run + 1) - run_start(cut, run);
    Place p = find_place(a, run_start(cut, run), lane, q0, w0, &unit);
    bool ok = true;
    for (bool head = true; left > 0 && ok; head = false) {
      const int tiles = block_tiles(a, p.q, p.b);
      const Seg c = take_block(a, work, p, tiles, run, unit, left, head, lane);
      left -= min((int64_t)tiles + 1, unit + left) - unit;
      unit = 0;
      if (c.N > 0 || tiles == 0) {
        const int ns = min(a.b.n_sink, a.b.n_sink + c.tq + c.tr);
        const int64_t slab = (int64_t)c.s * a.L.Hkv + c.h;
        auto row_of = [&](int r) {
          const int tok = (c.r0 + r) / a.G;
          return ((int)c.row0 + tok) * a.Hq + c.h * a.G + (c.r0 + r - tok * a.G);
        };
        // the packed groups of this part, pages 32 at a time, two groups in flight
        const int raw_end = min(c.n_raw, c.t_lo + c.N);
        const int g0 = max(c.t_lo - c.n_raw, 0), g1 = c.t_lo + c.N - c.n_raw;
        int page = 0, next = g0;
        auto fetch = [&]() {
          if (next >= g1) return;
          if (((next - g0) & 31) == 0) {
            page = next + lane < g1 ? __ldg(a.b.table + (int64_t)c.s * a.b.max_blocks + next + lane) : 0;
            if (page < 0 || page >= a.b.num_blocks) {
              flags |= KVQ_DEV_BOUNDS;
              page = 0;
            }
          }
          const int64_t at = (int64_t)__shfl_sync(0xffffffffu, page, (next - g0) & 31) * a.L.Hkv + c.h;
          if (lane == 0) {
            const uint32_t bar = smem_u32(&sm->in[warp][issued % kStages]);
            const uint32_t to = smem_u32(stages + (issued % kStages) * kStage);
            expect_bytes(bar, kStage);
            bulk_load(to, reinterpret_cast<const uint8_t*>(a.L.side[0].codes) + at * a.L.side[0].code_slab_bytes, 8192, bar);
            bulk_load(to + 8192, reinterpret_cast<const uint8_t*>(a.L.side[1].codes) + at * a.L.side[1].code_slab_bytes, 4096,
                      bar);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              bulk_load(to + kKMeta + 512 * v, reinterpret_cast<const __half*>(a.L.side[v].scale) + at * 128, 256, bar);
              bulk_load(to + kKMeta + 512 * v + 256, reinterpret_cast<const __half*>(a.L.side[v].zero) + at * 128, 256, bar);
            }
          }
          ++issued;
          ++next;
        };
        fetch();
        fetch();

        // queries g and g + 8, channels 32 t .. + 31
        uint32_t qp[2][16];      // [row][4 octet + pair], odd pairs over 16
        float cs_own[2];         // log2 units of one unit of the scaled query's product
        bool bad = false;
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float x[32];
          const int r = g + 8 * n;
          const bool there = r < c.nr;
          load32(a.q, there ? (int64_t)row_of(r) * 128 + 32 * t : 0, a.q_dtype, there, x);
          uint32_t top = 0;
#pragma unroll
          for (int j = 0; j < 32; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
          bad |= top >= 0x7f800000u;
          if (a.L.k_rotate) {
            wht_quarter(x, lane, a.L.rot_scale);
            top = 0;
#pragma unroll
            for (int j = 0; j < 32; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
          }
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          const int e = min(max((int)(top >> 23), 10), 250);             // 2^(e - 127) <= top < 2^(e - 126)
          const float up = __uint_as_float((uint32_t)(256 - e) << 23);   // to [4, 8)
          cs_own[n] = fmaxf(a.qscale * __uint_as_float((uint32_t)(e - 2) << 23), 1.2e-38f);
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int j = 0; j < 4; ++j) qp[n][4 * k + j] = octet_pair(x, k, j, j & 1 ? up * 0.0625f : up);
        }
        if (__any_sync(0xffffffffu, bad)) flags |= KVQ_DEV_NONFINITE;

        State st;
        float cs[4];
        Seen see[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = 8 * (q >> 1) + 2 * t + (q & 1);
          cs[q] = __shfl_sync(0xffffffffu, cs_own[q >> 1], 4 * (2 * t + (q & 1)));
          see[q] = {0, 0};
          if (r < c.nr) {
            AttnSeq sq;
            sq.n = c.n;
            sq.tq = c.tq;
            sq.tr = c.tr;
            see[q] = row_seen(a, sq, (c.r0 + r) / a.G);
          }
          st.m[q] = -INFINITY;
          st.l[q] = st.zp[q] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
#pragma unroll
          for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) st.o[k][n][e] = 0.0f;

        // raw tiles of 16 tokens: keys and values as fp16
#pragma unroll 1
        for (int r0 = 16 * c.t_lo; r0 < 16 * raw_end; r0 += 16) {
          // values: tokens 2 t, 2 t + 1, 2 t + 8, 2 t + 9, channels 8 g .. + 7 and 64 + 8 g .. + 7
          uint32_t v[2][2][8];   // [token pair][channel half][channel]: (token, token + 1)
#pragma unroll
          for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              float y[2][8];
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int r = r0 + 2 * t + 8 * u + e;
                const bool sink = r < ns;
#pragma unroll
                for (int j = 0; j < 8; ++j) y[e][j] = 0.0f;
                if (r < c.raw)
                  load8(sink ? a.sink[1] : a.res[1],
                        (sink ? slab * a.b.n_sink + r : slab * a.b.res_cap + r - ns) * 128 + 64 * half + 8 * g, a.L.src_dtype,
                        y[e]);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                  if (!(fabsf(y[e][j]) <= 65504.0f)) {
                    flags |= isfinite(y[e][j]) ? KVQ_DEV_RANGE : KVQ_DEV_NONFINITE;
                    y[e][j] = 0.0f;
                  }
              }
#pragma unroll
              for (int j = 0; j < 8; ++j) v[u][half][j] = pack_f16(y[0][j], y[1][j]);
            }
          float acc[2][4] = {};
          {
            float x[2][32];
#pragma unroll
            for (int n = 0; n < 2; ++n) {
              const int r = r0 + g + 8 * n;
              const bool there = r < c.raw;
              const bool sink = r < ns;
              load32(sink ? a.sink[0] : a.res[0],
                     there ? (sink ? slab * a.b.n_sink + r : slab * a.b.res_cap + r - ns) * 128 + 32 * t : 0, a.L.src_dtype,
                     there, x[n]);
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                if (!(fabsf(x[n][j]) <= 65504.0f)) {
                  flags |= isfinite(x[n][j]) ? KVQ_DEV_RANGE : KVQ_DEV_NONFINITE;
                  x[n][j] = 0.0f;
                }
              }
              if (a.L.k_rotate) {
                wht_quarter(x[n], lane, a.L.rot_scale);
#pragma unroll
                for (int j = 0; j < 32; ++j) x[n][j] = within_f16(x[n][j], flags);
              }
            }
            const uint32_t sixteen = 0x4C004C00u;
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int n = 0; n < 2; ++n)
                  mma16816(acc[n], octet_pair(x[0], k, 2 * h, 1.0f), octet_pair(x[1], k, 2 * h, 1.0f),
                           octet_pair(x[0], k, 2 * h + 1, 1.0f), octet_pair(x[1], k, 2 * h + 1, 1.0f), qp[n][4 * k + 2 * h],
                           h2mul(qp[n][4 * k + 2 * h + 1], sixteen));
          }
          int cols[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) cols[q] = see[q].raw - r0;
          const float none[4] = {0, 0, 0, 0}, one[2] = {1.0f, 1.0f}, zero[2] = {0.0f, 0.0f};
          uint32_t b[2][2];
          weigh(st, acc, cs, none, one, zero, zero, cols, true, g, b);
#pragma unroll
          for (int k = 0; k < 8; ++k)
#pragma unroll
            for (int n = 0; n < 2; ++n)
              mma16816(st.o[k][n], v[0][0][k], v[0][1][k], v[1][0][k], v[1][1][k], b[n][0], b[n][1]);
        }

        // packed groups
#pragma unroll 1
        for (int gi = g0; gi < g1; ++gi) {
          const int slot = taken % kStages;
          if (!mbar_wait(smem_u32(&sm->in[warp][slot]), (taken / kStages) & 1, &sm->stop)) {
            ok = false;
            break;
          }
          ++taken;
          uint8_t* in = stages + slot * kStage;
          const int valid = min(128, c.tq - 128 * gi);
          const float by = check_group(in, lane, valid, flags) ? 16.0f : 1.0f;   // n
          // this group's B fragments and zero-point sums
          uint32_t bs[2][16];
          float mul[4], add[4], zd[2] = {0.0f, 0.0f};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint4 s = reinterpret_cast<const uint4*>(in + kKMeta)[4 * t + k];
            const uint4 z = reinterpret_cast<const uint4*>(in + kKMeta + 256)[4 * t + k];
            const uint32_t sp[4] = {lo2(s.x, s.z), hi2(s.x, s.z), lo2(s.y, s.w), hi2(s.y, s.w)};
            const uint32_t zq[4] = {lo2(z.x, z.z), hi2(z.x, z.z), lo2(z.y, z.w), hi2(z.y, z.w)};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 zf = h2f(zq[j]), sf = h2f(sp[j]);
              const float f = j & 1 ? 16.0f : 1.0f;
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                const float2 qf = h2f(qp[n][4 * k + j]);
                bs[n][4 * k + j] = h2mul(qp[n][4 * k + j], sp[j]);
                // q z, and what the rounding of q s takes from a code of 8, so that the error goes with c - 8
                const float2 bf = h2f(bs[n][4 * k + j]);
                const float ex = fmaf(8.0f * by, fmaf(qf.x, sf.x, -bf.x), qf.x * zf.x);
                const float ey = fmaf(8.0f * by, fmaf(qf.y, sf.y, -bf.y), qf.y * zf.y);
                zd[n] = fmaf(f, ex + ey, zd[n]);
              }
            }
          }
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            zd[n] += __shfl_xor_sync(0xffffffffu, zd[n], 1);
            zd[n] += __shfl_xor_sync(0xffffffffu, zd[n], 2);
          }
          int cols[4];
          bool edge = false;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            add[q] = cs[q] * __shfl_sync(0xffffffffu, zd[q >> 1], 4 * (2 * t + (q & 1)));
            mul[q] = cs[q] * (16777216.0f * by);
            cols[q] = see[q].packed - 128 * gi;
            edge |= cols[q] < 128;
          }
          edge = __any_sync(0xffffffffu, edge);
          // the next 16 tokens' scores are under way while these are weighed
          auto scores = [&](int k0, float (&acc)[2][4]) {
            const uint4 ka = reinterpret_cast<const uint4*>(in)[(16 * k0 + g) * 4 + t];
            const uint4 kb = reinterpret_cast<const uint4*>(in)[(16 * k0 + g + 8) * 4 + t];
            const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[n][e] = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t ua = wa[k] >> 8, ub = wb[k] >> 8;
#pragma unroll
              for (int n = 0; n < 2; ++n) {
                mma16816(acc[n], wa[k] & 0x000F000Fu, wb[k] & 0x000F000Fu, wa[k] & 0x00F000F0u, wb[k] & 0x00F000F0u,
                         bs[n][4 * k], bs[n][4 * k + 1]);
                mma16816(acc[n], ua & 0x000F000Fu, ub & 0x000F000Fu, ua & 0x00F000F0u, ub & 0x00F000F0u, bs[n][4 * k + 2],
                         bs[n][4 * k + 3]);
              }
            }
          };
          float acc[2][4], ahead[2][4];
          scores(0, ahead);
#pragma unroll 1
          for (int k0 = 0; k0 < 8; ++k0) {
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[n][e] = ahead[n][e];
            if (k0 < 7) scores(k0 + 1, ahead);
            const __half* vs = reinterpret_cast<const __half*>(in + kVMeta) + 16 * k0 + g;
            float s[2], ls[2], z[2];
            int left[4];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              // behind the end anything may lie; what did not fit fp16 when it was packed counts as zero
              s[e] = __half2float(vs[8 * e]);
              z[e] = __half2float(vs[128 + 8 * e]);
              const bool there = 16 * k0 + g + 8 * e < valid && s[e] <= 65504.0f && fabsf(z[e]) <= 65504.0f;
              if (!there) s[e] = z[e] = 0.0f;
              asm("lg2.approx.f32 %0, %1;" : "=f"(ls[e]) : "f"(there ? s[e] : 1.0f));
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) left[q] = cols[q] - 16 * k0;
            uint32_t b[2][2];
            weigh(st, acc, mul, add, s, ls, z, left, edge, g, b);
            const uint32_t* vw = reinterpret_cast<const uint32_t*>(in + 8192) + (8 * k0 + t) * 16 + g;
            const uint32_t w[4] = {vw[0], vw[8], vw[64], vw[72]};
            const uint32_t u[4] = {w[0] >> 8, w[1] >> 8, w[2] >> 8, w[3] >> 8};
            value_tile<0x00030003u, 0x64006400u>(st, 0, w, b);
            value_tile<0x000C000Cu, 0x5C005C00u>(st, 1, w, b);
            value_tile<0x00300030u, 0x54005400u>(st, 2, w, b);
            value_tile<0x00C000C0u, 0x4C004C00u>(st, 3, w, b);
            value_tile<0x00030003u, 0x64006400u>(st, 4, u, b);
            value_tile<0x000C000Cu, 0x5C005C00u>(st, 5, u, b);
            value_tile<0x00300030u, 0x54005400u>(st, 6, u, b);
            value_tile<0x00C000C0u, 0x4C004C00u>(st, 7, u, b);
          }
          __syncwarp();   // every lane has read this stage
          fetch();
        }
        if (!ok) break;

        // sums over the lanes with the same queries, then the state out
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
          for (int k = 4; k < 32; k <<= 1) {
            st.l[q] += __shfl_xor_sync(0xffffffffu, st.l[q], k);
            st.zp[q] += __shfl_xor_sync(0xffffffffu, st.zp[q], k);
          }
          const int r = 8 * (q >> 1) + 2 * t + (q & 1), n = q >> 1, e = q & 1;
          if (r >= c.nr) continue;
          const bool part = c.slot >= 0;
          const float f = part ? 1.0f : st.l[q] > 0.0f ? 0.0078125f / st.l[q] : 0.0f, zf = part ? 128.0f * st.zp[q] : 128.0f * st.zp[q] * f;
          void* to = part ? static_cast<void*>(work.o) : a.out;
          const int64_t row = part ? (int64_t)c.slot * work.rows + r : row_of(r);
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float y[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = fmaf(st.o[k][n][e + 2 * half], f, zf);
            const int64_t at = row * 128 + 64 * half + 8 * g;
            if (part || a.out_dtype == KVQ_F32) {
              float4* d = reinterpret_cast<float4*>(reinterpret_cast<float*>(to) + at);
              d[0] = make_float4(y[0], y[1], y[2], y[3]);
              d[1] = make_float4(y[4], y[5], y[6], y[7]);
            } else {
              uint32_t h[4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                if (a.out_dtype == KVQ_F16) {
                  h[k] = pack_f16(y[2 * k], y[2 * k + 1]);
                } else {
                  const __nv_bfloat162 b2 = __floats2bfloat162_rn(y[2 * k], y[2 * k + 1]);
                  h[k] = *reinterpret_cast<const uint32_t*>(&b2);
                }
              }
              *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(to) + at) = make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
          if (g == 0) {
            if (part) {   // the factor 2^7 that the other kernels' sums carry
              work.m[row] = st.m[q];
              work.l[row] = 128.0f * st.l[q];
            } else if (a.lse) {
              a.lse[row] = st.l[q] > 0.0f ? kLn2 * (st.m[q] + log2f(st.l[q])) : -INFINITY;
            }
          }
        }
      }
      if (left > 0 && !next_block(a, &p)) break;
    }
    if (!ok) {   // copies still on their way must land before the memory is given up
      flags |= KVQ_DEV_TIMEOUT;
      int never = 0;
      for (int n = taken; n < issued; ++n) mbar_wait(smem_u32(&sm->in[warp][n % kStages]), (n / kStages) & 1, &never);
    }
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (flags && lane == 0) flag(a.status, flags);
}

}  // namespace

namespace attn {
cudaError_t launch_attn_narrow(const AttnArgs& a, const Work& w, int runs, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(attn_narrow_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_narrow_kernel, dim3(runs / kWarps), dim3(32 * kWarps), kSmem, s, a, w);
}
}  // namespace attn

}  // namespace kvq
