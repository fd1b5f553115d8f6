// Attention of several new tokens per sequence over the paged cache (D = 128, groups of 128
// tokens, 4-bit per-channel keys, 2-bit per-token values, raw sink and window rows) on the
// fifth-generation tensor cores.
//
// Work.  The query rows of one KV head, G per new token, are cut into blocks of up to 256.  A
// CTA takes one block over a run of KV tiles of 128 tokens: the visible raw (sink, window)
// tokens first, then the visible packed groups.  It keeps two streams busy, so that one's
// products run under the other's softmax: the block's two halves of 128 rows over the same
// tiles, or, for a block of at most 128 rows, those rows over the even and the odd tiles, the
// two states merged at the end.
//
// Mathematics.  S = Q K^T and O += P V as products of fp16 with fp32 sums, one pass over the
// tiles with a running maximum m and sum l per row in the log2 domain.  m moves (and O, l are
// rescaled) only when the new maximum exceeds it by more than 8, so a weight is at most 2^8
// relative to m; weights carry another factor 2^7, so that they reach down to 2^-39 of
// the largest as fp16 numbers and up to 2^15.  Queries are scaled by a power of two of their
// own row to lie well inside fp16.  A 4-bit or 2-bit code masked into the mantissa of an fp16
// number 2^(10 - p) (p the bit it starts at) is 2^(10 - p) + c exactly; less that constant, one fused
// c * s + z gives the fp16 key or value.
//
// Roles (16 warps).  Warps 0-3 and 4-7: softmax of stream 0 and 1, one thread per row, S in registers
// from tensor memory, P back over S's columns as the A operand of the value product.  Warps
// 8-11: codes from global memory (one tile ahead, in registers) to fp16 tiles in shared
// memory, K as [token][channel] with the channels of an octet in the order 0 4 1 5 2 6 3 7 (which
// the masks give; Q has the same), V transposed to [channel][token].  Warp 12: one thread issues the
// products.  K and V tiles pass through one ring of four slots in the order the products use them.
//
// Tensor memory: S0, S1, O0, O1, 128 columns each (all 512).  A product that overwrites S with the
// next scores is issued after the value product that reads P from it, in the same thread's order.
//
// Waits are bounded (tc05.cuh); one that runs out stops the CTA and raises KVQ_DEV_TIMEOUT.
#include "paged_batch.cuh"
#include "tc05.cuh"
#include "wht.cuh"

namespace kvq {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 512;
constexpr int kTile = 32768;              // 128 x 128 fp16
constexpr int kSlots = 4;
constexpr int kSlotsAt = 2 * kTile;       // after the two Q tiles
constexpr int kSmallAt = kSlotsAt + kSlots * kTile;
constexpr float kLazy = 8.0f;             // log2 slack of the running maximum
constexpr float kLift = 7.0f;             // log2 factor carried by the weights

struct Small {
  float rowscale[256];
  float m1[128], l1[128];                 // stream 1's state on its way to stream 0
  alignas(8) uint64_t full[kSlots], empty[kSlots], s_full[2], p_full[2], o_full[2], drain;
  uint32_t tmem;
  int stop;
};
constexpr size_t kSmem = kSmallAt + sizeof(Small);

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

// Row blocks of a sequence (one for a sequence to be refused, so that a CTA sees it).
__device__ __forceinline__ int attn_blocks(const AttnArgs& a, int s) {
  const AttnSeq q = attn_seq(a, s);
  return q.ok ? (int)(((int64_t)q.n * a.G + 255) / 256) : 1;
}

// What one query row sees: the first `raw` raw tokens (sink, then window) and the first `packed`
// packed ones.
struct Seen {
  int raw, packed;
};
__device__ __forceinline__ Seen row_seen(const AttnArgs& a, const AttnSeq& q, int i) {
  const int ns = a.b.n_sink;
  const int64_t L = (int64_t)ns + q.tq + q.tr;
  const int64_t see = a.causal ? max((int64_t)0, min(L, L - q.n + i + 1)) : L;
  const int64_t behind = see - ns;        // of packed and window tokens
  Seen r;
  r.packed = (int)min(max(behind, (int64_t)0), (int64_t)q.tq);
  r.raw = (int)min(see, (int64_t)ns) + (int)max(behind - q.tq, (int64_t)0);
  return r;
}

struct Cta {
  int s, h;
  int r0, nr;          // its rows of the sequence's n * G
  bool split;          // one half block, tiles dealt to the streams in turn
  int n_raw;           // raw tiles
  int t_lo, N;         // its tiles [t_lo, t_lo + N) of the block's
  int raw, packed;     // tokens its last row sees
};

// ---- producer: codes to fp16 tiles -------------------------------------------------------
__device__ __forceinline__ uint32_t h2sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t h2fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t lo2(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }   // (a.lo, b.lo)
__device__ __forceinline__ uint32_t hi2(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }   // (a.hi, b.hi)
__device__ __forceinline__ void st16(uint32_t addr, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 ldg16(const void* p) { return __ldg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ uint2 ldg8(const void* p) { return __ldg(reinterpret_cast<const uint2*>(p)); }
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// A packed group's keys as thread t of 128 takes them: words 4 (t % 4) .. + 3 (32 channels) of tokens
// t / 4 + 32 j, and those channels' scales and zero-points.
struct KCodes {
  uint4 w[4], s[4], z[4];
};
__device__ __forceinline__ void load_k(const AttnArgs& a, int64_t slab, int t, KCodes& k) {
  const uint8_t* c = reinterpret_cast<const uint8_t*>(a.L.side[0].codes) + slab * a.L.side[0].code_slab_bytes;
  const __half* s = reinterpret_cast<const __half*>(a.L.side[0].scale) + slab * 128 + 32 * (t & 3);
  const __half* z = reinterpret_cast<const __half*>(a.L.side[0].zero) + slab * 128 + 32 * (t & 3);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    k.w[j] = ldg16(c + ((t >> 2) + 32 * j) * 64 + (t & 3) * 16);
    k.s[j] = ldg16(s + 8 * j);
    k.z[j] = ldg16(z + 8 * j);
  }
}
__device__ __forceinline__ void put_k(const KCodes& k, uint32_t slot, int t) {
  const int q = t & 3;
  const uint32_t base = slot + (q >> 1) * 16384;
#pragma unroll
  for (int ii = 0; ii < 4; ++ii) {
    // the eight lanes of a store phase cover two tokens and four quads: quads of one half start
    // two chunks apart, which keeps their 16-byte chunks in different banks
    const uint4 sr = (ii == 0) ? (q < 2 ? k.s[0] : k.s[2]) : (ii == 1) ? (q < 2 ? k.s[1] : k.s[3])
                   : (ii == 2) ? (q < 2 ? k.s[2] : k.s[0]) : (q < 2 ? k.s[3] : k.s[1]);
    const uint4 zr = (ii == 0) ? (q < 2 ? k.z[0] : k.z[2]) : (ii == 1) ? (q < 2 ? k.z[1] : k.z[3])
                   : (ii == 2) ? (q < 2 ? k.z[2] : k.z[0]) : (q < 2 ? k.z[3] : k.z[1]);
    const int i = q < 2 ? ii : (ii + 2) & 3;
    const uint32_t s0 = lo2(sr.x, sr.z), s1 = hi2(sr.x, sr.z), s2 = lo2(sr.y, sr.w), s3 = hi2(sr.y, sr.w);
    const uint32_t z0 = lo2(zr.x, zr.z), z1 = hi2(zr.x, zr.z), z2 = lo2(zr.y, zr.w), z3 = hi2(zr.y, zr.w);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint4 wj = k.w[j];
      const uint32_t w = (ii == 0) ? (q < 2 ? wj.x : wj.z) : (ii == 1) ? (q < 2 ? wj.y : wj.w)
                       : (ii == 2) ? (q < 2 ? wj.z : wj.x) : (q < 2 ? wj.w : wj.y);
      const uint32_t v = w >> 8;
      const int r = (t >> 2) + 32 * j, c = 4 * (q & 1) + i;
      st16(base + r * 128 + ((c ^ (r & 7)) << 4),
           h2fma(h2sub((w & 0x000F000Fu) | 0x64006400u, 0x64006400u), s0, z0),
           h2fma(h2sub((w & 0x00F000F0u) | 0x54005400u, 0x54005400u), s1, z1),
           h2fma(h2sub((v & 0x000F000Fu) | 0x64006400u, 0x64006400u), s2, z2),
           h2fma(h2sub((v & 0x00F000F0u) | 0x54005400u, 0x54005400u), s3, z3));
    }
  }
}

// A packed group's values as thread t takes them: words 2 (t / 16), + 1 (16 channels) of the token octet
// t % 16 (pairs 4 (t % 16) + j), and those tokens' scales and zero-points.
struct VCodes {
  uint2 w[4];
  uint4 s, z;
};
__device__ __forceinline__ void load_v(const AttnArgs& a, int64_t slab, int t, VCodes& v) {
  const uint8_t* c = reinterpret_cast<const uint8_t*>(a.L.side[1].codes) + slab * a.L.side[1].code_slab_bytes;
#pragma unroll
  for (int j = 0; j < 4; ++j) v.w[j] = ldg8(c + (4 * (t & 15) + j) * 64 + (t >> 4) * 8);
  v.s = ldg16(reinterpret_cast<const __half*>(a.L.side[1].scale) + slab * 128 + 8 * (t & 15));
  v.z = ldg16(reinterpret_cast<const __half*>(a.L.side[1].zero) + slab * 128 + 8 * (t & 15));
}
template <uint32_t MASK, uint32_t MAGIC>
__device__ __forceinline__ uint32_t code2(uint32_t w, uint32_t s, uint32_t z) {
  return h2fma(h2sub((w & MASK) | MAGIC, MAGIC), s, z);
}
__device__ __forceinline__ void put_v(const VCodes& v, uint32_t slot, int t, int valid) {
  const int o = t & 15;
  const uint32_t base = slot + (o >> 3) * 16384;
  uint32_t s[4] = {v.s.x, v.s.y, v.s.z, v.s.w}, z[4] = {v.z.x, v.z.y, v.z.z, v.z.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {   // tokens past the group's end count as zero, whatever lies there
    const int left = valid - 8 * o - 2 * j;
    const uint32_t m = left >= 2 ? 0xffffffffu : left == 1 ? 0x0000ffffu : 0u;
    s[j] &= m;
    z[j] &= m;
  }
#pragma unroll
  for (int wi = 0; wi < 2; ++wi) {
    uint32_t w[4], u[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = wi ? v.w[j].y : v.w[j].x;
      u[j] = w[j] >> 8;
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const int r = 16 * (t >> 4) + 8 * wi + c;   // channel
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t y = c < 4 ? w[j] : u[j];
        x[j] = (c & 3) == 0   ? code2<0x00030003u, 0x64006400u>(y, s[j], z[j])
               : (c & 3) == 1 ? code2<0x000C000Cu, 0x5C005C00u>(y, s[j], z[j])
               : (c & 3) == 2 ? code2<0x00300030u, 0x54005400u>(y, s[j], z[j])
                              : code2<0x00C000C0u, 0x4C004C00u>(y, s[j], z[j]);
      }
      st16(base + r * 128 + (((o & 7) ^ (r & 7)) << 4), x[0], x[1], x[2], x[3]);
    }
  }
}

// Eight channels (octet o) of raw token r of sequence s, head h: the sink's rows, then the window's.
// What fp16 cannot hold counts as 0 and is flagged.
__device__ __forceinline__ void raw8(const AttnArgs& a, const Cta& c, int which, int ns, int r, int o, float (&x)[8],
                                     int& flags) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = 0.0f;
  if (r >= c.raw) return;
  const int64_t slab = (int64_t)c.s * a.L.Hkv + c.h;
  if (r < ns) load8(a.sink[which], (slab * a.b.n_sink + r) * 128 + 8 * o, a.L.src_dtype, x);
  else load8(a.res[which], (slab * a.b.res_cap + r - ns) * 128 + 8 * o, a.L.src_dtype, x);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (!(fabsf(x[j]) <= 65504.0f)) {
      flags |= isfinite(x[j]) ? KVQ_DEV_RANGE : KVQ_DEV_NONFINITE;
      x[j] = 0.0f;
    }
  }
}
__device__ __forceinline__ int put_raw_k(const AttnArgs& a, const Cta& c, int ns, int r0, uint32_t slot, int t) {
  int flags = 0;
  const int o = t & 15;
#pragma unroll 4
  for (int j = 0; j < 16; ++j) {
    const int r = (t >> 4) + 8 * j;
    float x[8];
    raw8(a, c, KVQ_KEYS, ns, r0 + r, o, x, flags);
    if (a.L.k_rotate) {   // packed keys and the queries are in the transformed basis
      wht128_octet_unscaled(x, t & 31);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fminf(fmaxf(x[e] * a.L.rot_scale, -65504.0f), 65504.0f);
    }
    st16(slot + (o >> 3) * 16384 + r * 128 + (((o & 7) ^ (r & 7)) << 4), pack_f16(x[0], x[4]), pack_f16(x[1], x[5]),
         pack_f16(x[2], x[6]), pack_f16(x[3], x[7]));
  }
  return flags;
}
__device__ __forceinline__ int put_raw_v(const AttnArgs& a, const Cta& c, int ns, int r0, uint32_t slot, int t) {
  int flags = 0;
  const int o = t & 15;   // token octet
#pragma unroll 1
  for (int b = 0; b < 2; ++b) {
    const int ch = (t >> 4) + 8 * b;
    uint32_t h[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float x[8];
      raw8(a, c, KVQ_VALUES, ns, r0 + 8 * o + j, ch, x, flags);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[j][e] = pack_f16(x[2 * e], x[2 * e + 1]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        y[j] = e & 1 ? hi2(h[2 * j][e / 2], h[2 * j + 1][e / 2]) : lo2(h[2 * j][e / 2], h[2 * j + 1][e / 2]);
      const int r = 8 * ch + e;
      st16(slot + (o >> 3) * 16384 + r * 128 + (((o & 7) ^ (r & 7)) << 4), y[0], y[1], y[2], y[3]);
    }
  }
  return flags;
}

// The ring's order: position p holds the keys or the values of one tile.
__device__ __forceinline__ bool is_value(const Cta& c, int p, int* tile) {
  if (!c.split) {
    *tile = p >> 1;
    return p & 1;
  }
  if (p == 0) { *tile = 0; return false; }
  if (p == 2 * c.N - 1) { *tile = c.N - 1; return true; }
  *tile = p & 1 ? (p + 1) >> 1 : (p >> 1) - 1;
  return !(p & 1);
}

__device__ __forceinline__ void producer(const AttnArgs& a, const Cta& c, const AttnSeq& q, Small* sm, uint32_t ring) {
  const int t = threadIdx.x - 256;
  const int ns = min(a.b.n_sink, (int)min((int64_t)a.b.n_sink, (int64_t)a.b.n_sink + q.tr + q.tq));
  int flags = 0;
  auto slab_of = [&](int tile) -> int64_t {   // packed tile of the block
    const int g = c.t_lo + tile - c.n_raw;
    if (g < 0 || tile >= c.N) return 0;
    int blk = __ldg(a.b.table + (int64_t)c.s * a.b.max_blocks + g);
    if (blk < 0 || blk >= a.b.num_blocks) {
      flags |= KVQ_DEV_BOUNDS;
      blk = 0;
    }
    return (int64_t)blk * a.L.Hkv + c.h;
  };
  KCodes k;
  VCodes v;
  // the pages of the next keys and values, one step ahead of their codes
  const int64_t first = slab_of(0);
  load_k(a, first, t, k);
  load_v(a, first, t, v);
  int64_t next_k = slab_of(1), next_v = next_k;
  for (int p = 0; p < 2 * c.N; ++p) {
    const int slot = p % kSlots, use = p / kSlots;
    int tile;
    const bool value = is_value(c, p, &tile);
    if (use > 0 && !mbar_wait(smem_u32(&sm->empty[slot]), (use - 1) & 1, &sm->stop)) break;
    const uint32_t dst = ring + slot * kTile;
    const int at = c.t_lo + tile;
    if (at < c.n_raw) {
      flags |= value ? put_raw_v(a, c, ns, 128 * at, dst, t) : put_raw_k(a, c, ns, 128 * at, dst, t);
    } else if (value) {
      put_v(v, dst, t, min(128, q.tq - 128 * (at - c.n_raw)));
    } else {
      put_k(k, dst, t);
    }
    fence_async_smem();
    mbar_arrive(smem_u32(&sm->full[slot]));
    if (value) {
      load_v(a, next_v, t, v);
      next_v = slab_of(tile + 2);
    } else {
      load_k(a, next_k, t, k);
      next_k = slab_of(tile + 2);
    }
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (flags && (t & 31) == 0) flag(a.status, flags);
}

// ---- the product-issuing thread -----------------------------------------------------------
__device__ __forceinline__ void issue_qk(uint32_t d, uint32_t q, uint32_t k) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t off = (i >> 2) * 16384 + (i & 3) * 32;
    mma_ss(d, smem_desc(q + off), smem_desc(k + off), i > 0);
  }
}
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t p, uint32_t v, bool accumulate) {
#pragma unroll
  for (int i = 0; i < 8; ++i)
    mma_ts(d, p + 8 * i, smem_desc(v + (i >> 2) * 16384 + (i & 3) * 32), accumulate || i > 0);
}

__device__ __forceinline__ bool products(const Cta& c, Small* sm, uint32_t qs, uint32_t ring, uint32_t tm) {
  volatile int* stop = &sm->stop;
  int pos = 0;   // ring position consumed next
  auto slot = [&](int p) { return ring + (p % kSlots) * kTile; };
  auto full = [&](int p) { return mbar_wait(smem_u32(&sm->full[p % kSlots]), (p / kSlots) & 1, stop); };
  auto freed = [&](int p) { tc_commit(smem_u32(&sm->empty[p % kSlots])); };
  auto weights = [&](int w, int i) {
    const bool ok = mbar_wait(smem_u32(&sm->p_full[w]), i & 1, stop);
    tc_fence_after();
    return ok;
  };
  if (!c.split) {
    if (!full(0)) return false;
    for (int w = 0; w < 2; ++w) {
      issue_qk(tm + 128 * w, qs + w * kTile, slot(0));
      tc_commit(smem_u32(&sm->s_full[w]));
    }
    freed(0);
    for (int i = 0; i < c.N; ++i) {
      const int pv = 2 * i + 1, pk = pv + 1;
      for (int w = 0; w < 2; ++w) {
        if (!weights(w, i)) return false;
        if (w == 0 && !full(pv)) return false;
        issue_pv(tm + 256 + 128 * w, tm + 128 * w, slot(pv), i > 0);
        if (w == 1) freed(pv);
        if (i + 1 < c.N) {
          if (w == 0 && !full(pk)) return false;
          issue_qk(tm + 128 * w, qs + w * kTile, slot(pk));
          tc_commit(smem_u32(&sm->s_full[w]));
          if (w == 1) freed(pk);
        } else {
          tc_commit(smem_u32(&sm->o_full[w]));
        }
      }
    }
    return true;
  }
  for (int w = 0; w < 2 && w < c.N; ++w, ++pos) {
    if (!full(pos)) return false;
    issue_qk(tm + 128 * w, qs, slot(pos));
    tc_commit(smem_u32(&sm->s_full[w]));
    freed(pos);
  }
  for (int t = 0; t < c.N; ++t) {
    const int w = t & 1;
    if (!weights(w, t >> 1) || !full(pos)) return false;
    issue_pv(tm + 256 + 128 * w, tm + 128 * w, slot(pos), t > 1);
    freed(pos++);
    if (t + 2 < c.N) {
      if (!full(pos)) return false;
      issue_qk(tm + 128 * w, qs, slot(pos));
      tc_commit(smem_u32(&sm->s_full[w]));
      freed(pos++);
    } else {
      tc_commit(smem_u32(&sm->o_full[w]));
    }
  }
  return true;
}

// ---- softmax ---------------------------------------------------------------------------------
__device__ __forceinline__ void pin32(uint32_t* r) {   // orders uses of r after the wait before it
#pragma unroll
  for (int j = 0; j < 32; ++j) asm volatile("" : "+r"(r[j]));
}

// Stream w's tiles; row of this thread: m (log2), l on return.
__device__ __forceinline__ bool softmax(const Cta& c, Small* sm, uint32_t s_col, uint32_t o_col, int w, Seen see,
                                        float cs, float* m_out, float* l_out) {
  float m = -INFINITY, l = 0.0f;
  const int n = c.split ? (c.N - w + 1) / 2 : c.N;
  bool ok = true;
  for (int i = 0; i < n; ++i) {
    if (!mbar_wait(smem_u32(&sm->s_full[w]), i & 1, &sm->stop)) { ok = false; break; }
    tc_fence_after();
    uint32_t x[128];
#pragma unroll
    for (int k = 0; k < 4; ++k) tmem_ld32(s_col + 32 * k, x + 32 * k);
    tmem_wait_ld();
#pragma unroll
    for (int k = 0; k < 4; ++k) pin32(x + 32 * k);
    const int at = c.t_lo + (c.split ? 2 * i + w : i);
    const int cols = at < c.n_raw ? see.raw - 128 * at : see.packed - 128 * (at - c.n_raw);
    if (__any_sync(0xffffffffu, cols < 128)) {
#pragma unroll
      for (int j = 0; j < 128; ++j)
        if (j >= cols) x[j] = 0xff800000u;   // -inf
    }
    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
    for (int j = 0; j < 128; j += 4)
#pragma unroll
      for (int e = 0; e < 4; ++e) mx[e] = fmaxf(mx[e], __uint_as_float(x[j + e]));
    const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * cs;
    const bool move = top > m + kLazy;       // true from -inf for any finite score
    if (__any_sync(0xffffffffu, move)) {
      const float mn = move ? top : m;
      const float f = move ? exp2_approx(m - mn) : 1.0f;
      l *= f;
      m = mn;
      if (i > 0) {
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          uint32_t o[32];
          tmem_ld32(o_col + 32 * k, o);
          tmem_wait_ld();
          pin32(o);
#pragma unroll
          for (int j = 0; j < 32; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
          tmem_st32(o_col + 32 * k, o);
        }
      }
    }
    const float off = kLift - (m == -INFINITY ? 0.0f : m);
    float sum[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      uint32_t h[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float p0 = exp2_approx(fmaf(__uint_as_float(x[32 * k + 2 * j]), cs, off));
        const float p1 = exp2_approx(fmaf(__uint_as_float(x[32 * k + 2 * j + 1]), cs, off));
        sum[(2 * j) & 3] += p0;
        sum[(2 * j + 1) & 3] += p1;
        h[j] = pack_f16(p0, p1);
      }
      tmem_st16(s_col + 16 * k, h);
    }
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    tmem_wait_st();
    tc_fence_before();
    mbar_arrive(smem_u32(&sm->p_full[w]));
  }
  *m_out = m;
  *l_out = l;
  return ok;
}

struct Plan {
  int splits;       // runs of tiles of a block (grid z), each `tiles` long
  int tiles;
  int64_t rows;     // n_rows * Hq
  float* m;         // [splits][rows], for splits > 1
  float* l;
  float* o;         // [splits][rows][128]
};

// One row's state to where it goes: the output, or the slot of this run of tiles.
__device__ __forceinline__ void put_state(const AttnArgs& a, const Plan& p, int64_t row, int z, float m, float l) {
  if (p.splits > 1) {
    p.m[z * p.rows + row] = m;
    p.l[z * p.rows + row] = l;
  } else if (a.lse) {
    a.lse[row] = l > 0.0f ? kLn2 * (m + log2f(l) - kLift) : -INFINITY;
  }
}
__device__ __forceinline__ void put_out(const AttnArgs& a, const Plan& p, int64_t row, int z, int c0, const float* x,
                                        float inv) {
  if (p.splits > 1) {
    float4* d = reinterpret_cast<float4*>(p.o + (z * p.rows + row) * 128 + c0);
#pragma unroll
    for (int j = 0; j < 8; ++j) d[j] = make_float4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]);
  } else if (a.out_dtype == KVQ_F32) {
    float4* d = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + row * 128 + c0);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      d[j] = make_float4(x[4 * j] * inv, x[4 * j + 1] * inv, x[4 * j + 2] * inv, x[4 * j + 3] * inv);
  } else {
    uint4* d = reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(a.out) + row * 128 + c0);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t h[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float u = x[8 * j + 2 * e] * inv, v = x[8 * j + 2 * e + 1] * inv;
        if (a.out_dtype == KVQ_F16) {
          h[e] = pack_f16(u, v);
        } else {
          const __nv_bfloat162 b2 = __floats2bfloat162_rn(u, v);
          h[e] = *reinterpret_cast<const uint32_t*>(&b2);
        }
      }
      d[j] = make_uint4(h[0], h[1], h[2], h[3]);
    }
  }
}

template <uint32_t N>
__device__ __forceinline__ void regs_more() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <uint32_t N>
__device__ __forceinline__ void regs_fewer() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }

// Grid (row blocks of all sequences, KV heads, runs of tiles).
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const __grid_constant__ AttnArgs a,
                                                              const __grid_constant__ Plan plan) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Small* sm = reinterpret_cast<Small*>(smem + kSmallAt);
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  Cta c;
  int unit;
  if (!find_unit(a.b.num_seqs, blockIdx.x, [&](int s) { return attn_blocks(a, s); }, &c.s, &unit)) return;
  const AttnSeq q = attn_seq(a, c.s);
  if (!q.ok) {
    if (blockIdx.y == 0 && blockIdx.z == 0 && threadIdx.x == 0) flag(a.status, KVQ_DEV_BOUNDS);
    return;
  }
  c.h = blockIdx.y;
  const int64_t all = (int64_t)q.n * a.G;
  unit = (int)((all + 255) / 256) - 1 - unit;     // blocks that see the most go first
  c.r0 = unit * 256;
  c.nr = (int)min((int64_t)256, all - c.r0);
  c.split = c.nr <= 128;
  const Seen last = row_seen(a, q, (c.r0 + c.nr - 1) / a.G);
  c.raw = last.raw;
  c.packed = last.packed;
  c.n_raw = (c.raw + 127) / 128;
  const int tiles = c.n_raw + (c.packed + 127) / 128;
  c.t_lo = blockIdx.z * plan.tiles;
  c.N = min(tiles, c.t_lo + plan.tiles) - c.t_lo;
  // row r of the block: token r / G of the chunk, query head h G + r % G
  auto out_row = [&](int r) { return (q.row0 + (c.r0 + r) / a.G) * a.Hq + c.h * a.G + (c.r0 + r) % a.G; };
  if (c.N <= 0) {   // nothing here to see
    if (plan.splits > 1 || tiles == 0) {
      for (int r = threadIdx.x; r < c.nr; r += kThreads) {
        const int64_t row = out_row(r);
        put_state(a, plan, row, blockIdx.z, -INFINITY, 0.0f);
        if (plan.splits == 1) {
          const float zero[32] = {};
          for (int k = 0; k < 4; ++k) put_out(a, plan, row, 0, 32 * k, zero, 0.0f);
        }
      }
    }
    return;
  }

  const uint32_t qs = smem_u32(smem), ring = qs + kSlotsAt;
  if (warp == 12) tmem_alloc(smem_u32(&sm->tmem), 512);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&sm->full[i]), 128);
      mbar_init(smem_u32(&sm->empty[i]), 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(smem_u32(&sm->s_full[w]), 1);
      mbar_init(smem_u32(&sm->p_full[w]), 128);
      mbar_init(smem_u32(&sm->o_full[w]), 1);
    }
    mbar_init(smem_u32(&sm->drain), 1);
    sm->stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  // queries: a warp per row, four channels per lane; scaled so that the row's largest lies in [2^8, 2^9)
  bool bad = false;
  for (int r = warp; r < (c.split ? 128 : 256); r += kThreads / 32) {
    float x[4] = {0, 0, 0, 0};
    if (r < c.nr) {
      const int64_t e = out_row(r) * 128 + 4 * lane;
      if (a.q_dtype == KVQ_F32) {
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.q) + e);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(a.q) + e);
        const uint32_t w[2] = {v.x, v.y};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          if (a.q_dtype == KVQ_F16) {
            x[2 * j] = half_bits_to_float((uint16_t)(w[j] & 0xffffu));
            x[2 * j + 1] = half_bits_to_float((uint16_t)(w[j] >> 16));
          } else {
            x[2 * j] = __uint_as_float(w[j] << 16);
            x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
          }
        }
      }
    }
    bad |= !(isfinite(x[0]) && isfinite(x[1]) && isfinite(x[2]) && isfinite(x[3]));
    if (a.L.k_rotate) {
      wht128_quad_unscaled(x, lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] *= a.L.rot_scale;
    }
    const float top = warp_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
    // 2^e <= top < 2^(e + 1); rows of zeros, subnormal or overflowing rows get the nearest e that serves
    const int e = min(max((int)(__float_as_uint(top) >> 23), 10), 250);
    const float up = __uint_as_float((uint32_t)(262 - e) << 23);   // 2^(8 - (e - 127))
    if (lane == 0) sm->rowscale[r] = __uint_as_float((uint32_t)(e - 8) << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] *= up;
    const bool odd = lane & 1;
    const float y0 = __shfl_xor_sync(0xffffffffu, odd ? x[0] : x[2], 1);
    const float y1 = __shfl_xor_sync(0xffffffffu, odd ? x[1] : x[3], 1);
    const uint32_t h0 = odd ? pack_f16(y0, x[2]) : pack_f16(x[0], y0);
    const uint32_t h1 = odd ? pack_f16(y1, x[3]) : pack_f16(x[1], y1);
    const int o = lane >> 1;
    const uint32_t at = qs + (r >> 7) * kTile + (o >> 3) * 16384 + (r & 127) * 128 + (((o & 7) ^ (r & 7)) << 4) + 8 * odd;
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(at), "r"(h0), "r"(h1) : "memory");
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) flag(a.status, KVQ_DEV_NONFINITE);
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = sm->tmem;

  if (warp < 8) {
    regs_more<184>();
    const int w = warp >> 2, t = threadIdx.x & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // lane 32 (warp % 4) in the address's upper half
    const int r = c.split ? t : 128 * w + t;
    Seen see = {0, 0};
    if (r < c.nr) see = row_seen(a, q, (c.r0 + r) / a.G);
    // never 0, so that a masked score of -inf stays one
    const float cs = fmaxf(a.qscale * sm->rowscale[r], 1.2e-38f);
    const uint32_t o_col = tm + lanes + 256 + 128 * w;
    float m, l;
    bool ok = softmax(c, sm, tm + lanes + 128 * w, o_col, w, see, cs, &m, &l);
    const bool two = c.split && c.N > 1;                  // two states per row to merge
    if (ok && (w == 0 || c.N > 1 || !c.split)) ok = mbar_wait(smem_u32(&sm->o_full[w]), 0, &sm->stop);
    if (two && w == 1) {
      // the other stream's products may still read the ring
      if (ok) ok = mbar_wait(smem_u32(&sm->o_full[0]), 0, &sm->stop);
      tc_fence_after();
      if (ok) {
        sm->m1[t] = m;
        sm->l1[t] = l;
        float4* d = reinterpret_cast<float4*>(smem + kSlotsAt) + t * 32;
#pragma unroll 1
        for (int k = 0; k < 4; ++k) {
          uint32_t o[32];
          tmem_ld32(o_col + 32 * k, o);
          tmem_wait_ld();
          pin32(o);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            d[(8 * k + j) ^ lane] = make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                                                __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
        }
      }
    }
    if (two) asm volatile("bar.sync 1, 256;" ::: "memory");
    if (ok && (w == 0 || !c.split)) {
      tc_fence_after();
      float f0 = 1.0f, f1 = 0.0f;
      if (two) {
        const float m1 = sm->m1[t], l1 = sm->l1[t], mm = fmaxf(m, m1);
        f0 = m == -INFINITY ? 0.0f : exp2_approx(m - mm);
        f1 = m1 == -INFINITY ? 0.0f : exp2_approx(m1 - mm);
        l = l * f0 + l1 * f1;
        m = mm;
      }
      const float inv = l > 0.0f ? 1.0f / l : 0.0f;
      const int64_t row = r < c.nr ? out_row(r) : 0;
      if (r < c.nr) put_state(a, plan, row, blockIdx.z, m, l);
      const float4* d = reinterpret_cast<const float4*>(smem + kSlotsAt) + t * 32;
#pragma unroll 1
      for (int k = 0; k < 4; ++k) {
        uint32_t o[32];
        float x[32];
        tmem_ld32(o_col + 32 * k, o);
        tmem_wait_ld();
        pin32(o);
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(o[j]);
        if (two) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float4 v = d[(8 * k + j) ^ lane];
            x[4 * j] = x[4 * j] * f0 + v.x * f1;
            x[4 * j + 1] = x[4 * j + 1] * f0 + v.y * f1;
            x[4 * j + 2] = x[4 * j + 2] * f0 + v.z * f1;
            x[4 * j + 3] = x[4 * j + 3] * f0 + v.w * f1;
          }
        }
        if (r < c.nr) put_out(a, plan, row, blockIdx.z, 32 * k, x, inv);
      }
    }
  } else if (warp < 12) {
    regs_fewer<104>();
    producer(a, c, q, sm, ring);
  } else {
    regs_fewer<40>();
    if (warp == 12 && lane == 0 && !products(c, sm, qs, ring, tm)) {
      // stopped: what was issued still has to end before its memory is given up
      flag(a.status, KVQ_DEV_TIMEOUT);
      tc_commit(smem_u32(&sm->drain));
      int never = 0;
      mbar_wait(smem_u32(&sm->drain), 0, &never);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) tmem_free(tm, 512);
}

// Merge of the runs of tiles: a warp per row, four channels per lane.
__global__ void __launch_bounds__(256) attn_merge_kernel(const __grid_constant__ AttnArgs a,
                                                         const __grid_constant__ Plan plan) {
  griddep_wait();
  griddep_launch_dependents();
  int s, unit;
  if (!find_unit(a.b.num_seqs, blockIdx.x, [&](int i) { return attn_blocks(a, i); }, &s, &unit)) return;
  const AttnSeq q = attn_seq(a, s);
  if (!q.ok) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t all = (int64_t)q.n * a.G;
  for (int64_t r = unit * 256 + warp; r < min(all, (int64_t)unit * 256 + 256); r += 8) {
    const int64_t row = (q.row0 + r / a.G) * a.Hq + blockIdx.y * a.G + r % a.G;
    float m = -INFINITY;
    for (int z = lane; z < plan.splits; z += 32) m = fmaxf(m, plan.m[z * plan.rows + row]);
    m = warp_max(m);
    float l = 0.0f, o[4] = {0, 0, 0, 0};
    for (int z = 0; z < plan.splits; ++z) {
      const float mz = plan.m[z * plan.rows + row];
      if (mz == -INFINITY) continue;
      const float f = exp2_approx(mz - m);
      l += f * plan.l[z * plan.rows + row];
      const float4 v = *reinterpret_cast<const float4*>(plan.o + (z * plan.rows + row) * 128 + 4 * lane);
      o[0] += f * v.x;
      o[1] += f * v.y;
      o[2] += f * v.z;
      o[3] += f * v.w;
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) store_elem(a.out, row * 128 + 4 * lane + j, a.out_dtype, o[j] * inv);
    if (a.lse && lane == 0) a.lse[row] = l > 0.0f ? kLn2 * (m + log2f(l) - kLift) : -INFINITY;
  }
}

int64_t row_blocks(int num_seqs, int G, int64_t n_rows) { return n_rows * G / 256 + num_seqs; }

// Runs of tiles: enough CTAs for two per SM when the row blocks alone do not give them, at least four
// tiles each.
Plan make_plan(int num_seqs, int Hq, int Hkv, int64_t n_rows, int64_t max_new, int64_t max_tq, int max_tr, int ns) {
  const int G = Hq / Hkv;
  const int64_t per_seq = (max_new * G + 255) / 256;
  const int64_t blocks = row_blocks(num_seqs, G, n_rows) < per_seq * num_seqs ? row_blocks(num_seqs, G, n_rows)
                                                                              : per_seq * num_seqs;
  const int64_t ctas = blocks * Hkv, tiles = (max_tq + 127) / 128 + (ns + max_tr + 127) / 128;
  const int64_t want = 2 * device_sm_count();
  Plan p = {};
  p.rows = n_rows * Hq;
  p.tiles = (int)tiles;
  if (ctas < want) {
    const int64_t t = (ctas * tiles + want - 1) / want;
    p.tiles = (int)(t < 4 ? 4 : t);
  }
  if (p.tiles < 1) p.tiles = 1;
  p.splits = (int)((tiles + p.tiles - 1) / p.tiles);
  if (p.splits < 1) p.splits = 1;
  return p;
}

size_t pad16(size_t n) { return (n + 15) & ~(size_t)15; }

}  // namespace

size_t attn_paged_workspace(int num_seqs, int Hq, int Hkv, int64_t n_rows, int64_t max_new, int64_t max_t_quant,
                            int max_t_res, int n_sink) {
  const Plan p = make_plan(num_seqs, Hq, Hkv, n_rows, max_new, max_t_quant, max_t_res, n_sink);
  if (p.splits == 1) return 16;
  return 2 * pad16((size_t)p.splits * p.rows * 4) + (size_t)p.splits * p.rows * 512;
}

cudaError_t launch_attn_paged(const AttnArgs& a, cudaStream_t s) {
  Plan p = make_plan(a.b.num_seqs, a.Hq, a.L.Hkv, a.b.n_rows, a.b.max_rows, a.max_t_quant, a.max_t_res, a.b.n_sink);
  const size_t part = pad16((size_t)p.splits * p.rows * 4);
  p.m = reinterpret_cast<float*>(a.ws);
  p.l = reinterpret_cast<float*>(reinterpret_cast<char*>(a.ws) + part);
  p.o = reinterpret_cast<float*>(reinterpret_cast<char*>(a.ws) + 2 * part);
  const unsigned blocks = (unsigned)row_blocks(a.b.num_seqs, a.G, a.b.n_rows);
  cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_tc_kernel, dim3(blocks, a.L.Hkv, p.splits), dim3(kThreads), kSmem, s, a, p);
  if (e != cudaSuccess || p.splits == 1) return e;
  return launch_pdl(attn_merge_kernel, dim3(blocks, a.L.Hkv), dim3(256), 0, s, a, p);
}

}  // namespace kvq
