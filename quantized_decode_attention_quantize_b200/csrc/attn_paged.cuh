// Shared by the two chunk-attention kernels: the partition of the work, the expansion of codes to
// fp16 tiles, the order of the products, and the softmax arithmetic.
#pragma once

#include "paged_batch.cuh"
#include "tc05.cuh"
#include "wht.cuh"

namespace kvq {
namespace attn {

constexpr float kLn2 = 0.6931471805599453f;
constexpr int kTile = 32768;              // 128 x 128 fp16
constexpr int kSlots = 4;
constexpr int kSlotsAt = 2 * kTile;       // after the two Q tiles
constexpr int kStagesAt = kSlotsAt + kSlots * kTile;
constexpr int kSegs = 2;                  // announced blocks
constexpr float kLazy = 8.0f;             // log2 slack of the running maximum
constexpr float kLift = 7.0f;             // log2 factor carried by the weights
constexpr int kMinRun = 2;                // units of a run at least

// The part of a block that this CTA does.
struct Seg {
  int64_t row0;        // the sequence's first query row
  int s, h, n, tq, tr;
  int r0, nr;          // rows of the block within the sequence's n * G
  int split;           // one half block, tiles dealt to the streams in turn
  int n_raw;           // raw tiles of the block
  int t_lo, N;         // tiles [t_lo, t_lo + N); N = 0: nothing to see; N < 0: no more blocks
  int raw, packed;     // tokens the block's last row sees
  int slot;            // partial slot, or -1 for the output itself
};

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


// What one query row sees: the first `raw` raw tokens (sink, then window) and the first `packed`
// packed ones.
struct Seen {
  int raw, packed;
};
__device__ __forceinline__ Seen row_seen(const AttnArgs& a, const AttnSeq& q, int i) {
  const int ns = a.b.n_sink, L = ns + q.tq + q.tr;   // the host keeps all of these below 2^31
  const int see = a.causal ? max(0, min(L, L - q.n + i + 1)) : L;
  const int behind = see - ns;            // of packed and window tokens
  Seen r;
  r.packed = min(max(behind, 0), q.tq);
  r.raw = min(see, ns) + max(behind - q.tq, 0);
  return r;
}

// Row blocks of a sequence and the KV tiles the last row of block b sees.
__device__ __forceinline__ int seq_blocks(const AttnArgs& a, const AttnSeq& q) {
  return (q.n * a.G + a.block - 1) / a.block;
}
__device__ __forceinline__ int block_tiles(const AttnArgs& a, const AttnSeq& q, int b) {
  const Seen v = row_seen(a, q, (min(q.n * a.G, (b + 1) * a.block) - 1) / a.G);
  return (v.raw + a.raw_tile - 1) / a.raw_tile + ((v.packed + 127) >> 7);
}

// ---- the partition (one warp) ----------------------------------------------------------------
// Units of a sequence's blocks (per KV head): tiles + 1 each.  `q` differs from lane to lane.
static __device__ __noinline__ int64_t seq_units(const AttnArgs& a, const AttnSeq& q, int lane) {
  const int nb = q.ok ? seq_blocks(a, q) : 0;
  int64_t w = nb == 1 ? block_tiles(a, q, 0) + 1 : 0;
  unsigned many = __ballot_sync(0xffffffffu, nb > 1);
  while (many) {   // sequences of several blocks: a lane per block
    const int l = __ffs(many) - 1;
    many &= many - 1;
    AttnSeq o = q;
    o.n = __shfl_sync(0xffffffffu, q.n, l);
    o.tq = __shfl_sync(0xffffffffu, q.tq, l);
    o.tr = __shfl_sync(0xffffffffu, q.tr, l);
    const int ob = seq_blocks(a, o);
    int64_t sum = 0;
    for (int b = lane; b < ob; b += 32) sum += block_tiles(a, o, b) + 1;
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
    if (lane == l) w = sum;
  }
  return w;
}
__device__ __forceinline__ int64_t scan64(int64_t v, int lane) {   // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// All units, and the number of runs they are cut into: the first `longer` of them one unit longer than `each`.
struct Cut {
  int64_t units, each;
  int runs, longer;
};
__device__ __forceinline__ int64_t run_start(const Cut& c, int i) { return c.each * i + min(i, c.longer); }
// q0, w0: the lane's sequence and its units among the first 32 (all, most often), for find_place.
__device__ __forceinline__ Cut find_cut(const AttnArgs& a, int runs, int lane, AttnSeq* q0, int64_t* w0) {
  int64_t total = 0;
  bool bad = false;
  for (int s0 = 0; s0 < a.b.num_seqs; s0 += 32) {
    AttnSeq q = {};
    if (s0 + lane < a.b.num_seqs) {
      q = attn_seq(a, s0 + lane);
      bad |= !q.ok;
    }
    const int64_t w = seq_units(a, q, lane);
    if (s0 == 0) {
      *q0 = q;
      *w0 = w;
    }
    total += __shfl_sync(0xffffffffu, scan64(w, lane), 31);
  }
  if (blockIdx.x == 0 && __any_sync(0xffffffffu, bad) && lane == 0) flag(a.status, KVQ_DEV_BOUNDS);
  Cut c;
  c.units = total * a.L.Hkv;
  c.runs = (int)max((int64_t)1, min((int64_t)runs, c.units / kMinRun));
  c.each = c.units / c.runs;
  c.longer = (int)(c.units - c.each * c.runs);
  return c;
}

// A place in the list of blocks: sequence s, its block b (the last, which sees the most, comes first), head h.
struct Place {
  AttnSeq q;
  int s, b, h;
};
__device__ __forceinline__ bool next_seq(const AttnArgs& a, Place* p) {   // the first from p->s on that has rows
  for (; p->s < a.b.num_seqs; ++p->s) {
    p->q = attn_seq(a, p->s);
    if (p->q.ok && p->q.n > 0) {
      p->b = seq_blocks(a, p->q) - 1;
      p->h = 0;
      return true;
    }
  }
  return false;
}
__device__ __forceinline__ bool next_block(const AttnArgs& a, Place* p) {
  if (++p->h < a.L.Hkv) return true;
  p->h = 0;
  if (--p->b >= 0) return true;
  ++p->s;
  return next_seq(a, p);
}
// The block that holds unit `at`, and the unit's index in it.
__device__ __forceinline__ Place find_place(const AttnArgs& a, int64_t at, int lane, const AttnSeq& q0, int64_t w0,
                                            int64_t* unit) {
  Place p = {};
  for (int s0 = 0; s0 < a.b.num_seqs; s0 += 32) {
    AttnSeq q = q0;
    int64_t w = w0;
    if (s0 > 0) {
      q = {};
      if (s0 + lane < a.b.num_seqs) q = attn_seq(a, s0 + lane);
      w = seq_units(a, q, lane);
    }
    w *= a.L.Hkv;
    const int64_t incl = scan64(w, lane);
    const unsigned hit = __ballot_sync(0xffffffffu, at < incl);
    if (hit) {
      const int l = __ffs(hit) - 1;
      at -= __shfl_sync(0xffffffffu, incl - w, l);
      p.s = s0 + l;
      p.q.row0 = __shfl_sync(0xffffffffu, q.row0, l);
      p.q.n = __shfl_sync(0xffffffffu, q.n, l);
      p.q.tq = __shfl_sync(0xffffffffu, q.tq, l);
      p.q.tr = __shfl_sync(0xffffffffu, q.tr, l);
      p.q.ok = true;
      break;
    }
    at -= __shfl_sync(0xffffffffu, incl, 31);
  }
  const int nb = seq_blocks(a, p.q);
  for (int b0 = nb - 1;; b0 -= 32) {   // lanes take blocks b0, b0 - 1, ...
    const int64_t w = b0 - lane >= 0 ? (int64_t)(block_tiles(a, p.q, b0 - lane) + 1) * a.L.Hkv : 0;
    const int64_t incl = scan64(w, lane);
    const unsigned hit = __ballot_sync(0xffffffffu, at < incl);
    if (hit || b0 < 32) {
      const int l = hit ? __ffs(hit) - 1 : b0;
      at -= __shfl_sync(0xffffffffu, incl - w, l);
      p.b = b0 - l;
      const int one = block_tiles(a, p.q, p.b) + 1;
      p.h = (int)(at / one);
      *unit = at - (int64_t)p.h * one;
      return p;
    }
    at -= __shfl_sync(0xffffffffu, incl, 31);
  }
}

// The workspace: the cut, every run's first block, and two partial slots per run (2 i: the rest of a block
// that an earlier run began; 2 i + 1: the beginning of one that run i does not finish).
struct First {
  int64_t row0;
  int h, r0, nr, pad;
  int64_t unit, units;   // where in its block the run starts, and the block's units
};
struct Work {
  Cut* cut;
  First* first;
  int runs;              // at most
  int rows;              // of a slot
  float* m;              // [slots][rows]
  float* l;
  float* o;              // [slots][rows][128]
};

// ---- producers: codes to fp16 tiles ------------------------------------------------------------
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
__device__ __forceinline__ uint32_t pack_f16(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Two codes of w under MASK, whose bit positions MAGIC's exponents make units, times s plus z.
template <uint32_t MASK, uint32_t MAGIC>
__device__ __forceinline__ uint32_t code2(uint32_t w, uint32_t s, uint32_t z) {
  return h2fma(h2sub((w & MASK) | MAGIC, MAGIC), s, z);
}

// All ones in the halves of x that hold finite numbers.
__device__ __forceinline__ uint32_t finite2(uint32_t x) {
  const __half2 h = __habs2(*reinterpret_cast<const __half2*>(&x));
  return __hle2_mask(h, __half2half2(__ushort_as_half(0x7BFF)));
}
// The largest fp16 number of the sign in place of an infinity.
__device__ __forceinline__ uint32_t cap2(uint32_t x) {
  const __half2 top = __half2half2(__ushort_as_half(0x7BFF));
  const __half2 h = __hmax2(__hmin2(*reinterpret_cast<const __half2*>(&x), top), __hneg2(top));
  return *reinterpret_cast<const uint32_t*>(&h);
}
constexpr uint32_t kFifteen2 = 0x4B804B80u, kThree2 = 0x42004200u;   // the largest codes, as fp16 pairs

// The expansions below form c s + z in fp16.  A scale and a zero-point that fit fp16 can still give numbers beyond
// it (bf16 and fp32 sources, and fp16 ones that span all of it: 3 s + z = 65536), and an infinity would reach every
// row of the tile, a weight of 0 included.  The numbers of a channel or token lie between z and c s + z of the
// largest code, so that one tells whether all are finite.  A thread that finds one which is not writes its part
// again by the capped form, which counts what has an infinity or NaN in its metadata as zero and other numbers beyond
// fp16 as its largest one, and raises KVQ_DEV_RANGE.  The capped forms stand apart, behind the usual stores: within
// them they cost the usual tiles more (128 rows of 8 sequences over 16384: 218 us, against 193 without any check).
static __device__ __noinline__ void put_keys_capped(const void* codes, const void* scale, const void* zero, uint32_t slot,
                                                    int t) {
  const int o = t & 15, r = t >> 4;
  const uint4 s = reinterpret_cast<const uint4*>(scale)[o], z = reinterpret_cast<const uint4*>(zero)[o];
  uint32_t sp[4] = {lo2(s.x, s.z), hi2(s.x, s.z), lo2(s.y, s.w), hi2(s.y, s.w)};
  uint32_t zp[4] = {lo2(z.x, z.z), hi2(z.x, z.z), lo2(z.y, z.w), hi2(z.y, z.w)};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t m = finite2(sp[k]) & finite2(zp[k]);
    sp[k] &= m;
    zp[k] &= m;
  }
#pragma unroll 1
  for (int j = 0; j < 16; ++j) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(codes)[t + 128 * j];
    uint32_t x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = cap2(code2<0x000F000Fu, 0x64006400u>(w >> (4 * k), sp[k], zp[k]));
    st16(slot + (o >> 3) * 16384 + (r + 8 * j) * 128 + (((o & 7) ^ r) << 4), x[0], x[1], x[2], x[3]);
  }
}
// All ones in the halves of token pair `pair` that lie before token `valid`.
__device__ __forceinline__ uint32_t tokens2(int pair, int valid) {
  const int left = valid - 2 * pair;
  return left >= 2 ? 0xffffffffu : left == 1 ? 0x0000ffffu : 0u;
}
static __device__ __noinline__ void put_values_capped(const void* codes, const void* scale, const void* zero, uint32_t slot,
                                                      int t, int valid) {
  const int W = t & 15;
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    const int o = (t >> 4) + 8 * half;
    uint32_t s[4], z[4], w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = reinterpret_cast<const uint32_t*>(codes)[64 * o + 16 * j + W];
      s[j] = reinterpret_cast<const uint32_t*>(scale)[4 * o + j];
      z[j] = reinterpret_cast<const uint32_t*>(zero)[4 * o + j];
      const uint32_t m = tokens2(4 * o + j, valid) & finite2(s[j]) & finite2(z[j]);
      s[j] &= m;
      z[j] &= m;
    }
#pragma unroll 1
    for (int e = 0; e < 8; ++e) {
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[j] = cap2(code2<0x00030003u, 0x64006400u>(w[j] >> (2 * (e & 3) + 8 * (e >> 2)), s[j], z[j]));
      st16(slot + half * 16384 + W * 128 + (((t >> 4) ^ (W & 7)) << 4) + 2048 * e, x[0], x[1], x[2], x[3]);
    }
  }
}

// A packed group's keys: thread t of 128 takes octet t % 16 (one word) of tokens t / 16 + 8 j.  The eight
// lanes of a store phase hold eight octets of one token, whose chunks lie in different banks.
__device__ __forceinline__ int put_keys(const void* codes, const void* scale, const void* zero, uint32_t slot, int t) {
  const int o = t & 15, r = t >> 4;
  const uint4 s = reinterpret_cast<const uint4*>(scale)[o], z = reinterpret_cast<const uint4*>(zero)[o];
  const uint32_t* w = reinterpret_cast<const uint32_t*>(codes) + t;
  const uint32_t at = slot + (o >> 3) * 16384 + r * 128 + (((o & 7) ^ r) << 4);
  const uint32_t s0 = lo2(s.x, s.z), s1 = hi2(s.x, s.z), s2 = lo2(s.y, s.w), s3 = hi2(s.y, s.w);
  const uint32_t z0 = lo2(z.x, z.z), z1 = hi2(z.x, z.z), z2 = lo2(z.y, z.w), z3 = hi2(z.y, z.w);
  const uint32_t fits = finite2(h2fma(kFifteen2, s0, z0)) & finite2(h2fma(kFifteen2, s1, z1)) &
                        finite2(h2fma(kFifteen2, s2, z2)) & finite2(h2fma(kFifteen2, s3, z3));
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t x = w[128 * j], y = x >> 8;
    st16(at + 1024 * j, code2<0x000F000Fu, 0x64006400u>(x, s0, z0), code2<0x00F000F0u, 0x54005400u>(x, s1, z1),
         code2<0x000F000Fu, 0x64006400u>(y, s2, z2), code2<0x00F000F0u, 0x54005400u>(y, s3, z3));
  }
  if (fits == 0xffffffffu) return 0;
  put_keys_capped(codes, scale, zero, slot, t);
  return KVQ_DEV_RANGE;
}
// A packed group's values: thread t takes word W = t % 16 (eight channels) of the token octets t / 16 and
// t / 16 + 8.  Tokens past the group's end count as zero, whatever lies there.
__device__ __forceinline__ int put_values(const void* codes, const void* scale, const void* zero, uint32_t slot, int t,
                                          int valid) {
  const int W = t & 15;
  uint32_t fits = 0xffffffffu;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int o = (t >> 4) + 8 * half;
    const uint4 sv = reinterpret_cast<const uint4*>(scale)[o], zv = reinterpret_cast<const uint4*>(zero)[o];
    uint32_t s[4] = {sv.x, sv.y, sv.z, sv.w}, z[4] = {zv.x, zv.y, zv.z, zv.w}, w[4];
    const uint32_t* c = reinterpret_cast<const uint32_t*>(codes) + 64 * o + W;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = c[16 * j];
      const uint32_t m = tokens2(4 * o + j, valid);
      s[j] &= m;
      z[j] &= m;
      fits &= finite2(h2fma(kThree2, s[j], z[j]));
    }
    const uint32_t at = slot + half * 16384 + W * 128 + (((t >> 4) ^ (W & 7)) << 4);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t y = e < 4 ? w[j] : w[j] >> 8;
        x[j] = (e & 3) == 0   ? code2<0x00030003u, 0x64006400u>(y, s[j], z[j])
               : (e & 3) == 1 ? code2<0x000C000Cu, 0x5C005C00u>(y, s[j], z[j])
               : (e & 3) == 2 ? code2<0x00300030u, 0x54005400u>(y, s[j], z[j])
                              : code2<0x00C000C0u, 0x4C004C00u>(y, s[j], z[j]);
      }
      st16(at + 2048 * e, x[0], x[1], x[2], x[3]);
    }
  }
  if (fits == 0xffffffffu) return 0;
  put_values_capped(codes, scale, zero, slot, t, valid);
  return KVQ_DEV_RANGE;
}

// Eight channels (octet o) of raw token r of sequence s, head h: the sink's rows, then the window's.
// What fp16 cannot hold counts as 0 and is flagged.
// `slab`: the sequence's row of heads times heads, plus the head; `count`: raw tokens there are.
__device__ __forceinline__ void raw8(const AttnArgs& a, int64_t slab, int count, int which, int ns, int r, int o,
                                     float (&x)[8], int& flags) {
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = 0.0f;
  if (r >= count) return;
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
// A raw key in the transformed basis, up to sqrt(128) times the row's largest magnitude: as the largest fp16 number
// of its sign where fp16 does not hold it, which is flagged.
__device__ __forceinline__ float within_f16(float x, int& flags) {
  if (fabsf(x) > 65504.0f) flags |= KVQ_DEV_RANGE;
  return fminf(fmaxf(x, -65504.0f), 65504.0f);
}
__device__ __forceinline__ int put_raw_k(const AttnArgs& a, int64_t slab, int count, int ns, int r0, uint32_t slot, int t) {
  int flags = 0;
  const int o = t & 15;
#pragma unroll 4
  for (int j = 0; j < 16; ++j) {
    const int r = (t >> 4) + 8 * j;
    float x[8];
    raw8(a, slab, count, KVQ_KEYS, ns, r0 + r, o, x, flags);
    if (a.L.k_rotate) {   // packed keys and the queries are in the transformed basis
      wht128_octet_unscaled(x, t & 31);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = within_f16(x[e] * a.L.rot_scale, flags);
    }
    st16(slot + (o >> 3) * 16384 + r * 128 + (((o & 7) ^ (r & 7)) << 4), pack_f16(x[0], x[4]), pack_f16(x[1], x[5]),
         pack_f16(x[2], x[6]), pack_f16(x[3], x[7]));
  }
  return flags;
}
__device__ __forceinline__ int put_raw_v(const AttnArgs& a, int64_t slab, int count, int ns, int r0, uint32_t slot, int t) {
  int flags = 0;
  const int o = t & 15;   // token octet
#pragma unroll 1
  for (int b = 0; b < 2; ++b) {
    const int ch = (t >> 4) + 8 * b;
    uint32_t h[8][4];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float x[8];
      raw8(a, slab, count, KVQ_VALUES, ns, r0 + 8 * o + j, ch, x, flags);
#pragma unroll
      for (int e = 0; e < 4; ++e) h[j][e] = pack_f16(x[2 * e], x[2 * e + 1]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        y[j] = e & 1 ? hi2(h[2 * j][e / 2], h[2 * j + 1][e / 2]) : lo2(h[2 * j][e / 2], h[2 * j + 1][e / 2]);
      const int r = 16 * e + ch;   // channel 8 ch + e
      st16(slot + (o >> 3) * 16384 + r * 128 + (((o & 7) ^ (r & 7)) << 4), y[0], y[1], y[2], y[3]);
    }
  }
  return flags;
}

// The ring's order: the position of tile i's keys and of its values, from the block's first on.  Two
// streams over one tile: K0 V0 K1 V1 ...; over tiles in turn: K0 K1 V0 K2 V1 ..., the last keys being
// followed by two values.
__device__ __forceinline__ int ring_k(const Seg& c, int i) { return c.split ? (i == 0 ? 0 : 2 * i - 1) : 2 * i; }
__device__ __forceinline__ int ring_v(const Seg& c, int i) {
  return c.split ? (i == c.N - 1 ? 2 * i + 1 : 2 * i + 2) : 2 * i + 1;
}

template <typename Small>
__device__ __forceinline__ bool seg_wait(Small* sm, int k) {
  return mbar_wait(smem_u32(&sm->seg_full[k % kSegs]), (k / kSegs) & 1, &sm->stop);
}
template <typename Small>
__device__ __forceinline__ void seg_done(Small* sm, int k, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(smem_u32(&sm->seg_empty[k % kSegs]));
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void prefetch_l2(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void expect_bytes(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// What run `run` does of the block at p, from its unit `unit` on with `left` units to go; the run's first block
// is noted for the merge.
__device__ __forceinline__ Seg take_block(const AttnArgs& a, const Work& work, const Place& p, int tiles, int run,
                                          int64_t unit, int64_t left, bool head, int lane) {
  Seg c;
  c.row0 = p.q.row0;
  c.s = p.s;
  c.h = p.h;
  c.n = p.q.n;
  c.tq = p.q.tq;
  c.tr = p.q.tr;
  c.r0 = p.b * a.block;
  c.nr = min(a.block, p.q.n * a.G - c.r0);
  c.split = c.nr <= 128;
  const Seen last = row_seen(a, p.q, (c.r0 + c.nr - 1) / a.G);
  c.raw = last.raw;
  c.packed = last.packed;
  c.n_raw = (c.raw + a.raw_tile - 1) / a.raw_tile;
  const int64_t end = min((int64_t)tiles + 1, unit + left);
  c.t_lo = (int)max(unit - 1, (int64_t)0);
  c.N = (int)max(end - 1 - c.t_lo, (int64_t)0);
  c.slot = unit <= 1 && end == tiles + 1 ? -1 : 2 * run + (unit <= 1);
  if (head && lane == 0) {
    First f;
    f.row0 = c.row0;
    f.h = c.h;
    f.r0 = c.r0;
    f.nr = c.nr;
    f.pad = 0;
    f.unit = unit;
    f.units = tiles + 1;
    work.first[run] = f;
  }
  return c;
}

// One warp: finds this CTA's run, announces its blocks one by one and calls loads(block) after each (false:
// stop); a last block with N < 0 ends the list.
template <typename Small, typename Loads>
__device__ __forceinline__ void announce(const AttnArgs& a, const Work& work, Small* sm, int lane, Loads loads) {
  AttnSeq q0 = {};
  int64_t w0 = 0;
  const Cut cut = find_cut(a, work.runs, lane, &q0, &w0);
  const int run = blockIdx.x;
  if (run == 0 && lane == 0) *work.cut = cut;
  int k = 0;
  bool ok = true;
  if (run < cut.runs && cut.units > 0) {
    int64_t unit, left = run_start(cut, run + 1) - run_start(cut, run);
    Place p = find_place(a, run_start(cut, run), lane, q0, w0, &unit);
    for (bool head = true; left > 0 && ok; head = false) {
      const int tiles = block_tiles(a, p.q, p.b);
      const Seg c = take_block(a, work, p, tiles, run, unit, left, head, lane);
      const int64_t end = min((int64_t)tiles + 1, unit + left);
      left -= end - unit;
      unit = 0;
      if (c.N > 0 || tiles == 0) {
        if (k >= kSegs && !(ok = mbar_wait(smem_u32(&sm->seg_empty[k % kSegs]), (k / kSegs - 1) & 1, &sm->stop))) break;
        if (lane == 0) {
          sm->seg[k % kSegs] = c;
          mbar_arrive(smem_u32(&sm->seg_full[k % kSegs]));
        }
        ++k;
        ok = loads(c);
      }
      if (left > 0 && !next_block(a, &p)) break;
    }
  }
  if (ok && (k < kSegs || mbar_wait(smem_u32(&sm->seg_empty[k % kSegs]), (k / kSegs - 1) & 1, &sm->stop))) {
    if (lane == 0) {
      sm->seg[k % kSegs].N = -1;
      mbar_arrive(smem_u32(&sm->seg_full[k % kSegs]));
    }
  }
}

// ---- the product-issuing thread -----------------------------------------------------------------
__device__ __forceinline__ void issue_qk(uint32_t d, uint32_t q, uint32_t k) {
  const uint64_t dq = smem_desc(q), dk = smem_desc(k);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t off = (i >> 2) * (16384 >> 4) + (i & 3) * 2;
    mma_ss(d, dq + off, dk + off, i > 0);
  }
}
__device__ __forceinline__ void issue_pv(uint32_t d, uint32_t p, uint32_t v, bool accumulate) {
  const uint64_t dv = smem_desc(v);
#pragma unroll
  for (int i = 0; i < 8; ++i) mma_ts(d, p + 8 * i, dv + (i >> 2) * (16384 >> 4) + (i & 3) * 2, accumulate || i > 0);
}

template <typename Small>
__device__ __forceinline__ bool products(Small* sm, uint32_t qs, uint32_t ring, uint32_t tm) {
  volatile int* stop = &sm->stop;
  int base = 0, blocks = 0, np[2] = {0, 0};   // ring positions, blocks and weights of each stream so far
  auto slot = [&](int p) { return ring + ((base + p) % kSlots) * kTile; };
  auto full = [&](int p) {
    const bool ok = mbar_wait(smem_u32(&sm->full[(base + p) % kSlots]), ((base + p) / kSlots) & 1, stop);
    tc_fence_after();
    return ok;
  };
  auto freed = [&](int p) { tc_commit(smem_u32(&sm->empty[(base + p) % kSlots])); };
  auto weights = [&](int w) {
    const bool ok = mbar_wait(smem_u32(&sm->p_full[w]), np[w]++ & 1, stop);
    tc_fence_after();
    return ok;
  };
  auto scores = [&](int w, int p) {
    issue_qk(tm + 128 * w, qs + (w ? kTile : 0), slot(p));
    tc_commit(smem_u32(&sm->s_full[w]));
  };
  for (int k = 0;; ++k) {
    if (!seg_wait(sm, k)) return false;
    const int N = sm->seg[k % kSegs].N, split = sm->seg[k % kSegs].split;
    mbar_arrive(smem_u32(&sm->seg_empty[k % kSegs]));
    if (N < 0) return true;
    if (N == 0) continue;
    if (!mbar_wait(smem_u32(&sm->q_full), blocks++ & 1, stop)) return false;
    tc_fence_after();
    if (!split) {
      if (!full(0)) return false;
      scores(0, 0);
      scores(1, 0);
      freed(0);
      for (int i = 0; i < N; ++i) {
        const int pv = 2 * i + 1, pk = pv + 1;
        for (int w = 0; w < 2; ++w) {
          if (!weights(w)) return false;
          if (w == 0 && !full(pv)) return false;
          issue_pv(tm + 256 + 128 * w, tm + 128 * w + 32, slot(pv), i > 0);
          if (w == 1) freed(pv);
          if (i + 1 < N) {
            if (w == 0 && !full(pk)) return false;
            scores(w, pk);
            if (w == 1) freed(pk);
          } else {
            tc_commit(smem_u32(&sm->o_full[w]));
          }
        }
      }
    } else {
      int pos = 0;
      auto first_scores = [&](int w) {   // both streams have the one Q tile
        issue_qk(tm + 128 * w, qs, slot(pos));
        tc_commit(smem_u32(&sm->s_full[w]));
        freed(pos++);
      };
      for (int w = 0; w < 2 && w < N; ++w) {
        if (!full(pos)) return false;
        first_scores(w);
      }
      for (int t = 0; t < N; ++t) {
        const int w = t & 1;
        if (!weights(w) || !full(pos)) return false;
        issue_pv(tm + 256 + 128 * w, tm + 128 * w + 32, slot(pos), t > 1);
        freed(pos++);
        if (t + 2 < N) {
          if (!full(pos)) return false;
          first_scores(w);
        } else {
          tc_commit(smem_u32(&sm->o_full[w]));
        }
      }
    }
    base += 2 * N;
  }
}

// ---- softmax --------------------------------------------------------------------------------------
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float* a, float* b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*a), "=f"(*b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <int N>
__device__ __forceinline__ void pin(uint32_t (&r)[N]) {   // orders uses of r after the wait before it
#pragma unroll
  for (int j = 0; j < N; ++j) asm volatile("" : "+r"(r[j]));
}
__device__ __forceinline__ void chunk_mask(uint32_t (&x)[32], int cols) {
#pragma unroll
  for (int j = 0; j < 32; ++j)
    if (j >= cols) x[j] = 0xff800000u;   // -inf
}
__device__ __forceinline__ float chunk_max(const uint32_t (&x)[32]) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int j = 0; j < 32; j += 8)
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = fmaxf(fmaxf(m[e], __uint_as_float(x[j + e])), __uint_as_float(x[j + e + 4]));
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
// 32 scores to weights 2^(score * cs + off): their sum in fp32, themselves as fp16 to 16 columns.
__device__ __forceinline__ void chunk_weights(const uint32_t (&x)[32], uint64_t cs2, uint64_t off2, uint64_t* sum0,
                                              uint64_t* sum1, uint32_t to) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    uint32_t h[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = 8 * k + e;
      float p0, p1;
      unpair(fma2(pair(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1])), cs2, off2), &p0, &p1);
      p0 = exp2_approx(p0);
      p1 = exp2_approx(p1);
      uint64_t* sum = j & 1 ? sum1 : sum0;
      *sum = add2(*sum, pair(p0, p1));
      h[e] = pack_f16(p0, p1);
    }
    tmem_st8(to + 8 * k, h);
  }
}

// The queries of 128 rows (tile w) by WARPS warps: a warp per row, four channels per lane; scaled so that
// the row's largest lies in [2^8, 2^9).  16-bit rows are first copied, all of them in flight, to where the
// tile holds them (two segments of 128 bytes each), then turned in place; fp32 rows are read one by one.
// Loops stay short: this code runs once per block, and would otherwise wait for its instructions.
template <int WARPS, typename Small>
__device__ __forceinline__ bool stage_queries(const AttnArgs& a, const Seg& c, Small* sm, uint32_t qs, int w, int wi,
                                              int lane) {
  bool bad = false;
  const int r0 = 128 * w + wi;
  const int t0 = (c.r0 + r0) / a.G, g0 = c.r0 + r0 - t0 * a.G, ts = WARPS / a.G, gs = WARPS - ts * a.G;
  const uint32_t tile = qs + w * kTile + (lane >> 4) * 16384;
  const int64_t head = c.row0 * a.Hq + c.h * a.G;
  auto advance = [&](int& t, int& g) {   // WARPS rows on
    t += ts;
    g += gs;
    if (g >= a.G) {
      g -= a.G;
      ++t;
    }
  };
  const bool wide = a.q_dtype == KVQ_F32;
  if (!wide) {
    int t = t0, g = g0;
#pragma unroll 2
    for (int r = r0; r < 128 * w + 128; r += WARPS) {
      const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + (head + (int64_t)t * a.Hq + g) * 128 + 4 * lane;
      const uint32_t dst = tile + (r & 127) * 128 + (lane & 15) * 8;
      if (r < c.nr) asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
      else asm volatile("st.shared.v2.b32 [%0], {%1, %1};" ::"r"(dst), "r"(0) : "memory");
      advance(t, g);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
  }
  int t = t0, g = g0;
#pragma unroll 4
  for (int r = r0; r < 128 * w + 128; r += WARPS) {
    float x[4] = {0, 0, 0, 0};
    const uint32_t row = tile + (r & 127) * 128;
    if (wide) {
      if (r < c.nr) {
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.q) +
                                                          (head + (int64_t)t * a.Hq + g) * 128 + 4 * lane);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
      }
      advance(t, g);
    } else {
      uint32_t u, v;
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(u), "=r"(v) : "r"(row + (lane & 15) * 8) : "memory");
      if (a.q_dtype == KVQ_F16) {
        x[0] = half_bits_to_float((uint16_t)(u & 0xffffu)); x[1] = half_bits_to_float((uint16_t)(u >> 16));
        x[2] = half_bits_to_float((uint16_t)(v & 0xffffu)); x[3] = half_bits_to_float((uint16_t)(v >> 16));
      } else {
        x[0] = __uint_as_float(u << 16); x[1] = __uint_as_float(u & 0xffff0000u);
        x[2] = __uint_as_float(v << 16); x[3] = __uint_as_float(v & 0xffff0000u);
      }
    }
    // the largest magnitude, as the bits of a positive number; those of Inf and NaN are the largest
    auto magnitude = [](float y) { return __float_as_uint(y) & 0x7fffffffu; };
    if (a.L.k_rotate) {
      bad |= max(max(magnitude(x[0]), magnitude(x[1])), max(magnitude(x[2]), magnitude(x[3]))) >= 0x7f800000u;
      wht128_quad_unscaled(x, lane);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] *= a.L.rot_scale;
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, max(max(magnitude(x[0]), magnitude(x[1])),
                                                            max(magnitude(x[2]), magnitude(x[3]))));
    bad |= top >= 0x7f800000u;
    // 2^(e - 127) <= top < 2^(e - 126); zero, subnormal or overflowing rows get the nearest e that serves
    const int e = min(max((int)(top >> 23), 10), 250);
    const float up = __uint_as_float((uint32_t)(262 - e) << 23);   // 2^(8 - (e - 127))
    if (lane == 0) sm->rowscale[r] = __uint_as_float((uint32_t)(e - 8) << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] *= up;
    const bool odd = lane & 1;
    const float y0 = __shfl_xor_sync(0xffffffffu, odd ? x[0] : x[2], 1);
    const float y1 = __shfl_xor_sync(0xffffffffu, odd ? x[1] : x[3], 1);
    const uint32_t h0 = odd ? pack_f16(y0, x[2]) : pack_f16(x[0], y0);
    const uint32_t h1 = odd ? pack_f16(y1, x[3]) : pack_f16(x[1], y1);
    // every lane has read its part of the row (the reduction above)
    asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(row + ((((lane >> 1) & 7) ^ (r & 7)) << 4) + 8 * odd), "r"(h0),
                 "r"(h1)
                 : "memory");
  }
  return bad;
}

// ---- the way out ------------------------------------------------------------------------------------
// A warp's 32 rows go out 32 channels at a time (words W = 4 part .. + 3) through 4 KB of shared memory, rows
// of 128 bytes with 16-byte chunk c of row i at c ^ (i % 8): a thread writes its row's chunks, then eight
// lanes each read and store a row's.  Columns 16 c + W of O hold channel 8 W + c.
__device__ __forceinline__ float4* out_chunk(uint8_t* box, int i, int c) {
  return reinterpret_cast<float4*>(box + 128 * i + 16 * (c ^ (i & 7)));
}
// This thread's 32 channels of part `part`: o[e][j] is channel 8 (4 part + j) + e.
__device__ __forceinline__ void load_part(uint32_t o_col, int part, uint32_t (&o)[8][4]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) tmem_ld4(o_col + 16 * e + 4 * part, o[e]);
  tmem_wait_ld();
#pragma unroll
  for (int e = 0; e < 8; ++e) pin(o[e]);
}
// f * o (+ g * what the box holds) into the box, as channels in order: chunk 2 j + (e / 4).
__device__ __forceinline__ void box_part(uint8_t* box, int lane, const uint32_t (&o)[8][4], float f, bool add, float g) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      float4* at = out_chunk(box, lane, 2 * j + k);
      float4 v = make_float4(__uint_as_float(o[4 * k][j]) * f, __uint_as_float(o[4 * k + 1][j]) * f,
                             __uint_as_float(o[4 * k + 2][j]) * f, __uint_as_float(o[4 * k + 3][j]) * f);
      if (add) {
        const float4 u = *at;
        v = make_float4(v.x + u.x * g, v.y + u.y * g, v.z + u.z * g, v.w + u.w * g);
      }
      *at = v;
    }
}
// The rows that this lane stores: row i = 4 k + lane / 8 of the warp's, as a row of the output or of the
// partial slot (the host keeps output rows below 2^31); -1 past the block's end.
__device__ __forceinline__ void store_rows(const AttnArgs& a, const Work& work, const Seg& c, int first, int lane,
                                           int (&rows)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const int r = first + 4 * k + (lane >> 3), t = (c.r0 + r) / a.G;
    rows[k] = r >= c.nr ? -1 : c.slot >= 0 ? c.slot * work.rows + r
                                           : ((int)c.row0 + t) * a.Hq + c.h * a.G + (c.r0 + r - t * a.G);
  }
}
__device__ __forceinline__ void store_part(const AttnArgs& a, const Work& work, const Seg& c, uint8_t* box,
                                           const int (&rows)[8], int part, int lane) {
  __syncwarp();
  const bool wide = c.slot >= 0 || a.out_dtype == KVQ_F32;
  void* to = c.slot >= 0 ? work.o : a.out;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const float4 v = *out_chunk(box, 4 * k + (lane >> 3), lane & 7);
    if (rows[k] < 0) continue;
    const int64_t at = (int64_t)rows[k] * 128 + 32 * part + 4 * (lane & 7);
    if (wide) {
      *reinterpret_cast<float4*>(reinterpret_cast<float*>(to) + at) = v;
    } else {
      uint2 h;
      if (a.out_dtype == KVQ_F16) {
        h = make_uint2(pack_f16(v.x, v.y), pack_f16(v.z, v.w));
      } else {
        const __nv_bfloat162 p = __floats2bfloat162_rn(v.x, v.y), q = __floats2bfloat162_rn(v.z, v.w);
        h = make_uint2(*reinterpret_cast<const uint32_t*>(&p), *reinterpret_cast<const uint32_t*>(&q));
      }
      *reinterpret_cast<uint2*>(reinterpret_cast<uint16_t*>(to) + at) = h;
    }
  }
  __syncwarp();
}
inline size_t pad16(size_t n) { return (n + 15) & ~(size_t)15; }
// The workspace for `runs` runs; with ws null only its size.
inline size_t make_work(int runs, int block, int G, int64_t max_new, void* ws, Work* w) {
  const int64_t rows = max_new * G < block ? max_new * G : block;
  const size_t head = 64, firsts = pad16(runs * sizeof(First)), states = pad16((size_t)2 * runs * rows * 4);
  w->runs = runs;
  w->rows = (int)rows;
  char* p = reinterpret_cast<char*>(ws);
  w->cut = reinterpret_cast<Cut*>(p);
  w->first = reinterpret_cast<First*>(p + head);
  w->m = reinterpret_cast<float*>(p + head + firsts);
  w->l = reinterpret_cast<float*>(p + head + firsts + states);
  w->o = reinterpret_cast<float*>(p + head + firsts + 2 * states);
  return head + firsts + 2 * states + (size_t)2 * runs * rows * 512;
}


// The merge of cut blocks after either kernel (attn_paged.cu).
cudaError_t launch_merge(const AttnArgs& a, const Work& w, int runs, cudaStream_t s);
// attn_wide.cu: the attention over pages expanded to fp16 tiles first, `tiles` bytes of them.
cudaError_t launch_attn_narrow(const AttnArgs& a, const Work& w, int runs, cudaStream_t s);   // attn_narrow.cu
size_t attn_wide_bytes(const AttnArgs& a);
cudaError_t launch_attn_wide(const AttnArgs& a, const Work& w, int runs, void* tiles, cudaStream_t s);

}  // namespace attn
}  // namespace kvq
