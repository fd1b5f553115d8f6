// Attention of long chunks: the pages are expanded to fp16 tiles once (expand_kernel), and the attention
// then reads them as they lie (attn_wide_kernel).  attn_paged.cu expands each page for every block of
// 256 query rows that reads it; from two blocks on the work on CUDA cores that this saves is worth
// the 64 KB per page and head written and read again (through L2 where they fit).
//
// The tiles of a sequence: its raw (sink, window) tokens, then its packed groups; per KV head 32 KB of keys
// [token][channel] and 32 KB of values [channel][token], laid out as the products read them.
#include "attn_paged.cuh"

namespace kvq {
namespace {

using namespace attn;

int64_t tile_bound(int64_t max_tq, int max_tr, int ns) { return (max_tq + 127) / 128 + (ns + max_tr + 127) / 128; }

// Raw tokens of a sequence: sink rows in use and window rows.
__device__ __forceinline__ int raw_tokens(const AttnArgs& a, int tq, int tr) {
  return (int)min((int64_t)a.b.n_sink, (int64_t)a.b.n_sink + tr + tq) + max(tr, 0);
}

// ---- expansion ----------------------------------------------------------------------------------
constexpr int kExpandThreads = 256;
constexpr size_t kExpandSmem = 2 * kTile;

// CTAs take (tile, head) in turn over all sequences that have query rows; threads 0-127 keys, the others
// values, both into shared memory, from where one bulk copy writes the 64 KB out.  Three CTAs per SM (shared
// memory) hide one another's loads; 13 sequences of 4096 tokens and fewer, 32 heads: 126 us, bound by the
// dependent loads of a tile (page, codes) and the 64 KB stored for each 13 KB read.
__global__ void __launch_bounds__(kExpandThreads, 3) expand_kernel(const __grid_constant__ AttnArgs a, char* tiles,
                                                                   int64_t bound) {
  extern __shared__ __align__(1024) uint8_t smem[];
  griddep_wait();
  griddep_launch_dependents();
  const PagedBatch& b = a.b;
  const int lane = threadIdx.x & 31, t = threadIdx.x & 127;
  int flags = 0;
  int s0 = 0;                       // 32 sequences at a time, and the items before them
  int64_t before = 0;
  for (int64_t item = blockIdx.x;; item += gridDim.x) {
    AttnSeq q = {};
    int64_t tile = -1;
    int s = 0, raw = 0;
    for (; s0 < b.num_seqs; s0 += 32) {
      int64_t n = 0;
      int r = 0;
      AttnSeq o = {};
      if (s0 + lane < b.num_seqs) {
        o = attn_seq(a, s0 + lane);
        if (o.n > 0) {
          r = (raw_tokens(a, o.tq, o.tr) + 127) / 128;
          n = (r + (o.tq + 127) / 128) * (int64_t)a.L.Hkv;
        }
      }
      const int64_t incl = scan64(n, lane);
      const unsigned hit = __ballot_sync(0xffffffffu, item - before < incl);
      if (hit) {
        const int l = __ffs(hit) - 1;
        tile = item - before - __shfl_sync(0xffffffffu, incl - n, l);
        raw = __shfl_sync(0xffffffffu, r, l);
        q.tq = __shfl_sync(0xffffffffu, o.tq, l);
        q.tr = __shfl_sync(0xffffffffu, o.tr, l);
        s = s0 + l;
        break;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (tile < 0) break;            // uniform: every warp counts alike
    const int h = (int)(tile % a.L.Hkv);
    tile /= a.L.Hkv;
    if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the last copy has left
    __syncthreads();
    const uint32_t dst = smem_u32(smem) + (threadIdx.x < 128 ? 0 : kTile);
    if (tile < raw) {
      const int64_t slab = (int64_t)s * a.L.Hkv + h;
      const int count = raw_tokens(a, q.tq, q.tr), ns = count - max(q.tr, 0);
      if (threadIdx.x < 128) flags |= put_raw_k(a, slab, count, ns, 128 * (int)tile, dst, t);
      else flags |= put_raw_v(a, slab, count, ns, 128 * (int)tile, dst, t);
    } else {
      const int g = (int)tile - raw;
      int blk = __ldg(b.table + (int64_t)s * b.max_blocks + g);
      if (blk < 0 || blk >= b.num_blocks) {
        flags |= KVQ_DEV_BOUNDS;
        blk = 0;
      }
      const int64_t slab = (int64_t)blk * a.L.Hkv + h;
      const Side& S = a.L.side[threadIdx.x >= 128];
      const char* codes = reinterpret_cast<const char*>(S.codes) + slab * S.code_slab_bytes;
      const char* scale = reinterpret_cast<const char*>(S.scale) + slab * 256;
      const char* zero = reinterpret_cast<const char*>(S.zero) + slab * 256;
      if (threadIdx.x < 128) flags |= put_keys(codes, scale, zero, dst, t);
      else flags |= put_values(codes, scale, zero, dst, t, min(128, q.tq - 128 * g));
    }
    fence_async_smem();
    __syncthreads();
    if (threadIdx.x == 0) {
      char* to = tiles + ((s * bound + tile) * a.L.Hkv + h) * (2 * (int64_t)kTile);
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(to), "r"(smem_u32(smem)),
                   "r"(2 * kTile)
                   : "memory");
      asm volatile("cp.async.bulk.commit_group;" ::: "memory");
    }
  }
  if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (flags && lane == 0) flag(a.status, flags);
}

// ---- attention ------------------------------------------------------------------------------------
// Ten warps.  0-7: softmax, stream warp / 4, a thread per row with its 128 scores in registers; they
// also stage the queries and write the output.  8: one thread issues the products.  9: announces the
// run's blocks and copies their tiles, 32 KB each, into the ring.
constexpr int kThreads = 320;

struct Small {
  float rowscale[256];
  float m1[128], l1[128];                 // stream 1's state on its way to stream 0
  Seg seg[kSegs];
  alignas(8) uint64_t full[kSlots], empty[kSlots];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t s_full[2], p_full[2], o_full[2], q_full, drain;
  uint64_t row_pair[4];                   // the warps of the two streams with the same rows
  uint64_t all;                           // the eight softmax warps
  uint32_t tmem;
  int stop;
};
constexpr size_t kSmem = kStagesAt + sizeof(Small);
static_assert(kSmem <= 232448, "shared memory of a CTA");

__device__ __forceinline__ void loader(const AttnArgs& a, const Work& work, Small* sm, uint32_t ring, const char* tiles,
                                       int64_t bound, int lane) {
  int issued = 0;
  announce(a, work, sm, lane, [&](const Seg& c) {
    const char* seq = tiles + (c.s * bound * a.L.Hkv + c.h) * (2 * (int64_t)kTile);
    // a block may see fewer raw tiles than the sequence has
    const int hidden = (raw_tokens(a, c.tq, c.tr) + 127) / 128 - c.n_raw;
    for (int p = 0; p < 2 * c.N; ++p) {
      // the inverse of ring_k and ring_v
      int i = p >> 1;
      bool value = p & 1;
      if (c.split) {
        value = p == 2 * c.N - 1 || (p > 0 && !(p & 1));
        i = p == 0 ? 0 : p == 2 * c.N - 1 ? c.N - 1 : value ? (p >> 1) - 1 : (p + 1) >> 1;
      }
      const int slot = issued % kSlots, use = issued / kSlots;
      if (use > 0 && !mbar_wait(smem_u32(&sm->empty[slot]), (use - 1) & 1, &sm->stop)) return false;
      if (lane == 0) {
        const uint32_t bar = smem_u32(&sm->full[slot]);
        expect_bytes(bar, kTile);
        const int64_t at = c.t_lo + i + (c.t_lo + i < c.n_raw ? 0 : hidden);
        bulk_load(ring + slot * kTile, seq + at * a.L.Hkv * (2 * kTile) + (value ? kTile : 0), kTile, bar);
      }
      ++issued;
    }
    return true;
  });
  if (sm->stop && lane == 0) {   // copies still on their way must land before the memory is given up
    int never = 0;
    for (int n = max(issued - kSlots, 0); n < issued; ++n)
      mbar_wait(smem_u32(&sm->full[n % kSlots]), (n / kSlots) & 1, &never);
  }
  __syncwarp();
}

__device__ __forceinline__ void softmax_warp(const AttnArgs& a, const Work& work, Small* sm, uint8_t* smem, uint32_t qs,
                                             uint32_t tm, int warp, int lane) {
  const int w = warp >> 2, row = 32 * (warp & 3) + lane;   // stream, row of its tile
  const uint32_t lanes = (uint32_t)(warp & 3) << 21;       // lane 32 (warp % 4) in the address's upper half
  const uint32_t s_col = tm + lanes + 128 * w, o_col = tm + lanes + 256 + 128 * w;
  const uint32_t s_bar = smem_u32(&sm->s_full[w]), p_bar = smem_u32(&sm->p_full[w]);
  volatile int* stop = &sm->stop;
  auto sync = [&](uint64_t* bar, int* count) {   // a barrier of counted warps
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(bar));
    return mbar_wait(smem_u32(bar), (*count)++ & 1, stop);
  };
  int ns = 0, no = 0, n_pair = 0, n_all = 0, blocks = 0;   // phases of the barriers waited on
  for (int k = 0;; ++k) {
    if (!seg_wait(sm, k)) return;
    const Seg c = sm->seg[k % kSegs];
    if (c.N < 0) return;
    const int r = c.split ? row : 128 * w + row;
    const int64_t out_row = (c.row0 + (c.r0 + r) / a.G) * a.Hq + c.h * a.G + (c.r0 + r) % a.G;
    if (c.N == 0) {   // no token for any row
      if (r < c.nr && !(c.split && w)) {
        for (int i = 0; i < 128; ++i) store_elem(a.out, out_row * 128 + i, a.out_dtype, 0.0f);
        if (a.lse) a.lse[out_row] = -INFINITY;
      }
      seg_done(sm, k, lane);
      continue;
    }
    const bool bad = c.split ? stage_queries<8>(a, c, sm, qs, 0, warp, lane)
                             : stage_queries<4>(a, c, sm, qs, w, warp & 3, lane);
    if (__any_sync(0xffffffffu, bad) && lane == 0) flag(a.status, KVQ_DEV_NONFINITE);
    fence_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm->q_full));
    if (!sync(&sm->all, &n_all)) return;   // row scales

    Seen see = {0, 0};
    if (r < c.nr) {
      AttnSeq q;
      q.n = c.n;
      q.tq = c.tq;
      q.tr = c.tr;
      see = row_seen(a, q, (c.r0 + r) / a.G);
    }
    const bool live = (r & ~31) < c.nr;      // a row of this warp is real
    // never 0, so that a masked score of -inf stays one
    const float cs = fmaxf(a.qscale * sm->rowscale[r], 1.2e-38f);
    float m = -INFINITY, l = 0.0f;
    const int n = c.split ? (c.N - w + 1) / 2 : c.N;
    for (int i = 0; i < n; ++i) {
      if (!mbar_wait(s_bar, ns++ & 1, stop)) return;
      if (!live) {   // these weights are never read
        if (lane == 0) mbar_arrive(p_bar);
        continue;
      }
      tc_fence_after();
      const int at = c.t_lo + (c.split ? 2 * i + w : i);
      const int cols = at < c.n_raw ? see.raw - 128 * at : see.packed - 128 * (at - c.n_raw);
      uint32_t x0[32], x1[32], x2[32], x3[32];
      tmem_ld32(s_col, x0);
      tmem_ld32(s_col + 32, x1);
      tmem_ld32(s_col + 64, x2);
      tmem_ld32(s_col + 96, x3);
      tmem_wait_ld();
      pin(x0);
      pin(x1);
      pin(x2);
      pin(x3);
      if (__any_sync(0xffffffffu, cols < 128)) {
        chunk_mask(x0, cols);
        chunk_mask(x1, cols - 32);
        chunk_mask(x2, cols - 64);
        chunk_mask(x3, cols - 96);
      }
      const float top = fmaxf(fmaxf(chunk_max(x0), chunk_max(x1)), fmaxf(chunk_max(x2), chunk_max(x3))) * cs;
      const bool move = top > m + kLazy;     // true from -inf for any finite score
      if (__any_sync(0xffffffffu, move)) {
        const float mn = move ? top : m;
        const float f = move ? exp2_approx(m - mn) : 1.0f;
        l *= f;
        m = mn;
        if (i > 0) {   // rare: few registers rather than few loads
#pragma unroll 1
          for (int e = 0; e < 16; ++e) {
            uint32_t o[8];
            tmem_ld8(o_col + 8 * e, o);
            tmem_wait_ld();
            pin(o);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st8(o_col + 8 * e, o);
          }
        }
      }
      const float off = kLift - (m == -INFINITY ? 0.0f : m);
      const uint64_t cs2 = pair(cs, cs), off2 = pair(off, off);
      uint64_t sum0 = 0, sum1 = 0;
      chunk_weights(x0, cs2, off2, &sum0, &sum1, s_col + 32);
      chunk_weights(x1, cs2, off2, &sum0, &sum1, s_col + 48);
      chunk_weights(x2, cs2, off2, &sum0, &sum1, s_col + 64);
      chunk_weights(x3, cs2, off2, &sum0, &sum1, s_col + 80);
      float e0, e1;
      unpair(add2(sum0, sum1), &e0, &e1);
      l += e0 + e1;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(p_bar);
    }

    const bool two = c.split && c.N > 1;
    if (n > 0 && !mbar_wait(smem_u32(&sm->o_full[w]), no++ & 1, stop)) return;
    // stream 1 is to write over Q, which the other stream's products may still read
    if (two && w == 1 && !mbar_wait(smem_u32(&sm->o_full[0]), blocks & 1, stop)) return;
    ++blocks;
    tc_fence_after();
    // boxes over Q: one per warp, or in a split block one per part of the warp's rows
    uint8_t* box = smem + (c.split ? 0 : w * kTile) + 4096 * (warp & 3);
    const int box_step = c.split ? 16384 : 0;
    uint32_t o[8][4];
    float f0 = 1.0f, f1 = 0.0f;
    if (two) {
      if (w == 1) {
        sm->m1[row] = m;
        sm->l1[row] = l;
#pragma unroll 1
        for (int p = 0; p < 4; ++p) {
          load_part(o_col, p, o);
          box_part(box + p * box_step, lane, o, 1.0f, false, 0.0f);
        }
      }
      if (!sync(&sm->row_pair[warp & 3], &n_pair)) return;
      if (w == 0) {
        const float m1 = sm->m1[row], l1 = sm->l1[row], mm = fmaxf(m, m1);
        f0 = m == -INFINITY ? 0.0f : exp2_approx(m - mm);
        f1 = m1 == -INFINITY ? 0.0f : exp2_approx(m1 - mm);
        l = l * f0 + l1 * f1;
        m = mm;
      }
    }
    if (live && (w == 0 || !c.split)) {
      if (r < c.nr) {
        if (c.slot >= 0) {
          work.m[(int64_t)c.slot * work.rows + r] = m;
          work.l[(int64_t)c.slot * work.rows + r] = l;
        } else if (a.lse) {
          a.lse[out_row] = l > 0.0f ? kLn2 * (m + log2f(l) - kLift) : -INFINITY;
        }
      }
      const float inv = c.slot >= 0 ? 1.0f : l > 0.0f ? 1.0f / l : 0.0f;
      int rows[8];
      store_rows(a, work, c, r - lane, lane, rows);
#pragma unroll 1
      for (int p = 0; p < 4; ++p) {
        load_part(o_col, p, o);
        box_part(box + p * box_step, lane, o, f0 * inv, two, f1 * inv);
        store_part(a, work, c, box + p * box_step, rows, p, lane);
      }
    }
    tc_fence_before();
    seg_done(sm, k, lane);
    if (!sync(&sm->all, &n_all)) return;   // Q and the states may be overwritten
  }
}

// 2048 tokens x 8 x 4 heads over 16384: 675 us with the expansion and the merge, 865 TFLOP/s; 2.7 us per pair of a
// 256-row block and a 128-token tile (64 KB per pair through L2), the tensor pipe busy for 45 % of the time.
__global__ void __launch_bounds__(kThreads, 1) attn_wide_kernel(const __grid_constant__ AttnArgs a,
                                                                const __grid_constant__ Work work, const char* tiles,
                                                                int64_t bound) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Small* sm = reinterpret_cast<Small*>(smem + kStagesAt);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t qs = smem_u32(smem), ring = qs + kSlotsAt;
  if (threadIdx.x == 0) {
    auto init = [](uint64_t& b, uint32_t n) { mbar_init(smem_u32(&b), n); };
    for (int i = 0; i < kSlots; ++i) {
      init(sm->full[i], 1);
      init(sm->empty[i], 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      init(sm->seg_full[i], 1);
      init(sm->seg_empty[i], 9);   // softmax warps and the product thread
    }
    for (int w = 0; w < 2; ++w) {
      init(sm->s_full[w], 1);
      init(sm->p_full[w], 4);
      init(sm->o_full[w], 1);
    }
    for (int i = 0; i < 4; ++i) init(sm->row_pair[i], 2);
    init(sm->q_full, 8);
    init(sm->all, 8);
    init(sm->drain, 1);
    sm->stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 8) tmem_alloc(smem_u32(&sm->tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = sm->tmem;
  if (warp < 8) {
    softmax_warp(a, work, sm, smem, qs, tm, warp, lane);
  } else if (warp == 8) {
    if (lane == 0 && !products(sm, qs, ring, tm)) {
      // stopped: what was issued still has to end before its memory is given up
      flag(a.status, KVQ_DEV_TIMEOUT);
      tc_commit(smem_u32(&sm->drain));
      int never = 0;
      mbar_wait(smem_u32(&sm->drain), 0, &never);
    }
    __syncwarp();
  } else {
    loader(a, work, sm, ring, tiles, bound, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) tmem_free(tm, 512);
}

}  // namespace

size_t attn_wide_tiles(int num_seqs, int Hkv, int64_t max_t_quant, int max_t_res, int n_sink) {
  return (size_t)num_seqs * tile_bound(max_t_quant, max_t_res, n_sink) * Hkv * 2 * kTile;
}

namespace attn {

size_t attn_wide_bytes(const AttnArgs& a) {
  return attn_wide_tiles(a.b.num_seqs, a.L.Hkv, a.max_t_quant, a.max_t_res, a.b.n_sink);
}

cudaError_t launch_attn_wide(const AttnArgs& a, const Work& w, int runs, void* tiles, cudaStream_t s) {
  const int64_t bound = tile_bound(a.max_t_quant, a.max_t_res, a.b.n_sink);
  cudaError_t e = cudaFuncSetAttribute(expand_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kExpandSmem);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(attn_wide_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(expand_kernel, dim3(3 * runs), dim3(kExpandThreads), kExpandSmem, s, a, reinterpret_cast<char*>(tiles),
                 bound);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_wide_kernel, dim3(runs), dim3(kThreads), kSmem, s, a, w,
                 reinterpret_cast<const char*>(tiles), bound);
  if (e != cudaSuccess) return e;
  return launch_merge(a, w, runs, s);
}

}  // namespace attn
}  // namespace kvq
