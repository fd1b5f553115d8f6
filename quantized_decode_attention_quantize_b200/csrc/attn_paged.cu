// Attention of several new tokens per sequence over the paged cache (D = 128, groups of 128
// tokens, 4-bit per-channel keys, 2-bit per-token values, raw sink and window rows) on the
// fifth-generation tensor cores.
//
// Work.  The query rows of one KV head, G per new token, are cut into blocks of up to 256; a
// block sees KV tiles of 128 tokens: its visible raw (sink, window) tokens first, then its
// visible packed groups.  The tiles of all blocks end to end, each block with one more unit for its
// fixed costs, are cut into equal runs, one per SM, whatever the lengths in the batch.  A block that
// one run holds whole is written out at once; of a block cut by runs every part leaves its softmax
// state in the workspace, and a second kernel, one CTA per cut, merges them.
//
// Within a block two streams keep the tensor core busy, so that one's products run under the
// other's softmax: the block's two halves of 128 rows over the same tiles, or, for a block of at
// most 128 rows, those rows over the even and the odd tiles, the two states merged at the end.
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
// Roles (26 warps).
//   0-15   softmax: stream w = warp / 8, two threads per row (64 columns each, the maxima exchanged in
//          shared memory); S from tensor memory in chunks of 32 columns, P back over S's columns
//          32-95 as the A operand of the value product.  They also stage the queries and write the
//          output.
//   16-19  keys: codes to an fp16 tile [token][channel], the channels of an octet in the order 0 4
//          1 5 2 6 3 7 (which the masks give; Q has the same).
//   20-23  values: codes to an fp16 tile [channel][token], channel 8 W + c in row 16 c + W (rows of
//          a store phase then differ modulo 8, and their chunks in bank).
//   24     one thread issues the products.
//   25     finds the run's blocks, announces them, and copies the packed groups' codes and metadata
//          into shared memory (bulk copies, two groups ahead).
// K and V tiles pass through one ring of four slots in the order the products use them.
//
// Tensor memory: S0, S1, O0, O1, 128 columns each (all 512).  A product that overwrites S with the
// next scores is issued after the value product that reads P from it, in the same thread's order.
//
// Waits are bounded (tc05.cuh); one that runs out stops the CTA and raises KVQ_DEV_TIMEOUT.
#include "attn_paged.cuh"

namespace kvq {
namespace {

using namespace attn;

constexpr int kThreads = 832;
constexpr int kStages = 2;                // packed groups in flight
constexpr int kStageK = 8192 + 512, kStageV = 4096 + 512;   // codes, scales, zero-points
constexpr int kSmallAt = kStagesAt + kStages * (kStageK + kStageV);

struct Small {
  float rowscale[256];
  float mx[2][2][128];                    // [stream][half][row]: maxima, at the end sums
  float m1[128], l1[128];                 // stream 1's state on its way to stream 0
  Seg seg[kSegs];
  alignas(8) uint64_t full[kSlots], empty[kSlots];
  uint64_t k_in[kStages], k_out[kStages], v_in[kStages], v_out[kStages];
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t s_full[2], p_full[2], o_full[2], q_full, drain;
  uint64_t row_pair[8];                   // the two warps of a stream's 32 rows
  uint64_t row_quad[4];                   // the four warps of both streams with the same rows
  uint64_t all;                           // the 16 softmax warps
  uint32_t tmem;
  int stop;
};
constexpr size_t kSmem = kSmallAt + sizeof(Small);
static_assert(kSmem <= 232448, "shared memory of a CTA");

template <bool VALUES>
__device__ __forceinline__ void producer(const AttnArgs& a, Small* sm, uint32_t ring, const uint8_t* stages) {
  const int t = threadIdx.x & 127, lane = t & 31;
  int flags = 0, base = 0, groups = 0;   // ring positions and packed groups before this block
  bool ok = true;
  for (int k = 0; ok && (ok = seg_wait(sm, k)); ++k) {
    const Seg c = sm->seg[k % kSegs];
    seg_done(sm, k, lane);
    if (c.N < 0) break;
    const int ns = (int)min((int64_t)a.b.n_sink, (int64_t)a.b.n_sink + c.tr + c.tq);
    for (int i = 0; i < c.N; ++i) {
      const int p = base + (VALUES ? ring_v(c, i) : ring_k(c, i)), slot = p % kSlots, use = p / kSlots;
      const uint32_t dst = ring + slot * kTile;
      const int at = c.t_lo + i;
      if (use > 0 && !(ok = mbar_wait(smem_u32(&sm->empty[slot]), (use - 1) & 1, &sm->stop))) break;
      if (at < c.n_raw) {
        const int64_t slab = (int64_t)c.s * a.L.Hkv + c.h;
        flags |= VALUES ? put_raw_v(a, slab, c.raw, ns, 128 * at, dst, t)
                        : put_raw_k(a, slab, c.raw, ns, 128 * at, dst, t);
        fence_async_smem();
        mbar_arrive(smem_u32(&sm->full[slot]));
      } else {
        const int st = groups % kStages, round = (groups / kStages) & 1;
        ++groups;
        if (!(ok = mbar_wait(smem_u32(VALUES ? &sm->v_in[st] : &sm->k_in[st]), round, &sm->stop))) break;
        const uint8_t* in = stages + st * (kStageK + kStageV) + (VALUES ? kStageK : 0);
        if (VALUES) flags |= put_values(in, in + 4096, in + 4352, dst, t, min(128, c.tq - 128 * (at - c.n_raw)));
        else flags |= put_keys(in, in + 8192, in + 8448, dst, t);
        fence_async_smem();
        mbar_arrive(smem_u32(&sm->full[slot]));
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(VALUES ? &sm->v_out[st] : &sm->k_out[st]));
      }
    }
    base += 2 * c.N;
  }
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (flags && lane == 0) flag(a.status, flags);
}

// ---- the loader ---------------------------------------------------------------------------------
__device__ __forceinline__ void loader(const AttnArgs& a, const Work& work, Small* sm, uint32_t stages, int lane) {
  int groups = 0, issued[2] = {0, 0}, flags = 0;
  announce(a, work, sm, lane, [&](const Seg& c) {
    bool ok = true;
    // the packed groups of this part, pages 32 at a time
    const int g0 = max(c.t_lo - c.n_raw, 0), g1 = c.t_lo + c.N - c.n_raw;
    int page = 0;
    for (int g = g0; g < g1 && ok; ++g) {
      if (((g - g0) & 31) == 0) {
        page = g + lane < g1 ? __ldg(a.b.table + (int64_t)c.s * a.b.max_blocks + g + lane) : 0;
        if (page < 0 || page >= a.b.num_blocks) {
          flags |= KVQ_DEV_BOUNDS;
          page = 0;
        }
        if (g + lane < g1) {   // towards L2 now: the two stages alone would wait for memory
#pragma unroll
          for (int v = 0; v < 2; ++v) {
            const Side& S = a.L.side[v];
            const int64_t slab = (int64_t)page * a.L.Hkv + c.h;
            prefetch_l2(reinterpret_cast<const uint8_t*>(S.codes) + slab * S.code_slab_bytes, v ? 4096 : 8192);
            prefetch_l2(reinterpret_cast<const __half*>(S.scale) + slab * 128, 256);
            prefetch_l2(reinterpret_cast<const __half*>(S.zero) + slab * 128, 256);
          }
        }
      }
      const int64_t slab = (int64_t)__shfl_sync(0xffffffffu, page, (g - g0) & 31) * a.L.Hkv + c.h;
      const int st = groups % kStages, use = groups / kStages;
      const uint32_t dst = stages + st * (kStageK + kStageV);
#pragma unroll
      for (int v = 0; v < 2 && ok; ++v) {
        const uint32_t out = smem_u32(v ? &sm->v_out[st] : &sm->k_out[st]);
        const uint32_t in = smem_u32(v ? &sm->v_in[st] : &sm->k_in[st]);
        if (use > 0) ok = mbar_wait(out, (use - 1) & 1, &sm->stop);
        if (ok && lane == 0) {
          const Side& S = a.L.side[v];
          const uint32_t codes = v ? 4096 : 8192, to = dst + (v ? kStageK : 0);
          expect_bytes(in, codes + 512);
          bulk_load(to, reinterpret_cast<const uint8_t*>(S.codes) + slab * S.code_slab_bytes, codes, in);
          bulk_load(to + codes, reinterpret_cast<const __half*>(S.scale) + slab * 128, 256, in);
          bulk_load(to + codes + 256, reinterpret_cast<const __half*>(S.zero) + slab * 128, 256, in);
        }
        if (ok) ++issued[v];
      }
      if (ok) ++groups;
    }
    return ok;
  });
  if (sm->stop && lane == 0) {   // copies still on their way must land before the memory is given up
    int never = 0;
    for (int v = 0; v < 2; ++v)
      for (int g = max(issued[v] - kStages, 0); g < issued[v]; ++g)
        mbar_wait(smem_u32(v ? &sm->v_in[g % kStages] : &sm->k_in[g % kStages]), (g / kStages) & 1, &never);
  }
  __syncwarp();
  flags = __reduce_or_sync(0xffffffffu, flags);
  if (flags && lane == 0) flag(a.status, flags);
}

__device__ __forceinline__ void softmax_warp(const AttnArgs& a, const Work& work, Small* sm, uint8_t* smem, uint32_t qs,
                                             uint32_t tm, int warp, int lane) {
  const int w = warp >> 3, hf = (warp >> 2) & 1, row = 32 * (warp & 3) + lane;   // stream, half, row of its tile
  const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // lane 32 (warp % 4) in the address's upper half
  const uint32_t s_col = tm + lanes + 128 * w, o_col = tm + lanes + 256 + 128 * w;
  // the half's two chunks: the one read twice, and the one kept, whose columns take the weights
  const uint32_t far = s_col + (hf ? 96 : 0), near = s_col + (hf ? 64 : 32);
  const int far_at = hf ? 96 : 0, near_at = hf ? 64 : 32;
  const uint32_t far_to = s_col + 32 + far_at / 2, near_to = s_col + 32 + near_at / 2;
  volatile int* stop = &sm->stop;
  auto sync2 = [&](uint64_t* bar, int* count) {   // a barrier of counted warps
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(bar));
    return mbar_wait(smem_u32(bar), (*count)++ & 1, stop);
  };
  int ns = 0, no = 0, n_rows = 0, n_quads = 0, n_all = 0, blocks = 0;   // phases of the barriers waited on
  for (int k = 0;; ++k) {
    if (!seg_wait(sm, k)) return;
    const Seg c = sm->seg[k % kSegs];
    if (c.N < 0) return;
    const int r = c.split ? row : 128 * w + row;
    const int64_t out_row = (c.row0 + (c.r0 + r) / a.G) * a.Hq + c.h * a.G + (c.r0 + r) % a.G;
    if (c.N == 0) {   // no token for any row
      if (r < c.nr && !(c.split && w)) {
        for (int i = 64 * hf; i < 64 * hf + 64; ++i) store_elem(a.out, out_row * 128 + i, a.out_dtype, 0.0f);
        if (a.lse && hf == 0) a.lse[out_row] = -INFINITY;
      }
      seg_done(sm, k, lane);
      continue;
    }
    bool bad = false;
    if (!c.split) bad = stage_queries<8>(a, c, sm, qs, w, warp & 7, lane);
    else bad = stage_queries<16>(a, c, sm, qs, 0, warp, lane);
    if (__any_sync(0xffffffffu, bad) && lane == 0) flag(a.status, KVQ_DEV_NONFINITE);
    fence_async_smem();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&sm->q_full));
    if (!sync2(&sm->all, &n_all)) return;   // row scales

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
      if (!mbar_wait(smem_u32(&sm->s_full[w]), ns++ & 1, stop)) return;
      if (!live) {   // these weights are never read
        if (lane == 0) mbar_arrive(smem_u32(&sm->p_full[w]));
        continue;
      }
      tc_fence_after();
      const int at = c.t_lo + (c.split ? 2 * i + w : i);
      const int cols = at < c.n_raw ? see.raw - 128 * at : see.packed - 128 * (at - c.n_raw);
      const bool edge = __any_sync(0xffffffffu, cols < 128);
      uint32_t x[32];
      tmem_ld32(far, x);
      tmem_wait_ld();
      pin(x);
      if (edge) chunk_mask(x, cols - far_at);
      float top = chunk_max(x);
      tmem_ld32(near, x);
      tmem_wait_ld();
      pin(x);
      if (edge) chunk_mask(x, cols - near_at);
      top = fmaxf(top, chunk_max(x));
      sm->mx[w][hf][row] = top;
      if (!sync2(&sm->row_pair[4 * w + (warp & 3)], &n_rows)) return;
      top = fmaxf(top, sm->mx[w][hf ^ 1][row]) * cs;
      const bool move = top > m + kLazy;     // true from -inf for any finite score
      if (__any_sync(0xffffffffu, move)) {
        const float mn = move ? top : m;
        const float f = move ? exp2_approx(m - mn) : 1.0f;
        l *= f;
        m = mn;
        if (i > 0) {   // this half's columns of O; rare: few registers rather than few loads
#pragma unroll 1
          for (int e = 0; e < 8; ++e) {
            uint32_t o[8];
            tmem_ld8(o_col + 64 * hf + 8 * e, o);
            tmem_wait_ld();
            pin(o);
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
            tmem_st8(o_col + 64 * hf + 8 * e, o);
          }
        }
      }
      const float off = kLift - (m == -INFINITY ? 0.0f : m);
      const uint64_t cs2 = pair(cs, cs), off2 = pair(off, off);
      uint64_t sum0 = 0, sum1 = 0;
      chunk_weights(x, cs2, off2, &sum0, &sum1, near_to);
      tmem_ld32(far, x);
      tmem_wait_ld();
      pin(x);
      if (edge) chunk_mask(x, cols - far_at);
      chunk_weights(x, cs2, off2, &sum0, &sum1, far_to);
      float e0, e1;
      unpair(add2(sum0, sum1), &e0, &e1);
      l += e0 + e1;
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm->p_full[w]));
    }

    // the state of stream w's rows: l over both halves, then over both streams of a split block
    const bool two = c.split && c.N > 1;
    if (n > 0 && !mbar_wait(smem_u32(&sm->o_full[w]), no++ & 1, stop)) return;
    // stream 1 is to write over Q, which the other stream's products may still read
    if (two && w == 1 && !mbar_wait(smem_u32(&sm->o_full[0]), blocks & 1, stop)) return;
    ++blocks;
    tc_fence_after();
    if (n > 0) {
      if (!sync2(&sm->row_pair[4 * w + (warp & 3)], &n_rows)) return;   // mx has been read
      sm->mx[w][hf][row] = l;
      if (!sync2(&sm->row_pair[4 * w + (warp & 3)], &n_rows)) return;
      l += sm->mx[w][hf ^ 1][row];
    }
    // boxes over Q: one per warp, or in a split block one per part of the warp's rows
    uint8_t* box = smem + (c.split ? 2 * hf * 16384 : w * kTile + hf * 16384) + 4096 * (warp & 3);
    const int box_step = c.split ? 16384 : 0;
    uint32_t o[8][4];
    float f0 = 1.0f, f1 = 0.0f;
    if (two) {
      if (w == 1) {
        sm->m1[row] = m;
        sm->l1[row] = l;
#pragma unroll 1
        for (int p = 0; p < 2; ++p) {
          load_part(o_col, 2 * hf + p, o);
          box_part(box + p * box_step, lane, o, 1.0f, false, 0.0f);
        }
      }
      if (!sync2(&sm->row_quad[warp & 3], &n_quads)) return;
      if (w == 0) {
        const float m1 = sm->m1[row], l1 = sm->l1[row], mm = fmaxf(m, m1);
        f0 = m == -INFINITY ? 0.0f : exp2_approx(m - mm);
        f1 = m1 == -INFINITY ? 0.0f : exp2_approx(m1 - mm);
        l = l * f0 + l1 * f1;
        m = mm;
      }
    }
    if (live && (w == 0 || !c.split)) {
      if (r < c.nr && hf == 0) {
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
      for (int p = 0; p < 2; ++p) {   // this half's words of the rows
        load_part(o_col, 2 * hf + p, o);
        box_part(box + p * box_step, lane, o, f0 * inv, two, f1 * inv);
        store_part(a, work, c, box + p * box_step, rows, 2 * hf + p, lane);
      }
    }
    tc_fence_before();
    seg_done(sm, k, lane);
    if (!sync2(&sm->all, &n_all)) return;   // Q and the states may be overwritten
  }
}

// One CTA per SM, each with its run of units.  64 tokens x 8 sequences over 16384, 8 x 4 heads: 261 us, 4.7 us per
// pair of a 256-row block and a 128-token tile, where the products need 1.5 at the measured bf16 rate: softmax and
// expansion share the SM's issue slots and its instruction cache, so the expansion has eight warps and no more.
__global__ void __launch_bounds__(kThreads, 1) attn_tc_kernel(const __grid_constant__ AttnArgs a,
                                                              const __grid_constant__ Work work) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Small* sm = reinterpret_cast<Small*>(smem + kSmallAt);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t qs = smem_u32(smem), ring = qs + kSlotsAt;
  if (threadIdx.x == 0) {
    auto init = [](uint64_t& b, uint32_t n) { mbar_init(smem_u32(&b), n); };
    for (int i = 0; i < kSlots; ++i) {
      init(sm->full[i], 128);
      init(sm->empty[i], 1);
    }
    for (int i = 0; i < kStages; ++i) {
      init(sm->k_in[i], 1);
      init(sm->v_in[i], 1);
      init(sm->k_out[i], 4);
      init(sm->v_out[i], 4);
    }
    for (int i = 0; i < kSegs; ++i) {
      init(sm->seg_full[i], 1);
      init(sm->seg_empty[i], 25);   // softmax and producer warps, the product thread
    }
    for (int w = 0; w < 2; ++w) {
      init(sm->s_full[w], 1);
      init(sm->p_full[w], 8);
      init(sm->o_full[w], 1);
    }
    for (int i = 0; i < 8; ++i) {
      init(sm->row_pair[i], 2);
      if (i < 4) init(sm->row_quad[i], 4);
    }
    init(sm->q_full, 16);
    init(sm->all, 16);
    init(sm->drain, 1);
    sm->stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  griddep_wait();
  griddep_launch_dependents();
  if (warp == 24) tmem_alloc(smem_u32(&sm->tmem), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = sm->tmem;
  if (warp < 16) {
    softmax_warp(a, work, sm, smem, qs, tm, warp, lane);
  } else if (warp < 20) {
    producer<false>(a, sm, ring, smem + kStagesAt);
  } else if (warp < 24) {
    producer<true>(a, sm, ring, smem + kStagesAt);
  } else if (warp == 24) {
    if (lane == 0 && !products(sm, qs, ring, tm)) {
      // stopped: what was issued still has to end before its memory is given up
      flag(a.status, KVQ_DEV_TIMEOUT);
      tc_commit(smem_u32(&sm->drain));
      int never = 0;
      mbar_wait(smem_u32(&sm->drain), 0, &never);
    }
    __syncwarp();
  } else {
    loader(a, work, sm, qs + kStagesAt, lane);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 24) tmem_free(tm, 512);
}

// Run i's CTA merges the block that run i continues if run i - 1 began it: that run's last slot, then
// the first slots of run i and of those after it that still belong to the block.  A warp per row, four
// channels per lane.
__global__ void __launch_bounds__(256) attn_merge_kernel(const __grid_constant__ AttnArgs a,
                                                         const __grid_constant__ Work work) {
  griddep_wait();
  griddep_launch_dependents();
  const Cut cut = *work.cut;
  const int run = blockIdx.x + 1;
  if (run >= cut.runs) return;
  const First f = work.first[run];
  const int64_t lo = run_start(cut, run), prev = run_start(cut, run - 1);
  if (f.unit < 2 || f.unit - (lo - prev) > 1) return;
  const int64_t end = lo - f.unit + f.units;   // where the block ends
  int parts = 2;
  while (run + parts - 1 < cut.runs && run_start(cut, run + parts - 1) < end) ++parts;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto slot = [&](int z) { return (int64_t)(z == 0 ? 2 * run - 1 : 2 * (run + z - 1)) * work.rows; };
  for (int r = warp + 8 * blockIdx.y; r < f.nr; r += 8 * gridDim.y) {
    const int64_t row = (f.row0 + (f.r0 + r) / a.G) * a.Hq + f.h * a.G + (f.r0 + r) % a.G;
    // states 32 parts at a time, a lane each; then their rows, several in flight
    float m = -INFINITY, l = 0.0f, o[4] = {0, 0, 0, 0};
    for (int z0 = 0; z0 < parts; z0 += 32) {
      const bool there = z0 + lane < parts;
      const float mz = there ? work.m[slot(z0 + lane) + r] : -INFINITY, lz = there ? work.l[slot(z0 + lane) + r] : 0.0f;
      const float top = fmaxf(m, warp_max(mz)), f = m == -INFINITY ? 0.0f : exp2_approx(m - top);
      const float gz = mz == -INFINITY ? 0.0f : exp2_approx(mz - top);
      m = top;
      l = l * f + warp_sum(gz * lz);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] *= f;
      const int n = min(32, parts - z0);
#pragma unroll 8
      for (int z = 0; z < n; ++z) {
        const float g = __shfl_sync(0xffffffffu, gz, z);
        const float4 v = *reinterpret_cast<const float4*>(work.o + (slot(z0 + z) + r) * 128 + 4 * lane);
        o[0] = fmaf(g, v.x, o[0]);
        o[1] = fmaf(g, v.y, o[1]);
        o[2] = fmaf(g, v.z, o[2]);
        o[3] = fmaf(g, v.w, o[3]);
      }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) store_elem(a.out, row * 128 + 4 * lane + j, a.out_dtype, o[j] * inv);
    if (a.lse && lane == 0) a.lse[row] = l > 0.0f ? kLn2 * (m + log2f(l) - kLift) : -INFINITY;
  }
}

}  // namespace

namespace attn {
cudaError_t launch_merge(const AttnArgs& a, const Work& w, int runs, cudaStream_t s) {
  if (runs < 2) return cudaSuccess;
  return launch_pdl(attn_merge_kernel, dim3(runs - 1, (w.rows + 7) / 8), dim3(256), 0, s, a, w);
}
}  // namespace attn

// Expanding the pages first pays from more than one row block (256 rows) per sequence on, in batches; a sequence by
// itself has to bring more than 512 (and fewer than 2048).  Measured, us, without / with, 8 x 4 heads, rows per sequence: 13 sequences of
// 4096 tokens 256 rows 171 / 190, 384 rows 304 / 256, 2048 rows 908 / 613; 32 sequences of 2048 256 rows 234 / 228,
// 384 rows 450 / 319; 1 sequence of 18432 256 rows 87 / 116, 512 rows 115 / 134, 2048 rows 281 / 243.
bool attn_wide_pays(int num_seqs, int G, int64_t n_rows) { return n_rows * G > (int64_t)num_seqs * 256; }

// Blocks of 16 rows, a warp each, up to 64 rows a sequence; blocks of 256 on the whole CTA above.  Measured, us,
// narrow / whole CTA, 8 x 4 heads: 8 sequences over 32768 and fewer 16 rows 130 / 273, 48 rows 255 / 284, 64 rows
// 321 / 263; 64 sequences of 4096 16 rows 202 / 507, 48 rows 540 / 517, 64 rows 693 / 488; 1 sequence of 32768 16
// rows 81 / 89, 64 rows 97 / 87.  These have 64 rows in every sequence (the pages pass four times); in a ragged
// batch that few reach the sides meet later: 64 rows 199, 68 to 96 rows on the whole CTA 211 to 222.
constexpr int kNarrowRows = 64, kNarrowWarps = 8;
bool narrow(int G, int64_t max_new) { return max_new * G <= kNarrowRows; }
size_t make_work_for(int G, int64_t max_new, void* ws, Work* w, int* runs) {
  *runs = device_sm_count() * (narrow(G, max_new) ? kNarrowWarps : 1);
  return make_work(*runs, narrow(G, max_new) ? 16 : 256, G, max_new, ws, w);
}

size_t attn_paged_workspace(int G, int64_t max_new) {
  Work w;
  int runs;
  return make_work_for(G, max_new, nullptr, &w, &runs);
}

size_t attn_paged_workspace_upto(int G, int64_t max_new) {   // the narrow kernel has more runs, and slots
  const int64_t few = max_new < kNarrowRows / G ? max_new : kNarrowRows / G;
  const size_t a = attn_paged_workspace(G, max_new), b = attn_paged_workspace(G, few);
  return a > b ? a : b;
}

cudaError_t launch_attn_paged(const AttnArgs& args, cudaStream_t s) {
  AttnArgs a = args;
  int runs;
  Work w;
  const size_t small = make_work_for(a.G, a.b.max_rows, a.ws, &w, &runs);
  a.block = narrow(a.G, a.b.max_rows) ? 16 : 256;
  a.raw_tile = a.block == 16 ? 16 : 128;
  if (a.block == 16) {
    const cudaError_t e = launch_attn_narrow(a, w, runs, s);
    return e != cudaSuccess ? e : launch_merge(a, w, runs, s);
  }
  if (attn_wide_pays(a.b.num_seqs, a.G, a.b.n_rows) && a.ws_bytes >= small + attn_wide_bytes(a))
    return launch_attn_wide(a, w, runs, reinterpret_cast<char*>(a.ws) + small, s);
  cudaError_t e = cudaFuncSetAttribute(attn_tc_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  e = launch_pdl(attn_tc_kernel, dim3(runs), dim3(kThreads), kSmem, s, a, w);
  if (e != cudaSuccess) return e;
  return launch_merge(a, w, runs, s);
}

}  // namespace kvq
