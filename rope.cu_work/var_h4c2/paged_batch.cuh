// Flat grids over ragged batches: the units of all sequences end to end.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

// The sequence and the unit within it of flat unit `u`, found by warp 0 (32 sequences at a
// time) and handed to the CTA through shared memory; false past the last one.
template <typename UnitsOf>
__device__ __forceinline__ bool find_unit(int num_seqs, int u, UnitsOf units_of, int* seq, int* unit) {
  __shared__ int found[2];
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int base = 0, s_hit = -1, u_hit = 0;
    for (int s0 = 0; s0 < num_seqs; s0 += 32) {
      const int s = s0 + lane;
      const int n = s < num_seqs ? units_of(s) : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const bool hit = u >= base + incl - n && u < base + incl;
      const unsigned m = __ballot_sync(0xffffffffu, hit);
      if (m) {
        const int l = __ffs(m) - 1;
        s_hit = s0 + l;
        u_hit = u - base - __shfl_sync(0xffffffffu, incl - n, l);
        break;
      }
      base += __shfl_sync(0xffffffffu, incl, 31);
    }
    if (lane == 0) {
      found[0] = s_hit;
      found[1] = u_hit;
    }
  }
  __syncthreads();
  *seq = found[0];
  *unit = found[1];
  return *seq >= 0;
}

}  // namespace kvq
