// Rotation of one octet (8 consecutive channels) of a head row by its table row, shared by
// the norm-and-rotate kernel and the paged append.
#pragma once

#include "kvq_internal.cuh"

namespace kvq {

// The octet that `o` turns against: itself for interleaved pairs, in the half layout the one
// half a rotation away.  Octets past the rotation have no partner (themselves).
__device__ __forceinline__ int rope_partner(const RopeArgs& r, int o) {
  const int turned = r.rot >> 3, half = turned >> 1;
  if (r.inter || o >= turned) return o;
  return o < half ? o + half : o - half;
}

// cos and sin of octet o from its table row: half layout, one pair per channel (8 and 8);
// interleaved, one per two channels (4 and 4, in the first entries).
struct OctetTurn {
  float c[8], s[8];
};
__device__ __forceinline__ void rope_load(const RopeArgs& r, int64_t pos, int o, OctetTurn& t) {
  const float* row = r.table + pos * r.rot;
  const int half = r.rot >> 1;
  if (r.inter) {
    const float4 c = *reinterpret_cast<const float4*>(row + 4 * o);
    const float4 s = *reinterpret_cast<const float4*>(row + half + 4 * o);
    t.c[0] = c.x; t.c[1] = c.y; t.c[2] = c.z; t.c[3] = c.w;
    t.s[0] = s.x; t.s[1] = s.y; t.s[2] = s.z; t.s[3] = s.w;
  } else {
    const int i = 8 * o < half ? 8 * o : 8 * o - half;
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const float4 c = *reinterpret_cast<const float4*>(row + i + j);
      const float4 s = *reinterpret_cast<const float4*>(row + half + i + j);
      t.c[j] = c.x; t.c[j + 1] = c.y; t.c[j + 2] = c.z; t.c[j + 3] = c.w;
      t.s[j] = s.x; t.s[j + 1] = s.y; t.s[j + 2] = s.z; t.s[j + 3] = s.w;
    }
  }
}

// x (octet o) turned in place; p: the partner octet (half layout only).  Products and sums
// are rounded one by one, so the result does not depend on the compiler's contraction.
__device__ __forceinline__ void rope_turn(const RopeArgs& r, int o, const OctetTurn& t, float (&x)[8],
                                          const float (&p)[8]) {
  if (r.inter) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float a = x[2 * j], b = x[2 * j + 1];
      x[2 * j] = __fsub_rn(__fmul_rn(a, t.c[j]), __fmul_rn(b, t.s[j]));
      x[2 * j + 1] = __fadd_rn(__fmul_rn(b, t.c[j]), __fmul_rn(a, t.s[j]));
    }
  } else if (16 * o < r.rot) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __fsub_rn(__fmul_rn(x[j], t.c[j]), __fmul_rn(p[j], t.s[j]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __fadd_rn(__fmul_rn(x[j], t.c[j]), __fmul_rn(p[j], t.s[j]));
  }
}

// 8 consecutive elements stored in `dtype` (16 bytes for 16-bit types, two 16-byte stores
// for fp32), rounded to nearest even.
__device__ __forceinline__ uint32_t pack2(float a, float b, int dtype) {
  if (dtype == KVQ_F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void store8(void* base, int64_t i, int dtype, const float (&x)[8]) {
  if (dtype == KVQ_F32) {
    float4* d = reinterpret_cast<float4*>(reinterpret_cast<float*>(base) + i);
    d[0] = make_float4(x[0], x[1], x[2], x[3]);
    d[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(reinterpret_cast<uint16_t*>(base) + i) =
        make_uint4(pack2(x[0], x[1], dtype), pack2(x[2], x[3], dtype), pack2(x[4], x[5], dtype),
                   pack2(x[6], x[7], dtype));
  }
}

}  // namespace kvq
