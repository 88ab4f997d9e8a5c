// The rotation of rotary positions on 16-byte vectors of bf16, shared by the
// rotary kernel and the cache's append kernel.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace kvz {

// Cosines and sines of pairs i0 .. i0 + 7 from a table row (cosines, then
// sines, `half` of each); the inverse turns the other way.
__device__ __forceinline__ void load_angles(const float* row, int half, int i0, int inverse, float (&c)[8],
                                            float (&s)[8]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float4 cc = reinterpret_cast<const float4*>(row + i0)[h];
    const float4 ss = reinterpret_cast<const float4*>(row + half + i0)[h];
    const float sg = inverse ? -1.0f : 1.0f;
    c[4 * h] = cc.x, c[4 * h + 1] = cc.y, c[4 * h + 2] = cc.z, c[4 * h + 3] = cc.w;
    s[4 * h] = sg * ss.x, s[4 * h + 1] = sg * ss.y, s[4 * h + 2] = sg * ss.z, s[4 * h + 3] = sg * ss.w;
  }
}

// (a, b) -> (a c - b s, b c + a s); products and sums rounded one by one.
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float x = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
  b = __fadd_rn(__fmul_rn(b, c), __fmul_rn(a, s));
  a = x;
}

__device__ __forceinline__ float rot_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float rot_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t rot_pack(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Pairs (element i of v0, element i of v1).
__device__ __forceinline__ void turn_halves(uint4& v0, uint4& v1, const float (&c)[8], const float (&s)[8]) {
  uint32_t* p = reinterpret_cast<uint32_t*>(&v0);
  uint32_t* q = reinterpret_cast<uint32_t*>(&v1);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a0 = rot_lo(p[i]), a1 = rot_hi(p[i]), b0 = rot_lo(q[i]), b1 = rot_hi(q[i]);
    turn_pair(a0, b0, c[2 * i], s[2 * i]);
    turn_pair(a1, b1, c[2 * i + 1], s[2 * i + 1]);
    p[i] = rot_pack(a0, a1);
    q[i] = rot_pack(b0, b1);
  }
}

// Pairs of neighbouring elements: 4 in v0 (angles 0..3), 4 in v1 (4..7).
__device__ __forceinline__ void turn_neighbours4(uint4& v, const float* c, const float* s) {
  uint32_t* p = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = rot_lo(p[i]), b = rot_hi(p[i]);
    turn_pair(a, b, c[i], s[i]);
    p[i] = rot_pack(a, b);
  }
}
__device__ __forceinline__ void turn_adjacent(uint4& v0, uint4& v1, const float (&c)[8], const float (&s)[8]) {
  turn_neighbours4(v0, c, s);
  turn_neighbours4(v1, c + 4, s + 4);
}

}  // namespace kvz
