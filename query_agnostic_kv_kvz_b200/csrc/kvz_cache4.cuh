// The paged 4-bit cache: its layout, and the device helpers that the kernels
// writing and reading it share.
//
// A page holds page_size rows of one head as page_size / 16 blocks.  A block
// of 16 rows is one contiguous record, so it moves as a single bulk copy, and
// its codes lie in the order in which the attention's matrix instructions
// take them: a lane reads its share of 16 keys as whole 16-byte words and
// widens it in registers, with nothing to transpose.  With NG = D / 64:
//   K codes   [16 rows][4 c][NG g][2 u] words: dims 64g + 16c + 8u + 0..7 as
//             nibbles 0, 2, 4, 6, 1, 3, 5, 7, the word rotated left by 3
//   V codes   [8 row pairs][8 r][NG g][2 w][2 rows] halves: dims 64g + 8r +
//             4w + 0..3 of one row as nibbles 0, 1, 2, 3
//   K scales  [16 rows][NG] words: bf16 step (low half), bf16 minimum (high)
//   V scales  the same
// The two rows of a V pair are the two halves of a word, so a row can be
// written without reading its neighbour's.
#pragma once

#include <cuda_bf16.h>

#include <cstdint>

#include "kvz.h"
#include "kvz_internal.h"
#include "kvz_sm100.cuh"

namespace kvz {

constexpr int kC4Rows = 16;                                   // rows of a block
constexpr uint32_t kFullMask = 0xffffffffu;

template <int D>
struct C4 {
  static constexpr int NG = D / 64;                           // groups of 64 dims, one (step, minimum) each
  static constexpr int V_OFF = 8 * D;
  static constexpr int KS_OFF = 16 * D;
  static constexpr int VS_OFF = 17 * D;
  static constexpr int BLOCK = 18 * D;                        // bytes of a block
  static constexpr int LPR = D / 8;                           // lanes that hold a row, 8 dims each
};

// The page id of block blk of head b (the caller has checked blk against the
// table's width), and the block's address there: null, and a report, for an
// id outside the pool.
__device__ __forceinline__ int32_t page_id(const Pages4& pg, int64_t b, uint32_t blk) {
  return pg.pages[b * pg.max_pages + page_of(pg, blk)];
}
template <int D>
__device__ __forceinline__ uint8_t* block_of(const Pages4& pg, int32_t id, uint32_t blk, int32_t* status) {
  if (id < 0 || id >= pg.n_pages) {
    report(status, KVZ_ERR_INVALID_ARG);
    return nullptr;
  }
  return pg.cache + (static_cast<int64_t>(id) * pg.blocks + (blk - page_of(pg, blk) * pg.blocks)) * C4<D>::BLOCK;
}
template <int D>
__device__ __forceinline__ uint8_t* block_at(const Pages4& pg, int64_t b, uint32_t blk, int32_t* status) {
  return block_of<D>(pg, page_id(pg, b, blk), blk, status);
}

// x (the low or high bf16 of w) + y, rounded once: one full-rate instruction,
// where a shift or mask to widen x first would take two issues of the
// half-rate integer pipe.
__device__ __forceinline__ float add_lo(uint32_t w, float y) {
  float d;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; add.rn.f32.bf16 %0, l, %2;}" : "=f"(d) : "r"(w), "f"(y));
  return d;
}
__device__ __forceinline__ float add_hi(uint32_t w, float y) {
  float d;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; add.rn.f32.bf16 %0, h, %2;}" : "=f"(d) : "r"(w), "f"(y));
  return d;
}
__device__ __forceinline__ float bf_lo(uint32_t w) { return add_lo(w, 0.0f); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return add_hi(w, 0.0f); }

__device__ __forceinline__ uint32_t min_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Quantisation of a row's group of 64 values, held by LANES lanes that differ
// in the low bits of the lane number (all lanes of the warp take part).  With m = min, r = max - min: step
// s = bf16(r * (1/15)), code = round((x - m) * (1/s)), every step one IEEE
// float32 operation, ties to even.  (r * (1/15) rounded to bf16 is at least
// r/15 * (1 - 2^-8), so a code is at most 15.06 before it is rounded.)  A step
// below 2^-126 is held as 0, with codes 0: its reciprocal leaves float32, and
// the whole group is within 2^-122 of m.  A group whose range is not finite (a
// NaN, an infinity or a range past float32) is held as step NaN, so reading it
// gives NaN.
struct Scale4 {
  float m, inv;
  uint32_t word;                                              // bf16 s, bf16 m
  bool fine;
};
// 1 / s for a positive normal bf16 s up to 2^125, correctly rounded: the
// approximate reciprocal and one Newton step, which agrees with division for
// every one of those 32,128 values, in 3 instructions without a slow path.
__device__ __forceinline__ float step_inverse(float s) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
  return __fmaf_rn(y, __fmaf_rn(-s, y, 1.0f), y);
}
// lo2, hi2: minima and maxima of the lane's own values, over even and odd ones.
template <int LANES>
__device__ __forceinline__ Scale4 group_scale(uint32_t lo2, uint32_t hi2) {
  // (min, -max) in one word, so that one minimum over the lanes serves both
  uint32_t v = __byte_perm(min_nan2(lo2, lo2 >> 16), max_nan2(hi2, hi2 >> 16) ^ 0x8000u, 0x5410);
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) v = min_nan2(v, __shfl_xor_sync(kFullMask, v, o));
  Scale4 q;
  q.m = bf_lo(v);
  const float r = add_hi(v ^ 0x80000000u, -q.m);
  q.fine = r < INFINITY;
  float s = __bfloat162float(__float2bfloat16_rn(__fmul_rn(r, 1.0f / 15.0f)));
  s = s < 0x1p-126f ? 0.0f : s;
  q.inv = s > 0.0f ? step_inverse(s) : 0.0f;
  q.word = q.fine ? ((__float_as_uint(s) >> 16) | (v << 16)) : 0x00007FC0u;
  return q;
}
// 0x4B400000 + the codes of the two values in w.
__device__ __forceinline__ void code2(uint32_t w, const Scale4& q, uint32_t& c0, uint32_t& c1) {
  c0 = __float_as_uint(__fadd_rn(__fmul_rn(add_lo(w, -q.m), q.inv), 12582912.0f));
  c1 = __float_as_uint(__fadd_rn(__fmul_rn(add_hi(w, -q.m), q.inv), 12582912.0f));
}
// Scale and codes (+ 0x4B400000) of a group that 8 lanes hold, 8 values each.
__device__ __forceinline__ bool quantise8(const uint4& x, uint32_t (&code)[8], uint32_t& sm) {
  const Scale4 q = group_scale<8>(min_nan2(min_nan2(x.x, x.y), min_nan2(x.z, x.w)),
                                  max_nan2(max_nan2(x.x, x.y), max_nan2(x.z, x.w)));
  code2(x.x, q, code[0], code[1]);
  code2(x.y, q, code[2], code[3]);
  code2(x.z, q, code[4], code[5]);
  code2(x.w, q, code[6], code[7]);
  sm = q.word;
  return q.fine;
}

// Sum of code[i] << shift with the constant 0x4B400000 parts taken out (the
// arithmetic is modulo 2^32, so they cancel exactly).
constexpr uint32_t kCodeBias = 0x4B400000u;

// A K word: 8 codes as nibbles 0, 2, 4, 6, 1, 3, 5, 7, rotated left by 3.
__device__ __forceinline__ uint32_t k_word(const uint32_t (&code)[8], bool fine) {
  constexpr uint32_t bias = kCodeBias * 0x11111111u;
  uint32_t w = code[0] + (code[1] << 16) + (code[2] << 4) + (code[3] << 20) + (code[4] << 8) + (code[5] << 24) +
               (code[6] << 12) + (code[7] << 28) - bias;
  w = fine ? w : 0u;
  return __funnelshift_l(w, w, 3);
}
// Two V units of one row: codes 0..3 in the low half, 4..7 in the high half.
__device__ __forceinline__ uint32_t v_units(const uint32_t (&code)[8], bool fine) {
  constexpr uint32_t bias = kCodeBias * 0x1111u;
  const uint32_t u0 = code[0] + (code[1] << 4) + (code[2] << 8) + (code[3] << 12) - bias;
  const uint32_t u1 = code[4] + (code[5] << 4) + (code[6] << 8) + (code[7] << 12) - bias;
  return fine ? __byte_perm(u0, u1, 0x5410) : 0u;
}

// Write one row pair's K codes: lane l of the row's D / 8 lanes holds dims
// 8l .. 8l + 7, which are one word of the row.
template <int D>
__device__ __forceinline__ void store_k(uint8_t* blk, int row, int l, const uint32_t (&code)[8], bool fine,
                                        uint32_t sm) {
  using L = C4<D>;
  const uint32_t w = k_word(code, fine);
  const int g = l / 8, c = (l % 8) / 2, u = l % 2;
  *reinterpret_cast<uint32_t*>(blk + row * (D / 2) + (c * L::NG * 2 + g * 2 + u) * 4) = w;
  if (l % 8 == 0) *reinterpret_cast<uint32_t*>(blk + L::KS_OFF + (row * L::NG + g) * 4) = sm;
}

// The same for V.  Lanes l and l ^ LPR hold the same dims of the pair's even
// and odd row; where both rows are written, each lane stores one whole word
// (all lanes take part in the exchange), else a written row's two halves.
template <int D>
__device__ __forceinline__ void store_v(uint8_t* blk, int row, int l, const uint32_t (&code)[8], bool fine,
                                        uint32_t sm, bool write) {
  using L = C4<D>;
  const uint32_t vu = v_units(code, fine), h0 = vu & 0xFFFFu, h1 = vu >> 16;
  const bool odd = (row & 1) != 0;
  const uint32_t got = __shfl_xor_sync(kFullMask, (odd ? h0 : h1) | (write ? 0x10000u : 0u), L::LPR);
  const bool both = write && (got & 0x10000u) != 0;
  const int g = l / 8, r = l % 8;
  uint8_t* at = blk + L::V_OFF + (row >> 1) * D + (r * L::NG + g) * 8;       // two words: dims 0..3, 4..7
  if (both) {
    const uint32_t w = odd ? ((got & 0xFFFFu) | (h1 << 16)) : (h0 | (got << 16));
    *reinterpret_cast<uint32_t*>(at + (odd ? 4 : 0)) = w;
  } else if (write) {
    *reinterpret_cast<uint16_t*>(at + (odd ? 2 : 0)) = static_cast<uint16_t>(h0);
    *reinterpret_cast<uint16_t*>(at + 4 + (odd ? 2 : 0)) = static_cast<uint16_t>(h1);
  }
  if (write && l % 8 == 0) *reinterpret_cast<uint32_t*>(blk + L::VS_OFF + (row * L::NG + g) * 4) = sm;
}

// Two codes, one in each half of w with its four bits from bit 3 up, as bf16.
__device__ __forceinline__ uint32_t code_bf2(uint32_t w) {
  uint32_t d;
  asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"((w & 0x00780078u) | 0x41804180u), "r"(0xC180C180u));   // 16 + code - 16
  return d;
}
__device__ __forceinline__ uint32_t fma_bf2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

}  // namespace kvz
