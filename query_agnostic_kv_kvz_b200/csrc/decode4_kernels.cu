// Decode attention over the paged 4-bit cache.  For KV head b with n_b rows
// and the G <= 8 grouped queries of the new token:
//   out[b, g] = sum_j softmax_j(scale * <q_g, k_j>) v_j,
//   k_j = s_j code_j + m_j (and v_j alike) per group of 64 dims.
//
// The codes are whole numbers, exact in fp16, so both products run on them and
// the scales are applied to what comes out.  Keys, and V's dims, are the rows
// of the products and the G <= 8 queries their columns (mma.sync m16n8k16).
// tcgen05 takes its rows from shared or tensor memory, so every code would
// have to be widened there first, 2 bytes written and read for half a byte of
// the cache; here it is widened in the register that it was loaded to.
//   <q, k_j> = sum_groups s_j <q, code_j> + m_j sum(q)
//   out = sum_groups sum_j (p_j s_j) (code_j - 8) + p_j (m_j + 8 s_j)
// The low 11 bits of an fp16 number count its 2^-24s (subnormal numbers, and
// the first normal ones that go on from them), so two codes of a word widen
// with one mask.  V's codes are brought around 0 by one fp16 addition: a sum
// over many rows of values around 0 is far smaller than the same sum of 0..15,
// and would drown in the latter's rounding.  The tensor core truncates what it
// adds to, so it sums 32 rows at a time and the running output adds those in
// float32.
//
// fp16 operands.  q is scaled by a power of two to a largest entry of 2^14
// (and half of the dims by 1/16 more): its 8 bits stay exact down to 2^-27 of
// the largest entry, and what is smaller is held to 2^-35 of it.  A weight p s
// is the sum of two fp16 numbers, hi + lo, after a power of two of its own
// query and group of 64 dims, which follows the largest weight so far: it is
// held to 2^-24 of itself, as float32 holds it, and to 2^-35 of that largest.
// So neither the other group's steps nor a row of large values that hardly
// counts costs a group its bits.  (Three bf16 numbers, which need no power of
// two: 87.4 us against 77.4 for the heads below, at that time; one power for all that a warp
// reads, which loses the smaller group's bits: 76.4.)
//
// Bytes: 9/8 d per row (144 at d = 128), against 4 d of a bf16 cache.  At HBM's
// rate an SM would have to widen and multiply a row (both of K and V, all
// queries) in 6 clocks.  What bounds it is instructions that wait for one
// another: 64 heads of 32,768 rows at d = 128, G = 5 (302 MB) take 76.9 us, 3.9
// TB/s, the same loads without the arithmetic 55.  A stage of 32 rows costs a
// warp 694 instructions, which would be 5.4 clocks a row if every slot issued;
// 58% do, with 3.7 warps to a scheduler of which 1.2 could issue on average.  A
// warp waits 1.8 cycles per instruction for a fixed latency, 1.0 for a pipe.
// The integer pipe is 43% busy, the tensor pipe (48 products) 32%.
//
// One CTA of 8 warps takes an equal share of the work of all heads, whatever
// the heads' lengths (a share may end one head and begin others).  A warp
// brings its blocks in by bulk copy through a ring of its own, 32 rows a stage
// (one copy where they share a page), and keeps a running (reference, sum,
// output) per query; the warps merge in shared memory at the end of each
// head's part.  A head that several CTAs read leaves one partial per CTA,
// which a second launch joins in order: no atomics, and identical inputs give
// identical results.  A wait that expires makes NaN of the heads that its CTA
// still had to read.  (One CTA of 16 warps per SM: 82.3 against 81 us, and
// 31.9 against 24.3 at 96 uneven heads; 12 warps of 168 registers: 88.)
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "kvz.h"
#include "kvz_cache4.cuh"
#include "kvz_internal.h"
#include "kvz_launch.cuh"
#include "kvz_sm100.cuh"

namespace cg = cooperative_groups;

namespace kvz {

namespace {

constexpr int kD4Warps = 8;
constexpr int kD4Threads = kD4Warps * 32;
constexpr int kD4Stages = 2;
constexpr int kD4MinBlocks = 2 * kD4Warps;                    // a CTA's share is at least a stage per warp
// What beginning another head costs a CTA (its queries, the ring's switch, the
// join of the warps), counted as blocks.  us with 0, 16, 24, 40 and 72 (the
// least for every d, G, page size and spread of lengths that was measured):
//   64 heads of 32,768 rows    d 128  G 5  pages 128   80.6  78.9  77.6  77.2  78.5
//                              d 128  G 1         64   78.8  77.4  75.6  75.6  77.2
//                              d 64   G 8         64   51.0  50.2  48.6  48.2  49.7
//   96 uneven heads, 5,001     d 64   G 8         16   23.9  21.5  20.8  20.2  20.6
//   rows in the mean           d 128  G 4         64   33.0  30.0  28.4  27.8  28.7
//   40 uneven of 20,000        d 128  G 8         16   42.7  41.2  40.4  39.5  40.8
//   500 uneven of 1,500        d 64   G 2        128   37.7  32.3  31.4  29.6  32.3
//   12 uneven of 60,000        d 64   G 1         64   23.5  22.6  22.3  21.2  21.5
constexpr int kD4HeadCost = 40;
constexpr int kD4Counts = 1024;                               // head counts kept in shared memory
constexpr float kD4Slack = 7.0f;                              // log2 by which a logit may pass the reference
// Outputs are summed times 2^-16, so they leave float32 later than the values'
// own sum would, although a weight may be 2^7: V may come as near to float32's
// end as quantisation takes it.  (As a reference 2^16 higher, which scales the
// weights themselves, it cost their exponents 4 bits: errors of 4.2e-7 instead
// of 2.5e-7 of 8 heads of 2,457 rows.)
constexpr float kD4Out = 0x1p-16f;

// Weights p s go to fp16 times a power of two per query and group that follows
// the largest of them: one past kD4WeightTop brings it down so that the stage's
// largest is between 2^10 and 2^11, and it grows again as weights shrink under
// a reference that moves.
constexpr float kD4WeightTop = 32768.0f;
constexpr float kD4MulTop = 0x1p126f;                         // where the power begins
__device__ __forceinline__ uint32_t field(float x) { return __float_as_uint(x) >> 23; }
__device__ __forceinline__ float power(uint32_t field) { return __uint_as_float(field << 23); }

template <int D>
struct D4 {
  static constexpr int KS = D / 16;                           // k-steps of Q K^T
  static constexpr int MT = D / 16;                           // 16-dim tiles of the output
  static constexpr int STAGE = 2 * C4<D>::BLOCK;              // 32 rows
  static constexpr int RING = kD4Warps * kD4Stages * STAGE;
  static constexpr int O_OFF = RING;                          // float [warps][8][D]
  static constexpr int SMEM = RING + kD4Warps * 8 * D * 4;
};
static_assert(D4<128>::SMEM <= 107 * 1024, "two CTAs per SM");

__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1, float c0, float c1, float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
// Two float32 operations in one instruction.
__device__ __forceinline__ void add2(float& a0, float& a1, float b0, float b1) {
  asm("{.reg .b64 x, y; mov.b64 x, {%0, %1}; mov.b64 y, {%2, %3}; add.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x;}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}
__device__ __forceinline__ void fma2(float& a0, float& a1, float b0, float b1, float c0, float c1) {
  asm("{.reg .b64 x, y, z; mov.b64 x, {%0, %1}; mov.b64 y, {%2, %3}; mov.b64 z, {%4, %5}; fma.rn.f32x2 x, x, y, z; "
      "mov.b64 {%0, %1}, x;}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void mul2(float& a0, float& a1, float b0, float b1) {
  asm("{.reg .b64 x, y; mov.b64 x, {%0, %1}; mov.b64 y, {%2, %3}; mul.rn.f32x2 x, x, y; mov.b64 {%0, %1}, x;}"
      : "+f"(a0), "+f"(a1)
      : "f"(b0), "f"(b1));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The low 11 bits of a small fp16 number count its 2^-24s (exponents 0 and 1
// join there), so codes masked out of a word are fp16 numbers already.  V's,
// times 2^15, are normal ones: the tensor core aligns products by exponent
// fields and cuts a subnormal operand's short, which costs a sum of thousands
// of rows 4 of its bits, a logit's 128 products nothing that its rounding to
// float32 does not.
constexpr uint32_t kNormal = 0x78007800u;                     // 2^15, twice
// Two codes, one in each half of w with its four bits from bit SH up, as fp16
// 2^SH (code - 8) 2^-9.
template <int SH>
__device__ __forceinline__ uint32_t around0(uint32_t w) {
  static_assert(SH == 0 || SH == 4, "");
  constexpr uint32_t mask = 0x000F000Fu << SH, off = SH == 0 ? 0xA400A400u : 0xB400B400u;     // -8 2^-9, -128 2^-9
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(w & mask), "r"(kNormal), "r"(off));
  return d;
}
__device__ __forceinline__ uint32_t pack_h2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// w less the fp16 in the low (high) half of h, exact where h is w rounded; s kD4Out for
// the bf16 s in the low half of its word; and (s * 8 + m) kD4Out for the m in its high
// half.  Mixed instructions, where widening first would take another.
__device__ __forceinline__ float less_lo(float w, uint32_t h) {
  float d;
  asm("{.reg .b16 l, h, m; mov.b32 {l, h}, %1; mov.b16 m, 0xBC00; fma.rn.f32.f16 %0, l, m, %2;}" : "=f"(d) : "r"(h), "f"(w));
  return d;
}
__device__ __forceinline__ float less_hi(float w, uint32_t h) {
  float d;
  asm("{.reg .b16 l, h, m; mov.b32 {l, h}, %1; mov.b16 m, 0xBC00; fma.rn.f32.f16 %0, h, m, %2;}" : "=f"(d) : "r"(h), "f"(w));
  return d;
}
__device__ __forceinline__ float step_out(uint32_t w) {
  float d;
  asm("{.reg .b16 l, h, f; mov.b32 {l, h}, %1; mov.b16 f, 0x3780; fma.rn.f32.bf16 %0, l, f, 0f00000000;}"
      : "=f"(d)
      : "r"(w));
  return d;
}
__device__ __forceinline__ float middle(uint32_t w) {
  float d;
  asm("{.reg .b16 l, h, f, f8; .reg .f32 m; mov.b32 {l, h}, %1; mov.b16 f, 0x3780; mov.b16 f8, 0x3900; "
      "fma.rn.f32.bf16 m, h, f, 0f00000000; fma.rn.f32.bf16 %0, l, f8, m;}"
      : "=f"(d) : "r"(w));
  return d;
}
// 8x8 matrix of 16-bit entries, a row's pair 2c, 2c + 1 in lane (row, c): transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "");
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 4) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  }
}

// Summed outputs over their denominator.
__device__ __forceinline__ float4 quotient(const float4& sum, float Ls) {
  const float l = Ls * kD4Out;
  return make_float4(sum.x / l, sum.y / l, sum.z / l, sum.w / l);
}

// Loads that stay behind the wait for the kernels before this one.
__device__ __forceinline__ int load_int(const int32_t* p) {
  int v;
  asm volatile("ld.global.b32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}
__device__ __forceinline__ uint4 load_16(const void* p) {
  uint4 v;
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ int64_t blocks_of(int c, int64_t cap) {
  return c < 0 || c > cap ? 0 : (c + kC4Rows - 1) / kC4Rows;
}
// A head's weight in the shares: its blocks, behind kD4HeadCost more that stand for its beginning.
__device__ __forceinline__ int64_t weight_of(int c, int64_t cap) {
  const int64_t n = blocks_of(c, cap);
  return n > 0 ? n + kD4HeadCost : 0;
}

// Inclusive scan over the CTA's threads; returns the sum.
__device__ __forceinline__ int64_t cta_scan(int64_t v, int64_t& inc, int64_t* s_red) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(kFullMask, inc, o);
    if (lane >= o) inc += y;
  }
  __syncthreads();                                            // the last scan's sums are read
  if (lane == 31) s_red[warp] = inc;
  __syncthreads();
  int64_t all = 0;
#pragma unroll
  for (int i = 0; i < kD4Warps; ++i) {
    if (i < warp) inc += s_red[i];
    all += s_red[i];
  }
  return all;
}

// Blocks [a0, a1) of head b's `count` rows; none: b < 0.  Of their 32-row
// stages every 2^spread-th is the CTA's; those go to its warps in turn.
struct Part4 {
  int b, count, a0, a1;
  __device__ __forceinline__ int stages(int warp, int spread) const {
    const int n = b < 0 ? 0 : (a1 - a0 + (2 << spread) - 1) >> (1 + spread);
    return n > warp ? (n - warp + kD4Warps - 1) / kD4Warps : 0;
  }
  __device__ __forceinline__ int block(int warp, int i, int spread) const {
    return a0 + ((2 * (warp + kD4Warps * i)) << spread);
  }
};

// A warp's ring of stages, kept full across the parts that its CTA reads one
// after another.  Where stages lie in the pool is looked up 32 at a time, a
// lane each.
template <int D, bool TEST>
struct Ring4 {
  uint8_t* ring;
  uint64_t* bar;
  uint32_t used;                                              // stages taken
  int issued;                                                 // of the current part's (and then the next one's) stages
  int at0, at1;                                               // pool blocks of stage lane, lane + 32, ...
  bool placed;                                                // the first 32 of them are there from the start

  // The page ids of a stage's two blocks, blk and blk + 1, of head b (the second as the first from block `end` on).
  static __device__ __forceinline__ int2 ids(const Dec4Args& p, int b, int blk, int end) {
    const int32_t* const row_pages = p.pg.pages + static_cast<int64_t>(b) * p.pg.max_pages;
    const uint32_t pi0 = page_of(p.pg, static_cast<uint32_t>(blk));
    const uint32_t pi1 = blk + 1 < end ? page_of(p.pg, static_cast<uint32_t>(blk) + 1) : pi0;
    return make_int2(load_int(row_pages + pi0), load_int(row_pages + pi1));
  }
  __device__ __forceinline__ void place(const Dec4Args& p, int2 id, int blk) {
    if (id.x < 0 || id.x >= p.pg.n_pages || id.y < 0 || id.y >= p.pg.n_pages) {
      report(p.status, KVZ_ERR_INVALID_ARG);                  // page 0 stands in, so the read stays inside
      id.x = id.x < 0 || id.x >= p.pg.n_pages ? 0 : id.x;
      id.y = id.y < 0 || id.y >= p.pg.n_pages ? 0 : id.y;
    }
    const uint32_t pi0 = page_of(p.pg, static_cast<uint32_t>(blk)), pi1 = page_of(p.pg, static_cast<uint32_t>(blk) + 1);
    at0 = id.x * static_cast<int>(p.pg.blocks) + blk - static_cast<int>(pi0 * p.pg.blocks);
    at1 = pi1 == pi0 ? at0 + 1 : id.y * static_cast<int>(p.pg.blocks);
  }
  __device__ __forceinline__ void look_up(const Dec4Args& p, const Part4& t, int warp, int i, int spread) {
    if (i >= t.stages(warp, spread)) return;
    const int blk = t.block(warp, i, spread);
    place(p, ids(p, t.b, blk, t.a1), blk);
  }
  // Issue the copies of stage i of part t, `ahead` stages past the one now due.
  __device__ __forceinline__ void issue(const Dec4Args& p, const Part4& t, int warp, int lane, int i, int ahead,
                                        int spread) {
    using L = C4<D>;
    if ((i & 31) == 0 && !(placed && i == 0)) look_up(p, t, warp, i + lane, spread);
    const int from0 = __shfl_sync(kFullMask, at0, i & 31), from1 = __shfl_sync(kFullMask, at1, i & 31);
    if (TEST && i == 0 && warp == 0 && t.b == p.hold_head && (p.hold_cta < 0 || blockIdx.x == p.hold_cta)) return;
    if (lane == 0) {
      const uint32_t st = (used + static_cast<uint32_t>(ahead)) % kD4Stages;
      uint8_t* const dst = ring + st * D4<D>::STAGE;
      const bool two = t.block(warp, i, spread) + 1 < t.a1, joined = two && from1 == from0 + 1;
      mbar_arrive_expect_tx(&bar[st], two ? 2 * L::BLOCK : L::BLOCK);
      bulk_load(dst, p.pg.cache + static_cast<int64_t>(from0) * L::BLOCK, joined ? 2 * L::BLOCK : L::BLOCK, &bar[st]);
      if (two && !joined)
        bulk_load(dst + L::BLOCK, p.pg.cache + static_cast<int64_t>(from1) * L::BLOCK, L::BLOCK, &bar[st]);
    }
  }
  // The next stage that is not under way: of part t (n stages), then of the part after it (all - n), which lies in
  // shared memory since it is looked at so rarely.
  __device__ __forceinline__ void issue_next(const Dec4Args& p, const Part4& t, const Part4* then, int n, int warp,
                                             int lane, int ahead, int spread) {
    if (issued < n) issue(p, t, warp, lane, issued, ahead, spread);
    else issue(p, *then, warp, lane, issued - n, ahead, spread);
    ++issued;
  }
  // Let the copies under way land (bounded), behind `taken` stages done with, before the CTA leaves early.
  __device__ __forceinline__ void drain(int lane, int taken) {
    if (lane == 0)
      for (int k = 0; k < issued - taken; ++k)
        mbar_wait_for(&bar[(used + k) % kD4Stages], ((used + k) / kD4Stages) & 1u, 20000000ull);
  }
};

// A lane's share of head b's queries: query lane / 4, 16 dims of each group.
template <int D>
struct Query4 {
  uint4 v[D / 64][2];
  __device__ __forceinline__ void load(const Dec4Args& p, int64_t b) {
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int g = 0; g < D / 64; ++g)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        v[g][u] = make_uint4(0u, 0u, 0u, 0u);
        if (r < p.G) v[g][u] = load_16(p.q + (b * p.G + r) * D + 64 * g + 16 * c + 8 * u);
      }
  }
};

// One part of a head, read by the CTA's warps 32 rows at a time; each leaves its
// reference, sum and output per query in shared memory.  `then` (in shared
// memory) is the part that the CTA reads next.  False in a warp whose wait
// expired.
template <int D, bool TEST>
__device__ __forceinline__ bool read_part(const Dec4Args& p, const Query4<D>& query, const Part4& part,
                                          const Part4* then, Ring4<D, TEST>& q,
                                          volatile int* abort_flag, float* s_o, float (*s_m)[8], float (*s_l)[8],
                                          int spread) {
  using L = C4<D>;
  using S = D4<D>;
  constexpr int NG = L::NG;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int r = lane >> 2, c = lane & 3;
  const auto& v = query.v;
  const int n = part.stages(warp, spread), all = n + then->stages(warp, spread);
  while (q.issued < kD4Stages && q.issued < all) q.issue_next(p, part, then, n, warp, lane, q.issued, spread);   // warp-uniform

  // Q^T fragments (columns = queries; those >= G are zero), scaled by a power of
  // two to a largest exponent of 14; lane (r, c) loads query r and then works on
  // queries 2c, 2c + 1, so it takes their factor and sum(q) per group from there
  uint32_t qb[S::KS][2];
  float qs[NG][2], c2[2];
  {
    uint32_t ef = 0;                                        // largest exponent field of the query
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t w[4] = {v[g][u].x, v[g][u].y, v[g][u].z, v[g][u].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) ef = max(ef, max((w[k] >> 23) & 0xFFu, (w[k] >> 7) & 0xFFu));
      }
    ef = max(ef, __shfl_xor_sync(kFullMask, ef, 1));
    ef = max(ef, __shfl_xor_sync(kFullMask, ef, 2));
    // an infinity or NaN stays one whatever the factor; an exponent below -112 needs no more than 2^126
    const uint32_t fe = ef == 255u || ef == 0u ? 127u : min(268u - ef, 253u);
    const float f = __uint_as_float(fe << 23), back = p.c2 * __uint_as_float((254u - fe) << 23);
    constexpr float unit = 0x1p-21f;                        // 8 * 2^-24: what one code counts in the products
    c2[0] = __shfl_sync(kFullMask, back, 8 * c) * (1.0f / unit);
    c2[1] = __shfl_sync(kFullMask, back, 8 * c + 4) * (1.0f / unit);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float sum = 0.0f;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t w[4] = {v[g][u].x, v[g][u].y, v[g][u].z, v[g][u].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float x0 = bf_lo(w[k]) * f, x1 = bf_hi(w[k]) * f;
          constexpr float form[2] = {1.0f, 0.0625f};        // the codes these dims meet are 8- and 128-fold
          qb[4 * g + 2 * u + k / 2][k % 2] = pack_h2(x0 * form[k % 2], x1 * form[k % 2]);
          sum += x0 + x1;
        }
      }
      sum += __shfl_xor_sync(kFullMask, sum, 1);
      sum += __shfl_xor_sync(kFullMask, sum, 2);
      qs[g][0] = __shfl_sync(kFullMask, sum, 8 * c) * unit;
      qs[g][1] = __shfl_sync(kFullMask, sum, 8 * c + 4) * unit;
    }
  }

  float o[S::MT][4];                                        // out^T tiles (dims x queries 2c, 2c + 1), times mul
#pragma unroll
  for (int t = 0; t < S::MT; ++t) o[t][0] = o[t][1] = o[t][2] = o[t][3] = 0.0f;
  float m_neg[2] = {INFINITY, INFINITY}, thr[2] = {-INFINITY, -INFINITY};   // -reference of queries 2c, 2c + 1
  float l_run[2] = {0.0f, 0.0f};                            // of the same, this lane's keys
  float om[NG][2];                                          // sum of p (m + 8 s), the same
#pragma unroll
  for (int g = 0; g < NG; ++g) om[g][0] = om[g][1] = 0.0f;
  float mul[NG][2];                                         // the weights' power of two, the same
#pragma unroll
  for (int g = 0; g < NG; ++g) mul[g][0] = mul[g][1] = kD4MulTop;

  bool ok = true;
  for (int i = 0; i < n; ++i) {
    const uint32_t st = q.used % kD4Stages;
    ok = mbar_wait_warp(&q.bar[st], (q.used / kD4Stages) & 1u, abort_flag, p.status, TEST ? p.wait_ns : kWaitLimitNs);
    if (!ok) {                                                // warp-uniform
      q.drain(lane, i);
      break;
    }
    const uint8_t* stage = q.ring + st * S::STAGE;
    const int blk0 = part.block(warp, i, spread);
    // rows of the stage that count: the head may end inside it, and this CTA's share after its first block (what
    // lies past them, in the page or left in the stage, has no influence)
    const int rows = min(part.count - blk0 * kC4Rows, (part.a1 - blk0) * kC4Rows);

    // ---- scores of keys 16k + 8h + r of the stage and queries 2c + e
    float x[2][2][2];                                       // [k][h][e]
    uint32_t vp[2][2][NG];                                  // V scales of those keys
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      __syncwarp();                                         // keeps the next block's loads (and registers) behind this one's use
      const uint8_t* blk = stage + k * L::BLOCK;
      uint32_t kw[2][2 * NG], kp[2][NG];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        lds_words(blk + (8 * h + r) * (D / 2) + c * (8 * NG), kw[h]);
        lds_words(blk + L::KS_OFF + (8 * h + r) * (4 * NG), kp[h]);
        lds_words(blk + L::VS_OFF + (8 * h + r) * (4 * NG), vp[k][h]);
        x[k][h][0] = x[k][h][1] = 0.0f;
      }
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          // nibbles 0, 4 and 1, 5 of the rotated words, then 2, 6 and 3, 7: bits 3..6 and 7..10 of either half
          const uint32_t w0 = kw[0][2 * g + u], w1 = kw[1][2 * g + u];
          const uint32_t y0 = __funnelshift_r(w0, w0, 8), y1 = __funnelshift_r(w1, w1, 8);
          constexpr uint32_t lo = 0x00780078u, hi = 0x07800780u;
          const uint32_t(&q0)[2] = qb[4 * g + 2 * u], (&q1)[2] = qb[4 * g + 2 * u + 1];
          mma_16816(acc, w0 & lo, w1 & lo, w0 & hi, w1 & hi, q0[0], q0[1], acc[0], acc[1], acc[2], acc[3]);
          mma_16816(acc, y0 & lo, y1 & lo, y0 & hi, y1 & hi, q1[0], q1[1], acc[0], acc[1], acc[2], acc[3]);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float s = bf_lo(kp[h][g]), m = bf_hi(kp[h][g]);
#pragma unroll
          for (int e = 0; e < 2; ++e) x[k][h][e] = fmaf(s, acc[2 * h + e], fmaf(m, qs[g][e], x[k][h][e]));
        }
      }
    }
    if (rows < 2 * kC4Rows) {                               // warp-uniform
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (16 * k + 8 * h + r >= rows) {
            x[k][h][0] = x[k][h][1] = -INFINITY;
#pragma unroll
            for (int g = 0; g < NG; ++g) vp[k][h][g] = 0u;
          }
    }
    // ---- softmax against references that move only when a logit passes them by 2^7
    float xm[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) xm[e] = fmaxf(max3(x[0][0][e], x[0][1][e], x[1][0][e]), x[1][1][e]);
    if (__any_sync(kFullMask, xm[0] > thr[0] || xm[1] > thr[1])) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = xm[e];
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kFullMask, mx, sh));
        if (mx > thr[e]) {
          const float mn = mx * c2[e];
          const float al = ex2(-m_neg[e] - mn);             // 0 the first time
          m_neg[e] = -mn;
          thr[e] = (mn + kD4Slack) / c2[e];
          l_run[e] *= al;
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            om[g][e] *= al;
            // weights shrink by al, so their power of two grows by as many bits
            const uint32_t now = field(mul[g][e]), to = min(now + 127u - field(al), field(kD4MulTop));
            const float f = al * power(127u + min(to - now, 127u));
            mul[g][e] = power(to);
#pragma unroll
            for (int t = 4 * g; t < 4 * g + 4; ++t) o[t][e] *= f, o[t][2 + e] *= f;
          }
        }
      }
    }
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int h = 0; h < 2; ++h) {                           // the weights p
        fma2(x[k][h][0], x[k][h][1], c2[0], c2[1], m_neg[0], m_neg[1]);
        x[k][h][0] = ex2(x[k][h][0]);
        x[k][h][1] = ex2(x[k][h][1]);
        add2(l_run[0], l_run[1], x[k][h][0], x[k][h][1]);
      }

    // ---- the weights p s times their power of two
    float w[NG][2][2][2], wm = 0.0f;
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float m8 = middle(vp[k][h][g]);
          float y0 = x[k][h][0], y1 = x[k][h][1];
          fma2(y0, y1, m8, m8, om[g][0], om[g][1]);
          om[g][0] = y0, om[g][1] = y1;
#pragma unroll
          for (int e = 0; e < 2; ++e) w[g][k][h][e] = step_out(vp[k][h][g]);
          mul2(w[g][k][h][0], w[g][k][h][1], x[k][h][0], x[k][h][1]);   // (not past 2^115; the power alone may be)
          mul2(w[g][k][h][0], w[g][k][h][1], mul[g][0], mul[g][1]);
          wm = max3(wm, w[g][k][h][0], w[g][k][h][1]);
        }
    if (__any_sync(kFullMask, wm > kD4WeightTop)) {
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = 0.0f;                                   // the stage's largest weight
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h) top = fmaxf(top, x[k][h][e] * step_out(vp[k][h][g]));
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) top = fmaxf(top, __shfl_xor_sync(kFullMask, top, sh));
          const uint32_t now = field(mul[g][e]), to = min(now, 264u - field(top));
          const float f = power(127u - min(now - to, 127u));  // (past 2^-126: 0)
          mul[g][e] = power(to);
#pragma unroll
          for (int t = 4 * g; t < 4 * g + 4; ++t) o[t][e] *= f, o[t][2 + e] *= f;
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              w[g][k][h][e] = x[k][h][e] * step_out(vp[k][h][g]) * mul[g][e];
        }
    }

    // ---- out^T += V^T (p s)
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      // the weights as hi + lo in fp16, transposed from (key r; queries) to (query r; keys 2c, 2c + 1)
      uint32_t hi[2][2], lo[2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t part = pack_h2(w[g][k][h][0], w[g][k][h][1]);
          hi[k][h] = transpose8(part);
          lo[k][h] = transpose8(pack_h2(less_lo(w[g][k][h][0], part), less_hi(w[g][k][h][1], part)));
        }
      __syncwarp();
      uint32_t vw[2][2][2];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int t = 0; t < 2; ++t)
          lds_words(stage + k * L::BLOCK + L::V_OFF + (4 * t + c) * D + (r * NG + g) * 8, vw[k][t]);
#pragma unroll
      for (int wl = 0; wl < 2; ++wl)
#pragma unroll
        for (int h = 0; h < 2; ++h) {                       // dims 64g + 8r + 4wl + 2h, + 1
          uint32_t a[2][4];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t y0 = vw[k][0][wl], y1 = vw[k][1][wl];
            if (h == 1) y0 >>= 8, y1 >>= 8;
            a[k][0] = around0<0>(y0), a[k][1] = around0<4>(y0), a[k][2] = around0<0>(y1), a[k][3] = around0<4>(y1);
          }
          float d[4];
          mma_16816(d, a[0][0], a[0][1], a[0][2], a[0][3], lo[0][0], lo[0][1], 0.0f, 0.0f, 0.0f, 0.0f);
          mma_16816(d, a[1][0], a[1][1], a[1][2], a[1][3], lo[1][0], lo[1][1], d[0], d[1], d[2], d[3]);
          mma_16816(d, a[0][0], a[0][1], a[0][2], a[0][3], hi[0][0], hi[0][1], d[0], d[1], d[2], d[3]);
          mma_16816(d, a[1][0], a[1][1], a[1][2], a[1][3], hi[1][0], hi[1][1], d[0], d[1], d[2], d[3]);
          float(&acc)[4] = o[4 * g + 2 * wl + h];
          add2(acc[0], acc[1], d[0], d[1]);
          add2(acc[2], acc[3], d[2], d[3]);
        }
    }
    __syncwarp();                                             // the stage is read
    ++q.used;
    if (q.issued < all) q.issue_next(p, part, then, n, warp, lane, kD4Stages - 1, spread);
  }
  if (ok) q.issued -= n;                                      // the rest belongs to the next part

  // ---- this head's part is read: the warps' states to shared memory (free again since the CTA's last barrier)
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int sh = 4; sh < 32; sh <<= 1) {
      l_run[e] += __shfl_xor_sync(kFullMask, l_run[e], sh);
#pragma unroll
      for (int g = 0; g < NG; ++g) om[g][e] += __shfl_xor_sync(kFullMask, om[g][e], sh);
    }
    if (r == 0) {
      s_m[warp][2 * c + e] = -m_neg[e];
      s_l[warp][2 * c + e] = l_run[e];
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float* d0 = s_o + (warp * 8 + 2 * c + e) * D + 64 * g + 8 * r;
      const float s_out = power(254u + 9u - field(mul[g][e]));   // 2^9 / mul
#pragma unroll
      for (int wl = 0; wl < 2; ++wl) {
        const float(&x0)[4] = o[4 * g + 2 * wl], (&x1)[4] = o[4 * g + 2 * wl + 1];
        // odd dims' codes were taken 16-fold
        *reinterpret_cast<float4*>(d0 + 4 * wl) =
            make_float4(fmaf(x0[e], s_out, om[g][e]), fmaf(x0[2 + e], s_out * 0.0625f, om[g][e]),
                        fmaf(x1[e], s_out, om[g][e]), fmaf(x1[2 + e], s_out * 0.0625f, om[g][e]));
      }
    }
  }
  return ok;
}

// The warps' states of query g joined, for the four dims from 4 e4 on (of the
// G * D): reference M, sum, output relative to M.
template <int D>
__device__ __forceinline__ float4 join_warps(int e4, const float* s_o, const float (*s_m)[8], const float (*s_l)[8],
                                             float& M, float& Ls) {
  const int g = 4 * e4 / D;
  M = -INFINITY, Ls = 0.0f;
#pragma unroll
  for (int w = 0; w < kD4Warps; ++w) M = fmaxf(M, s_m[w][g]);
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int w = 0; w < kD4Warps; ++w) {
    const float mw = s_m[w][g], lw = s_l[w][g];
    const bool none = mw == -INFINITY && lw == 0.0f;          // the warp had no block
    const float wgt = none ? 0.0f : exp2f(mw - M);
    const float4 v = *reinterpret_cast<const float4*>(s_o + w * 8 * D + 4 * e4);
    Ls = fmaf(lw, wgt, Ls);
    acc.x = fmaf(v.x, wgt, acc.x), acc.y = fmaf(v.y, wgt, acc.y);
    acc.z = fmaf(v.z, wgt, acc.z), acc.w = fmaf(v.w, wgt, acc.w);
  }
  return acc;
}

template <int D, bool TEST>
__global__ void __launch_bounds__(kD4Threads, 2) decode_int4_kernel(Dec4Args p) {
  using S = D4<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kD4Warps * kD4Stages];
  __shared__ int s_abort;
  __shared__ int s_cnt[kD4Counts];
  __shared__ int64_t s_red[kD4Warps];
  __shared__ int64_t s_find[2];                               // head that holds the first block, its first block
  __shared__ Part4 s_then;
  __shared__ float s_m[kD4Warps][8], s_l[kD4Warps][8];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int G = p.G;

  if (tid < kD4Warps * kD4Stages) mbar_init(&full[tid], 1);   // (the scan's barriers order this before its use)
  if (tid == 0) s_abort = 0;
  fence_mbar_init();

  let_next_start();                                           // the merge may take its places as CTAs leave
  after_prior();

  // ---- this CTA's share [u0, u1) of all heads' weights: their sum, then the head that holds u0
  int64_t mine = 0;
  for (int64_t b = tid; b < p.B; b += kD4Threads) {
    const int n = load_int(p.counts + b);
    if (b < kD4Counts) s_cnt[b] = n;
    mine += weight_of(n, p.cap);
  }
  int64_t inc;                                                // weights of the threads up to this one
  int64_t total = cta_scan(mine, inc, s_red);
  int64_t quota = (total + kD4Workers - 1) / kD4Workers;
  quota = quota < kD4MinBlocks ? kD4MinBlocks : quota;
  const int64_t u0 = blockIdx.x * quota;
  const int64_t u1 = u0 + quota < total ? u0 + quota : total;
  auto count_of = [&](int64_t b) -> int { return b < kD4Counts ? s_cnt[b] : load_int(p.counts + b); };

  // heads without rows get their outputs here, heads with a bad count a report
  for (int64_t b = blockIdx.x; b < p.B; b += kD4Workers) {
    const int n = count_of(b);
    if (n == 0) {
      for (int e = tid; e < G * D; e += kD4Threads) p.out[b * G * D + e] = 0.0f;
      if (p.lse2 != nullptr && tid < G) p.lse2[b * G + tid] = -INFINITY;
    } else if ((n < 0 || n > p.cap) && tid == 0) {
      report(p.status, KVZ_ERR_INVALID_ARG);
    }
  }
  if (u0 >= u1) {
    if (tid == 0) p.cont[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  if (p.B <= kD4Threads) {                                    // a head per thread: the scan has it already
    if (u0 >= inc - mine && u0 < inc) {
      s_find[0] = tid;
      s_find[1] = inc - mine;
    }
  } else {                                                    // again, a CTA's width of heads at a time
    int64_t carry = 0;
    for (int64_t b0 = 0; b0 < p.B && carry <= u0; b0 += kD4Threads) {
      const int64_t b = b0 + tid;
      const int64_t n = b < p.B ? weight_of(count_of(b), p.cap) : 0;
      const int64_t all = cta_scan(n, inc, s_red);
      const int64_t start = carry + inc - n;
      if (u0 >= start && u0 < start + n) {
        s_find[0] = b;
        s_find[1] = start;
      }
      carry += all;
    }
  }
  __syncthreads();
  int64_t start = s_find[1] + kD4HeadCost;                    // where the blocks of the part's head start
  auto part_of = [&](int64_t b, int64_t at) -> Part4 {
    const int count = count_of(b);
    const int64_t n = blocks_of(count, p.cap);
    return Part4{static_cast<int>(b), count, static_cast<int>(u0 > at ? u0 - at : 0),
                 static_cast<int>(u1 - at < n ? u1 - at : n)};
  };
  Part4 part = part_of(s_find[0], start);
  if (part.a1 <= 0) {                                         // a share of a head's beginning alone
    if (tid == 0) p.cont[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }

  Ring4<D, TEST> ring{smem + warp * (kD4Stages * S::STAGE), full + warp * kD4Stages, 0u, 0, 0, 0, false};
  float* s_o = reinterpret_cast<float*>(smem + S::O_OFF);
  int4 cont = make_int4(-1, 0, 0, 0);

  bool failed = false;
  for (;;) {
    Query4<D> query;                                          // on its way before the first stages are issued
    query.load(p, part.b);
    const int64_t n_blk = blocks_of(part.count, p.cap);
    if (tid == 0) {
      s_then.b = -1;
      const int64_t next = start + n_blk + kD4HeadCost;
      if (next < u1) {                                        // there is a next head: u1 is at most the sum of weights
        int64_t nb = part.b;
        do ++nb; while (blocks_of(count_of(nb), p.cap) == 0);
        s_then = part_of(nb, next);
      }
    }
    __syncthreads();                                          // also: the warps' states of the last part are read
    if (!failed) {
      const bool ok = read_part<D, TEST>(p, query, part, &s_then, ring, &s_abort, s_o, s_m, s_l, 0);
      failed = __syncthreads_or(!ok);                         // uniform: the share's heads from this one on come out as
      if (failed && ok) ring.drain(lane, 0);                  // NaN, also those that other CTAs read a part of
    }
    const bool whole = part.a0 == 0 && part.a1 == n_blk, past = part.a1 < n_blk;
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (past ? 1 : 0);
    for (int e4 = tid; e4 < G * D / 4; e4 += kD4Threads) {
      const int g = 4 * e4 / D;
      float M, Ls;
      const float4 acc = join_warps<D>(e4, s_o, s_m, s_l, M, Ls);
      if (failed) Ls = NAN;
      if (whole) {
        reinterpret_cast<float4*>(p.out + static_cast<int64_t>(part.b) * G * D)[e4] =
            quotient(acc, Ls);
        if ((4 * e4) % D == 0 && p.lse2 != nullptr) p.lse2[static_cast<int64_t>(part.b) * G + g] = M + log2f(Ls);
      } else {
        reinterpret_cast<float4*>(p.part_o + slot * G * D)[e4] = acc;
        if ((4 * e4) % D == 0) p.part_ml[slot * 8 + g] = make_float2(M, Ls);
      }
    }
    if (part.a0 == 0 && past)                                 // this CTA begins the head, others go on with it
      cont = make_int4(part.b, static_cast<int>((start + n_blk - 1) / quota), 0, 0);
    if (s_then.b < 0) break;
    start += n_blk + kD4HeadCost;
    part = s_then;
    __syncthreads();                                          // s_then is read
  }
  if (tid == 0) p.cont[blockIdx.x] = cont;
}

// Write to the same shared variable of CTA `rank` of the cluster; its barrier,
// likewise, counts the bytes as they land.
__device__ __forceinline__ uint32_t mapa(const void* p, int rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  return a;
}
__device__ __forceinline__ void send(uint32_t at, const float4& v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(at),
               "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
               : "memory");
}
__device__ __forceinline__ void send(uint32_t at, const float2& v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(at),
               "f"(v.x), "f"(v.y), "r"(bar)
               : "memory");
}

// Few rows a head: latency counts, and the shares of the other kernel (a scan
// of all counts, parts of two heads in a CTA, a second launch) cost more than
// equal work gains.  Here the CTAs of a cluster read a head, its 32-row stages
// in turn over all their warps.  Every CTA sends its state to the cluster's CTAs, each of
// which joins a part of the dims: four dims in the lanes of a warp, a lane per
// CTA that sent them.  8 heads of 2,457 rows (d = 128, G = 4): 6.6 us in a
// chain of calls, of which the first 1.6 pass before the first rows are there
// (count and page, then rows) and 1.2 in the join; a microsecond more when
// every CTA fetched the others' states, two round trips and a barrier more.
template <int D, bool TEST>
__global__ void __launch_bounds__(kD4Threads, 2) decode_int4_cluster_kernel(Dec4Args p) {
  using S = D4<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kD4Warps * kD4Stages];
  __shared__ int s_abort;
  __shared__ float s_m[kD4Warps][8], s_l[kD4Warps][8];
  __shared__ Part4 s_then;
  __shared__ float4 s_co[2 * D];                              // [C][8 D / 4 / C] outputs of the cluster's CTAs
  __shared__ float2 s_cml[2 * D];                             // and (reference, sum) of their queries
  __shared__ uint64_t s_all;                                  // counts both as they land
  const cg::cluster_group cluster = cg::this_cluster();
  const int C = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x, warp = tid >> 5, G = p.G;
  const int64_t b = blockIdx.x / C;
  const int n4 = G * D / 4;
  let_next_start();
  if (tid < kD4Warps * kD4Stages) mbar_init(&full[tid], 1);
  if (tid == 0) {
    s_abort = 0;
    mbar_init(&s_all, 1);
    mbar_arrive_expect_tx(&s_all, static_cast<uint32_t>(n4 * (sizeof(float4) + sizeof(float2))));
  }
  fence_mbar_init();
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // this CTA may be sent to
  after_prior();
  // stages in turn over the cluster's CTAs and their warps, so that where a warp's stages are does not depend on the
  // head's rows: their pages are looked up beside the count
  const int lane = tid & 31, blk = 2 * (rank + C * (warp + kD4Warps * lane)), tab = static_cast<int>(p.cap / kC4Rows);
  const int2 early = blk < tab ? Ring4<D, TEST>::ids(p, static_cast<int>(b), blk, tab) : make_int2(0, 0);
  const int count = load_int(p.counts + b);                   // the same in all CTAs of the cluster
  Query4<D> query;
  query.load(p, b);
  if (count <= 0 || count > p.cap) {
    if (rank == 0 && count == 0) {
      for (int e = tid; e < G * D; e += kD4Threads) p.out[b * G * D + e] = 0.0f;
      if (p.lse2 != nullptr && tid < G) p.lse2[b * G + tid] = -INFINITY;
    } else if (rank == 0 && tid == 0) {
      report(p.status, KVZ_ERR_INVALID_ARG);
    }
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    return;
  }
  const Part4 part{static_cast<int>(b), count, 2 * rank, (count + kC4Rows - 1) / kC4Rows};
  const int spread = 31 - __clz(C);                           // (C is a power of two)
  float* s_o = reinterpret_cast<float*>(smem + S::O_OFF);
  Ring4<D, TEST> ring{smem + warp * (kD4Stages * S::STAGE), full + warp * kD4Stages, 0u, 0, 0, 0, true};
  if (blk < part.a1) ring.place(p, make_int2(early.x, blk + 1 < part.a1 ? early.y : early.x), blk);
  if (tid == 0) s_then.b = -1;
  __syncthreads();                                            // the barriers are initialised
  const bool ok = read_part<D, TEST>(p, query, part, &s_then, ring, &s_abort, s_o, s_m, s_l, spread);
  const bool failed = __syncthreads_or(!ok);
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (tid < n4) {                                             // n4 <= 2 D <= kD4Threads
    float M, Ls;
    const float4 acc = join_warps<D>(tid, s_o, s_m, s_l, M, Ls);
    if (failed) Ls = NAN;                                     // a part that was not read spoils its head, not others
    const int to = tid & (C - 1), at = rank * (2 * D / C) + tid / C;
    const uint32_t bar = mapa(&s_all, to);
    send(mapa(s_co + at, to), acc, bar);
    send(mapa(s_cml + at, to), make_float2(M, Ls), bar);
  }
  // (past the limit of the others' own waits: each sends in any case)
  if (!mbar_wait_for(&s_all, 0, 2 * kWaitLimitNs)) report(p.status, KVZ_ERR_TIMEOUT);
  const int j = tid & (C - 1), e4 = rank + (tid & ~(C - 1));  // C lanes of a warp join output e4
  const float2 ml = e4 < n4 ? s_cml[j * (2 * D / C) + tid / C] : make_float2(-INFINITY, 0.0f);
  float4 acc = e4 < n4 ? s_co[j * (2 * D / C) + tid / C] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float M = ml.x;
  for (int o = 1; o < C; o <<= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, o));
  const float w = ml.x == -INFINITY && ml.y == 0.0f ? 0.0f : exp2f(ml.x - M);   // 0: a CTA without rows
  float Ls = ml.y * w;
  acc = make_float4(acc.x * w, acc.y * w, acc.z * w, acc.w * w);
  for (int o = 1; o < C; o <<= 1) {
    Ls += __shfl_xor_sync(kFullMask, Ls, o);
    acc.x += __shfl_xor_sync(kFullMask, acc.x, o), acc.y += __shfl_xor_sync(kFullMask, acc.y, o);
    acc.z += __shfl_xor_sync(kFullMask, acc.z, o), acc.w += __shfl_xor_sync(kFullMask, acc.w, o);
  }
  if (e4 < n4 && j == 0) {
    const float inv = 1.0f / (Ls * kD4Out);
    reinterpret_cast<float4*>(p.out + b * G * D)[e4] = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if ((4 * e4) % D == 0 && p.lse2 != nullptr) p.lse2[b * G + 4 * e4 / D] = M + log2f(Ls);
  }
}

// The heads that CTA blockIdx.x began and others went on with: their partials
// (reference m, sum l, output o) join as M = max m, sum l 2^(m - M), sum o
// 2^(m - M), in the CTAs' order.  Launched while the shares still run; what
// they wrote is read after the wait, the first outputs before their weights
// are known.
template <int D>
__global__ void __launch_bounds__(kD4Threads) merge_int4_kernel(Dec4Args p) {
  constexpr int C = D / 4, RS = kD4Threads / C;               // float4 columns, partials read side by side
  constexpr int AHEAD = 4;
  __shared__ float s_w[kD4Workers];
  __shared__ float s_red[kD4Warps], s_red2[kD4Warps];
  __shared__ float4 s_acc[kD4Threads];
  const int first = blockIdx.x, g = blockIdx.y, tid = threadIdx.x, G = p.G;
  let_next_start();
  after_prior();
  const int4 cont = p.cont[first];
  if (cont.x < 0) return;
  const int np = cont.y - first + 1;                          // CTAs first .. last: all but the last run past their range
  auto slot = [&](int i) -> int64_t { return 2 * static_cast<int64_t>(first + i) + (i + 1 < np ? 1 : 0); };
  const int col = tid % C, lanep = tid / C;
  auto output = [&](int i) -> float4 {
    return i < np ? reinterpret_cast<const float4*>(p.part_o + (slot(i) * G + g) * D)[col]
                  : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  };
  float2 ml[2];                                               // np <= kD4Workers <= 2 per thread
  static_assert(kD4Workers <= 2 * kD4Threads, "");
#pragma unroll
  for (int k = 0; k < 2; ++k)
    ml[k] = tid + k * kD4Threads < np ? p.part_ml[slot(tid + k * kD4Threads) * 8 + g] : make_float2(-INFINITY, 0.0f);
  float4 v[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) v[k] = output(lanep + k * RS);
  float M = fmaxf(ml[0].x, ml[1].x);
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFullMask, M, o));
  if ((tid & 31) == 0) s_red[tid >> 5] = M;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kD4Warps; ++i) M = fmaxf(M, s_red[i]);
  float Ls = 0.0f;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = tid + k * kD4Threads;
    if (i < np) {
      const float w = exp2f(ml[k].x - M);
      s_w[i] = w;
      Ls = fmaf(ml[k].y, w, Ls);
    }
  }
  for (int o = 16; o > 0; o >>= 1) Ls += __shfl_xor_sync(kFullMask, Ls, o);
  if ((tid & 31) == 0) s_red2[tid >> 5] = Ls;
  __syncthreads();
  Ls = 0.0f;
#pragma unroll
  for (int i = 0; i < kD4Warps; ++i) Ls += s_red2[i];
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i0 = lanep; i0 < np; i0 += AHEAD * RS) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int i = i0 + k * RS;
      if (i < np) {
        const float w = s_w[i];
        acc.x = fmaf(v[k].x, w, acc.x), acc.y = fmaf(v[k].y, w, acc.y);
        acc.z = fmaf(v[k].z, w, acc.z), acc.w = fmaf(v[k].w, w, acc.w);
      }
      v[k] = output(i + AHEAD * RS);
    }
  }
  s_acc[tid] = acc;
  __syncthreads();
  if (tid < C) {
    for (int i = 1; i < RS; ++i) {
      const float4 x = s_acc[i * C + tid];
      acc.x += x.x, acc.y += x.y, acc.z += x.z, acc.w += x.w;
    }
    const int64_t at = static_cast<int64_t>(cont.x) * G + g;
    reinterpret_cast<float4*>(p.out + at * D)[tid] = quotient(acc, Ls);
    if (tid == 0 && p.lse2 != nullptr) p.lse2[at] = M + log2f(Ls);
  }
}

// The widest cluster of at most `want` CTAs (a power of two) that the device
// has room for: a process may be limited to a part of its SMs, where 16 CTAs
// of their own find no place.  Asked once per device, size and shared memory.
template <auto Kernel>
int widest_cluster(int want, int smem, bool alone) {
  static std::atomic<uint8_t> known[64][2][5];                // [device][alone][log2 want]
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return want;
  std::atomic<uint8_t>& answer = known[dev][alone ? 1 : 0][31 - __builtin_clz(static_cast<unsigned>(want))];
  int c = answer.load(std::memory_order_relaxed);
  if (c > 0) return c;
  for (c = want; c > 1; c /= 2) {
    if (c > 8 && wide_clusters_once<Kernel>() != cudaSuccess) continue;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = static_cast<unsigned>(c);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(c));
    cfg.blockDim = dim3(kD4Threads);
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, Kernel, &cfg) == cudaSuccess && n > 0) break;
  }
  cudaGetLastError();                                         // (a size that was refused is not this call's error)
  answer.store(static_cast<uint8_t>(c), std::memory_order_relaxed);
  return c;
}

template <int D, bool TEST>
cudaError_t launch_decode4(const Dec4Args& a, cudaStream_t stream) {
  const Decode4Form form = decode4_form(a.B, a.cap);
  if (form.cluster > 0) {
    constexpr int kAlone = 115 * 1024;                        // of an SM's 228 KB: one CTA
    static_assert(D4<D>::SMEM <= kAlone, "");
    const cudaError_t e = smem_limit_once<decode_int4_cluster_kernel<D, TEST>>(kAlone);
    if (e != cudaSuccess) return e;
    const int smem = form.alone ? kAlone : D4<D>::SMEM;
    const int c = widest_cluster<decode_int4_cluster_kernel<D, TEST>>(
        TEST && a.max_cluster < form.cluster ? a.max_cluster : form.cluster, smem, form.alone);
    return launch_after(decode_int4_cluster_kernel<D, TEST>, dim3(static_cast<unsigned>(a.B * c)), dim3(kD4Threads), smem,
                        stream, c, a);
  }
  cudaError_t e = smem_limit_once<decode_int4_kernel<D, TEST>>(D4<D>::SMEM);
  if (e != cudaSuccess) return e;
  e = launch_after(decode_int4_kernel<D, TEST>, dim3(kD4Workers), dim3(kD4Threads), D4<D>::SMEM, stream, 0, a);
  if (e != cudaSuccess) return e;
  return launch_after(merge_int4_kernel<D>, dim3(kD4Workers, static_cast<unsigned>(a.G)), dim3(kD4Threads), 0, stream, 0,
                      a);
}

}  // namespace

cudaError_t launch_decode_int4(int d, const Dec4Args& a, cudaStream_t stream) {
  if (a.wait_ns > 0) return d == 128 ? launch_decode4<128, true>(a, stream) : launch_decode4<64, true>(a, stream);
  return d == 128 ? launch_decode4<128, false>(a, stream) : launch_decode4<64, false>(a, stream);
}

}  // namespace kvz
