// Writing and reading the paged 4-bit cache (layout and quantisation in
// kvz_cache4.cuh): kept rows into it (compaction), new rows behind them with
// the position rotation on the way (append), and rows back to bf16 (expand).
//
// All three move rows through registers.  HBM-bound at length: 4 d bytes of
// bf16 and 9/8 d bytes of the cache per row; a layer's few thousand rows are a
// chain of dependent loads (head, page, index, row) behind a launch.  At d =
// 128, in chains of calls: 311,051 of 32 x 32,768 rows compacted in 39.2 us
// (5.2 TB/s) and expanded in 37.0 us (5.5 TB/s); 8 heads of 2,457 rows 5.8 and
// 4.8 us; 32 ragged prompts, 8,716 tokens with 4 query heads each, appended in
// 9.1 us (2.6 TB/s); one token for 128 heads in 2.2 us.
#include <cuda_runtime.h>

#include <cstdint>

#include "kvz.h"
#include "kvz_cache4.cuh"
#include "kvz_internal.h"
#include "kvz_launch.cuh"
#include "kvz_rotary.cuh"
#include "kvz_sm100.cuh"

namespace kvz {

namespace {

// Small CTAs, since a warp's chain of loads is its time: 32 x 515 ragged
// tokens appended (and read back) took 15.8, 14.2 and 16.3 us with 256, 128
// and 64 threads; 32 heads of about 9,830 of 32,768 rows compacted (and read
// back) 75.1, 74.5 and 74.3.
constexpr int kC4Threads = 64, kAppendThreads = 128;
constexpr int kQHeads = 2;                                    // query heads a thread turns by one set of angles
// Blocks up to which the rows read back go by two warps a block, one for K and
// one for V: where a warp has one block, its instructions are its time (8 heads
// of 2,457 rows 4.7 us against 5.6); where it has several, looking them up
// twice costs more (64 uneven heads, 567,000 rows, 35.8 against 33.8).
// Compaction, whose warps look up each row's index too, gains nothing (6.0
// against 5.4).
constexpr int64_t kExpandSplit = 2368;
constexpr int kCompactCtas = 8;                               // CTAs per SM of the largest grids: resident at once, and
constexpr int kExpandCtas = 48;                               // several waves (8 to 24 and 12 to 96 were measured)

template <int N>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x, w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  }
}

// The blocks of all heads as one index space: head b's start at
// base_of(offsets[b], b) = offsets[b] / 16 + SPARE * b and the first one's at
// its own (the offsets may start anywhere: one layer's heads among a stack's,
// rows kept in front), so heads of any lengths share the grid evenly: a warp
// (SPLIT: two) takes an equal run of blocks, finds the first one's head by
// search and walks on from there.  A head of n rows has at most
// n / 16 + 1 blocks from its row 0 on (SPARE = 1), and a run of n rows that
// begins inside one touches at most n / 16 + 2 (SPARE = 2).  Offsets may leave
// a head more room than its rows, any amount of it: a warp that comes to the
// end of a head's rows goes on at the next head's first unit in one step.
template <int SPARE, bool SPLIT>
struct BlockWalk {
  int64_t u, end;                                             // the next unit to look up, the end of this warp's run
  int64_t b, base, next, o;                                   // head, its first unit, the next head's, offsets[b]
  int32_t n, f;                                               // rows [f, n) of the head count (none for a bad head)

  static __device__ __forceinline__ int64_t base_of(int64_t o, int64_t b) { return (o >> 4) + SPARE * b; }
  __device__ __forceinline__ void run(const int64_t* offsets, int64_t B) {
    const int64_t at0 = base_of(offsets[0], 0), at1 = base_of(offsets[B], B);
    const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kC4Threads + threadIdx.x) >> (SPLIT ? 6 : 5);
    const int64_t n_warps = static_cast<int64_t>(gridDim.x) * (kC4Threads / (SPLIT ? 64 : 32));
    const int64_t each = (at1 - at0 + n_warps - 1) / n_warps;
    u = at0 + warp * each;
    end = u + each < at1 ? u + each : at1;
  }
  // the unit after u where u is past its head's rows
  __device__ __forceinline__ int64_t skip(int64_t u, int64_t B) const {
    return b + 1 < B ? (next > u ? next : u + 1) : end;
  }
  __device__ __forceinline__ int64_t head(const int64_t* offsets, int64_t B) const {
    int64_t lo = 0;                                           // largest b whose base is at most u: 32 steps of the
    for (int64_t n = B; n > 1;) {                             // range at a time (lane 0 stands for "at least lo")
      const int lane = threadIdx.x & 31;
      const int64_t step = (n + 31) >> 5, at = lane * step;
      const unsigned below = __ballot_sync(kFullMask, lane == 0 || (at < n && base_of(offsets[lo + at], lo + at) <= u));
      const int64_t pass = (31 - __clz(below)) * step;
      lo += pass;
      n = n - pass < step ? n - pass : step;
    }
    return lo;
  }
};

// Both kernels below take a block of 16 rows per warp: lane (r, c) = (lane / 4,
// lane % 4) holds dims 64g + 16c .. 64g + 16c + 15 of rows r and r + 8, which
// are its words of the K layout.  All index arithmetic is per block; the
// block's codes move as one 16-byte access per lane and tensor half.

// A row's V halves meet their pair's other row's here: lanes 4 apart hold rows
// r and r ^ 1.  vv[g][j]: the lane's own units of r' = 2c + j (two halves of a
// word); after the exchange an even row's lane holds both rows' words of r' =
// 2c, an odd row's those of 2c + 1: words [g][w].
template <int NG>
__device__ __forceinline__ void pair_up(const uint32_t (&vv)[NG][2], bool odd, uint32_t (&out)[2 * NG]) {
#pragma unroll
  for (int g = 0; g < NG; ++g) {
    const uint32_t mine = odd ? vv[g][1] : vv[g][0];
    const uint32_t got = __shfl_xor_sync(kFullMask, odd ? vv[g][0] : vv[g][1], 4);
    const uint32_t even_row = odd ? got : mine, odd_row = odd ? mine : got;
    out[2 * g] = __byte_perm(even_row, odd_row, 0x5410);
    out[2 * g + 1] = __byte_perm(even_row, odd_row, 0x7632);
  }
}
template <int NG>
__device__ __forceinline__ void store_words(uint8_t* p, const uint32_t (&w)[2 * NG]) {
  if constexpr (NG == 2) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}

template <int D>
__global__ void __launch_bounds__(kC4Threads, 512 / kC4Threads)
    compact_int4_kernel(const uint16_t* K, const uint16_t* V, int64_t B, int64_t n_c,
                        const int32_t* idx, const int32_t* counts,
                        const int64_t* offsets, Pages4 pg, int64_t cap, int32_t* status) {
  using L = C4<D>;
  constexpr int NG = L::NG;
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  let_next_start();
  after_prior(K, V, idx, counts, offsets, pg.cache, pg.pages);
  BlockWalk<1, false> h;
  h.run(offsets, B);
  if (h.u >= h.end) return;                                   // warp-uniform, as is all that follows per block
  int64_t o1 = 0;
  bool fresh = false;
  auto enter = [&](int64_t b) {
    h.b = b;
    h.o = offsets[b];
    o1 = offsets[b + 1];
    h.base = h.base_of(h.o, b);
    h.next = h.base_of(o1, b + 1);
    h.n = counts[b];
    fresh = true;
  };
  auto settle = [&]() {                                       // the head's count, once it is there
    if (fresh && (h.n < 0 || h.o < 0 || h.n > o1 - h.o || h.n > cap)) {
      if (lane == 0) report(status, KVZ_ERR_INVALID_ARG);
      h.n = 0;
    }
    fresh = false;
  };
  enter(h.head(offsets, B));
  // where a block goes and its rows come from, looked up a step before they move
  uint8_t* blk = nullptr;
  int rows = 0;                                               // rows of it that count
  int64_t src[2];                                             // element of row r + 8h's first dims here; < 0: zeros
  auto look_up = [&]() {
    blk = nullptr;
    const int64_t u = h.u;
    if (u >= h.end) return;
    while (u >= h.next && h.b + 1 < B) {
      settle();
      enter(h.b + 1);
    }
    // the page is on its way with the count and the indexes, and looked at after them (5% of the time of a large
    // compaction; expanding, whose chain is shorter, lost 9% to the registers)
    const int64_t p0 = (u - h.base) * kC4Rows;
    const uint32_t q = static_cast<uint32_t>(u - h.base);
    const int32_t id = p0 >= 0 && p0 < cap ? page_id(pg, h.b, q) : -1;
    settle();
    if (p0 < 0 || p0 >= h.n) {                                // (below 0: offsets that do not ascend)
      h.u = h.skip(u, B);
      return;
    }
    h.u = u + 1;
    rows = static_cast<int>(h.n - p0 < kC4Rows ? h.n - p0 : kC4Rows);
    int32_t from[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) from[k] = r + 8 * k < rows ? idx[h.o + p0 + r + 8 * k] : -1;
    blk = block_of<D>(pg, id, q, status);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      src[k] = -1;
      if (r + 8 * k >= rows) continue;
      const int64_t j = from[k];
      if (j >= 0 && j < n_c) src[k] = (h.b * n_c + j) * D + 16 * c;
      else if (c == 0) report(status, KVZ_ERR_INVALID_ARG);   // idx out of [0, n_c): a row of zeros
    }
  };
  look_up();
  while (blk != nullptr || h.u < h.end) {
    uint8_t* const to = blk;
    const int live = rows;
    uint4 x[2][2][NG][2];                                     // [K, V][row r + 8k][g][half]
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int g = 0; g < NG; ++g)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const bool on = to != nullptr && r + 8 * k < live && src[k] >= 0;
          x[0][k][g][j] = on ? *reinterpret_cast<const uint4*>(K + src[k] + 64 * g + 8 * j) : make_uint4(0, 0, 0, 0);
          x[1][k][g][j] = on ? *reinterpret_cast<const uint4*>(V + src[k] + 64 * g + 8 * j) : make_uint4(0, 0, 0, 0);
        }
    look_up();
    if (to == nullptr) continue;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int row = r + 8 * k;
        const bool on = row < live;
        uint32_t kw[2 * NG], vv[NG][2], sm = 0u;
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint4 (&v)[2] = x[t][k][g];
          const Scale4 q = group_scale<4>(
              min_nan2(min_nan2(min_nan2(v[0].x, v[0].y), min_nan2(v[0].z, v[0].w)),
                       min_nan2(min_nan2(v[1].x, v[1].y), min_nan2(v[1].z, v[1].w))),
              max_nan2(max_nan2(max_nan2(v[0].x, v[0].y), max_nan2(v[0].z, v[0].w)),
                       max_nan2(max_nan2(v[1].x, v[1].y), max_nan2(v[1].z, v[1].w))));
          if (c == g) sm = q.word;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t code[8];
            code2(v[j].x, q, code[0], code[1]);
            code2(v[j].y, q, code[2], code[3]);
            code2(v[j].z, q, code[4], code[5]);
            code2(v[j].w, q, code[6], code[7]);
            if (t == 0) kw[2 * g + j] = k_word(code, q.fine);
            else vv[g][j] = v_units(code, q.fine);
          }
        }
        if (on && c < NG)
          *reinterpret_cast<uint32_t*>(to + (t == 0 ? L::KS_OFF : L::VS_OFF) + (row * NG + c) * 4) = sm;
        if (t == 0) {
          if (on) store_words<NG>(to + row * (D / 2) + c * (8 * NG), kw);
          continue;
        }
        const bool odd = (row & 1) != 0;
        uint8_t* const pair = to + L::V_OFF + (row >> 1) * D;
        uint32_t both[2 * NG];
        pair_up<NG>(vv, odd, both);
        if ((row | 1) < live) {
          store_words<NG>(pair + (2 * c + (odd ? 1 : 0)) * (8 * NG), both);
        } else if (on) {                                      // the last row of an odd count: its halves alone
#pragma unroll
          for (int g = 0; g < NG; ++g)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              uint16_t* const at = reinterpret_cast<uint16_t*>(pair + (2 * c + j) * (8 * NG) + g * 8);
              at[0] = static_cast<uint16_t>(vv[g][j]);
              at[2] = static_cast<uint16_t>(vv[g][j] >> 16);
            }
        }
      }
  }
}

// Rows first[b] .. counts[b] - 1 as bf16 rows offsets[b], offsets[b] + 1, ...
// A value is one fused bf16 multiply-add, s * code + m rounded once.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(kC4Threads)
    expand_int4_kernel(Pages4 pg, const int32_t* counts, const int32_t* first,
                       const int64_t* offsets, int64_t B, int64_t cap, uint16_t* K_out,
                       uint16_t* V_out, int64_t n_rows, int32_t* status) {
  using L = C4<D>;
  constexpr int NG = L::NG;
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  let_next_start();
  after_prior(pg.cache, pg.pages, counts, first, offsets, K_out, V_out);
  const bool do_k = !SPLIT || (threadIdx.x & 32) == 0, do_v = !SPLIT || !do_k;   // warp-uniform
  BlockWalk<2, SPLIT> h;
  h.run(offsets, B);
  if (h.u >= h.end) return;
  auto enter = [&](int64_t b) {
    h.b = b;
    h.o = offsets[b];
    const int64_t o1 = offsets[b + 1];
    h.base = h.base_of(h.o, b);
    h.next = h.base_of(o1, b + 1);
    h.n = counts[b];
    h.f = first == nullptr ? 0 : first[b];
    if (h.f < 0 || h.n < h.f || h.n > cap || h.n - h.f > o1 - h.o || h.o < 0 || h.o + (h.n - h.f) > n_rows) {
      if (lane == 0) report(status, KVZ_ERR_INVALID_ARG);
      h.n = h.f = 0;
    }
  };
  enter(h.head(offsets, B));
  const uint8_t* blk = nullptr;
  int from = 0, to = 0;                                       // rows of the block that count
  int64_t dst = 0;                                            // output row of the block's row 0
  auto look_up = [&]() {
    blk = nullptr;
    const int64_t u = h.u;
    if (u >= h.end) return;
    while (u >= h.next && h.b + 1 < B) enter(h.b + 1);
    const int64_t q = (h.f >> 4) + u - h.base, p0 = q * kC4Rows;
    if (p0 < 0 || p0 >= h.n) {                                // (below 0: offsets that do not ascend)
      h.u = h.skip(u, B);
      return;
    }
    h.u = u + 1;
    blk = block_at<D>(pg, h.b, static_cast<uint32_t>(q), status);
    from = static_cast<int>(h.f > p0 ? h.f - p0 : 0);
    to = static_cast<int>(h.n - p0 < kC4Rows ? h.n - p0 : kC4Rows);
    dst = h.o + p0 - h.f;
  };
  // 32 bytes of a row, as one store where the outputs allow it
  const bool wide = ((reinterpret_cast<uintptr_t>(K_out) | reinterpret_cast<uintptr_t>(V_out)) & 31u) == 0;
  auto put32 = [&](uint16_t* at, const uint32_t (&w)[8]) {
    if (wide) {
      asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                   "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                   : "memory");
    } else {
      *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(at + 8) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  };
  look_up();
  while (blk != nullptr || h.u < h.end) {
    const uint8_t* const p = blk;
    const int lo = from, hi = to;
    const int64_t out = dst;
    uint32_t kw[2][2 * NG], ks[2][NG], vw[2][2 * NG], vs[2][2 * NG];
    if (p != nullptr) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (do_k) {
          load_words<2 * NG>(p + (r + 8 * k) * (D / 2) + c * (8 * NG), kw[k]);
          load_words<NG>(p + L::KS_OFF + (r + 8 * k) * (4 * NG), ks[k]);
        }
        if (!do_v) continue;
        // V: lane (r, c) takes r' = r of the pairs c and c + 4, rows 2c + 8k and 2c + 8k + 1
        load_words<2 * NG>(p + L::V_OFF + (c + 4 * k) * D + r * (8 * NG), vw[k]);
        load_words<2 * NG>(p + L::VS_OFF + (2 * c + 8 * k) * (4 * NG), vs[k]);
      }
    }
    look_up();
    if (p == nullptr) continue;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int row = r + 8 * k;
      if (do_k && row >= lo && row < hi) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const uint32_t s2 = __byte_perm(ks[k][g], 0u, 0x1010), m2 = __byte_perm(ks[k][g], 0u, 0x3232);
          uint32_t y[8];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const uint32_t w = kw[k][2 * g + u];
            y[4 * u] = fma_bf2(s2, code_bf2(w), m2);
            y[4 * u + 1] = fma_bf2(s2, code_bf2(w >> 4), m2);
            y[4 * u + 2] = fma_bf2(s2, code_bf2(w >> 8), m2);
            y[4 * u + 3] = fma_bf2(s2, code_bf2(__funnelshift_r(w, w, 12)), m2);
          }
          put32(K_out + (out + row) * D + 64 * g + 16 * c, y);
        }
      }
      if (!do_v) continue;
      const int even = 2 * c + 8 * k;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        // (even row, odd row) in the halves of every word
        const uint32_t s2 = __byte_perm(vs[k][g], vs[k][NG + g], 0x5410);
        const uint32_t m2 = __byte_perm(vs[k][g], vs[k][NG + g], 0x7632);
        uint32_t z[8];
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          const uint32_t v = vw[k][2 * g + w];
          z[4 * w] = fma_bf2(s2, code_bf2(v << 3), m2);
          z[4 * w + 1] = fma_bf2(s2, code_bf2(v >> 1), m2);
          z[4 * w + 2] = fma_bf2(s2, code_bf2(v >> 5), m2);
          z[4 * w + 3] = fma_bf2(s2, code_bf2(v >> 9), m2);
        }
        uint16_t* const at = V_out + (out + even) * D + 64 * g + 8 * r;
        if (even >= lo && even < hi)
          *reinterpret_cast<uint4*>(at) = make_uint4(__byte_perm(z[0], z[1], 0x5410), __byte_perm(z[2], z[3], 0x5410),
                                                     __byte_perm(z[4], z[5], 0x5410), __byte_perm(z[6], z[7], 0x5410));
        if (even + 1 >= lo && even + 1 < hi)
          *reinterpret_cast<uint4*>(at + D) =
              make_uint4(__byte_perm(z[0], z[1], 0x7632), __byte_perm(z[2], z[3], 0x7632),
                         __byte_perm(z[4], z[5], 0x7632), __byte_perm(z[6], z[7], 0x7632));
      }
    }
  }
}

// Rotate the row whose dims 8l .. 8l + 7 this lane holds (all lanes of the
// warp take part; `on` rows have a valid position).
template <int D>
__device__ __forceinline__ void turn_row(uint4& x, int lane, int l, const RotArgs& rot, int64_t p, bool on) {
  if (rot.interleaved) {
    if (on && 8 * l < rot.rot) {
      const float* t = rot.table + p * rot.rot + 4 * l;
      const float4 c = *reinterpret_cast<const float4*>(t);
      const float4 s = *reinterpret_cast<const float4*>(t + rot.rot / 2);
      const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
      turn_neighbours4(x, cc, ss);
    }
    return;
  }
  const int step = rot.rot / 16;                              // lanes from a pair's first half to its second
  const bool lo = l < step, hi = l >= step && l < 2 * step;
  const int from = lo ? lane + step : (hi ? lane - step : lane);
  uint4 y;
  y.x = __shfl_sync(kFullMask, x.x, from);
  y.y = __shfl_sync(kFullMask, x.y, from);
  y.z = __shfl_sync(kFullMask, x.z, from);
  y.w = __shfl_sync(kFullMask, x.w, from);
  if (on && (lo || hi)) {
    float c[8], s[8];
    load_angles(rot.table + p * rot.rot, rot.rot / 2, 8 * (lo ? l : l - step), 0, c, s);
    if (lo) {
      turn_halves(x, y, c, s);
    } else {
      turn_halves(y, x, c, s);
    }
  }
}

// Append.  Warps take, in this order: one head each for the new counts (the
// longest chain of loads), K row pairs, V row pairs, query rows.  Pair j of
// head b covers the slots 2 (counts[b] / 2 + j) and the next, of which those
// in [counts[b], counts[b] + n_new[b]) are written; a slot's other half and
// all later rows stay as they were.  What a row needs is a chain of loads (its
// head's count, then its page, position and values, then its angles), so a
// single token is latency, and K, V and queries go to warps of their own; two
// and four chains side by side in a warp were no faster on long prompts either.
template <int D>
__global__ void __launch_bounds__(kAppendThreads) append_int4_kernel(Append4Args a, uint32_t n_warps, uint32_t n_pairs,
                                                                 uint32_t kv_warps, uint32_t q_warps, int64_t cap) {
  using L = C4<D>;
  constexpr int PW = 16 / L::LPR;
  const int lane = threadIdx.x & 31, l = lane % L::LPR;
  uint32_t w = blockIdx.x * (kAppendThreads / 32) + (threadIdx.x >> 5);   // below 2^30; its threads may pass 2^32
  let_next_start();
  after_prior(a.k, a.v, a.q, a.rot.pos, a.rot.table, a.pg.cache, a.pg.pages, a.counts, a.n_new);
  const bool turning = a.rot.pos != nullptr;

  if (w < n_warps) {
    // the new count, if every page and position of the head's new rows is valid
    const int64_t b = w, base = a.counts[b], len = a.n_new == nullptr ? a.T : a.n_new[b];
    bool ok = base >= 0 && len >= 0 && len <= a.T && base + len <= cap;
    if (ok && len > 0) {
      const int64_t p0 = page_of(a.pg, static_cast<uint32_t>(base >> 4));
      const int64_t p1 = page_of(a.pg, static_cast<uint32_t>((base + len - 1) >> 4));
      int64_t worst = 0;                                      // the sign bit collects every bad id and position
#pragma unroll 4
      for (int64_t i = p0 + lane; i <= p1; i += 32) {
        const int64_t id = a.pg.pages[b * a.pg.max_pages + i];
        worst |= id | (a.pg.n_pages - 1 - id);
      }
      if (turning) {
#pragma unroll 8
        for (int64_t t = lane; t < len; t += 32) {
          const int64_t p = a.rot.pos[b * a.rot.pos_sb + t];
          worst |= p | (a.rot.n_pos - 1 - p);
        }
      }
      ok = worst >= 0;
    }
    ok = __all_sync(kFullMask, ok);
    if (lane == 0) a.counts_out[b] = static_cast<int32_t>(ok ? base + len : base);
    return;
  }
  w -= n_warps;
  if (w < 2 * kv_warps) {
    const bool is_k = w < kv_warps;
    if (!is_k) w -= kv_warps;
    const int e = (lane / L::LPR) & 1, sub = lane / (2 * L::LPR);
    const uint32_t f = w * PW + sub, b = f / n_pairs, j = f - b * n_pairs;
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    uint8_t* blk = nullptr;
    int row = e;
    int32_t p = 0;
    if (b < a.B) {
      const int32_t base = a.counts[b], len = a.n_new == nullptr ? static_cast<int32_t>(a.T) : a.n_new[b];
      const bool head_ok = base >= 0 && len >= 0 && len <= a.T && static_cast<int64_t>(base) + len <= cap;
      if (!head_ok && is_k && j == 0 && e == 0 && l == 0) report(a.status, KVZ_ERR_INVALID_ARG);
      const int32_t slot = head_ok ? 2 * ((base >> 1) + static_cast<int32_t>(j)) + e : 0, t = slot - base;
      if (head_ok && t >= 0 && t < len) {
        x = is_k ? *reinterpret_cast<const uint4*>(a.k + b * a.k_sb + t * a.k_st + 8 * l)
                 : *reinterpret_cast<const uint4*>(a.v + b * a.v_sb + t * a.v_st + 8 * l);
        if (turning) p = a.rot.pos[b * a.rot.pos_sb + t];
        blk = block_at<D>(a.pg, b, static_cast<uint32_t>(slot) >> 4, a.status);
        row = slot & 15;
      }
    }
    if (turning && (p < 0 || p >= a.rot.n_pos)) {
      report(a.status, KVZ_ERR_INVALID_ARG);
      blk = nullptr;
    }
    if (!__any_sync(kFullMask, blk != nullptr)) return;
    uint32_t code[8], sm;
    if (is_k) {                                               // warp-uniform
      if (turning) turn_row<D>(x, lane, l, a.rot, p, blk != nullptr);
      const bool fine = quantise8(x, code, sm);
      if (blk != nullptr) store_k<D>(blk, row, l, code, fine, sm);
    } else {
      const bool fine = quantise8(x, code, sm);
      store_v<D>(blk, row, l, code, fine, sm, blk != nullptr);
    }
    return;
  }
  w -= 2 * kv_warps;
  if (w < q_warps) {
    // a thread per 16 dims (whole pairs) of a token in kQHeads heads, its values on the way before its angles (all
    // heads in a thread: 15.9 us against 14.2 for 32 x 515 ragged tokens)
    constexpr uint32_t IT = D / 16;
    const uint32_t n_g = (static_cast<uint32_t>(a.G) + kQHeads - 1) / kQHeads, T = static_cast<uint32_t>(a.T);
    const uint32_t item = lane % IT, rest = w * (32 / IT) + lane / IT, bt = rest / n_g;
    const int g0 = static_cast<int>(rest - bt * n_g) * kQHeads;
    const uint32_t b = bt / T, t = bt - b * T;
    if (b >= a.B || (a.n_new != nullptr && static_cast<int32_t>(t) >= a.n_new[b])) return;
    const int rot = a.rot.rot, nrot = turning ? rot / 16 : 0;
    const bool turn = static_cast<int>(item) < nrot, il = a.rot.interleaved != 0;
    const int d0 = turn ? (il ? 16 * item : 8 * item) : (turning ? rot : 0) + 16 * (static_cast<int>(item) - nrot);
    const int d1 = turn && !il ? d0 + rot / 2 : d0 + 8;
    const uint16_t* const q = a.q + b * a.q_sb + t * a.q_st;
    uint4 v0[kQHeads], v1[kQHeads];
#pragma unroll
    for (int i = 0; i < kQHeads; ++i)
      if (g0 + i < a.G) {
        v0[i] = *reinterpret_cast<const uint4*>(q + (g0 + i) * a.q_sg + d0);
        v1[i] = *reinterpret_cast<const uint4*>(q + (g0 + i) * a.q_sg + d1);
      }
    float c[8], s[8];
    if (turning) {
      const int32_t p = a.rot.pos[b * a.rot.pos_sb + t];
      if (p < 0 || p >= a.rot.n_pos) return;                  // (reported with the head's keys)
      if (turn) load_angles(a.rot.table + static_cast<int64_t>(p) * rot, rot / 2, 8 * item, 0, c, s);
    }
#pragma unroll
    for (int i = 0; i < kQHeads; ++i)
      if (g0 + i < a.G) {
        if (turn) {
          if (il) turn_adjacent(v0[i], v1[i], c, s);
          else turn_halves(v0[i], v1[i], c, s);
        }
        uint16_t* const y = a.q_out + ((static_cast<int64_t>(b) * a.G + g0 + i) * T + t) * D;
        *reinterpret_cast<uint4*>(y + d0) = v0[i];
        *reinterpret_cast<uint4*>(y + d1) = v1[i];
      }
    return;
  }
}

// CTAs for `units` warp units: one each, up to per_sm on every SM, over which the units are then shared out evenly.
unsigned grid_for(int64_t units, int per_sm) {
  const int64_t n = (units + kC4Threads / 32 - 1) / (kC4Threads / 32), top = int64_t(148) * per_sm;
  return static_cast<unsigned>(n < 1 ? 1 : (n < top ? n : top));
}

int64_t table_rows(const Pages4& pg) { return pg.max_pages * pg.blocks * kC4Rows; }

}  // namespace

cudaError_t launch_compact_int4(const void* K, const void* V, int64_t B, int64_t n_c, int d, const int32_t* idx,
                                const int32_t* counts, const int64_t* offsets, const Pages4& pg, int32_t* status,
                                cudaStream_t stream) {
  const uint16_t *k = static_cast<const uint16_t*>(K), *v = static_cast<const uint16_t*>(V);
  const unsigned grid = grid_for(B * (table_rows(pg) / kC4Rows + 1), kCompactCtas);   // (the counts are on the device)
  return launch_after(d == 128 ? compact_int4_kernel<128> : compact_int4_kernel<64>, dim3(grid), dim3(kC4Threads), 0, stream,
                      0, k, v, B, n_c, idx, counts, offsets, pg, table_rows(pg), status);
}

cudaError_t launch_expand_int4(const Pages4& pg, const int32_t* counts, const int32_t* first, const int64_t* offsets,
                               int64_t B, int d, void* K_out, void* V_out, int64_t n_rows, int32_t* status,
                               cudaStream_t stream) {
  uint16_t *k = static_cast<uint16_t*>(K_out), *v = static_cast<uint16_t*>(V_out);
  const int64_t units = n_rows / kC4Rows + 2 * B;
  const bool split = units <= kExpandSplit;
  const unsigned grid = grid_for(split ? 2 * units : units, kExpandCtas);
  const auto kernel = split ? (d == 128 ? expand_int4_kernel<128, true> : expand_int4_kernel<64, true>)
                            : (d == 128 ? expand_int4_kernel<128, false> : expand_int4_kernel<64, false>);
  return launch_after(kernel, dim3(grid), dim3(kC4Threads), 0, stream, 0, pg, counts, first, offsets, B, table_rows(pg), k, v,
                      n_rows, status);
}

cudaError_t launch_append_int4(int d, const Append4Args& a, cudaStream_t stream) {
  const int64_t pw = 16 / (d / 8);                            // pairs per warp
  const int64_t n_pairs = a.T / 2 + 1;                        // a run of T slots touches at most this many
  const int64_t n_warps = a.counts_out == nullptr ? 0 : a.B;
  const int64_t kv_warps = (a.B * n_pairs + pw - 1) / pw;
  const int64_t q_warps = a.q == nullptr ? 0 : (a.B * a.T * ((a.G + kQHeads - 1) / kQHeads) * (d / 16) + 31) / 32;
  const int64_t grid = ((n_warps + 2 * kv_warps + q_warps) * 32 + kAppendThreads - 1) / kAppendThreads;
  return launch_after(d == 128 ? append_int4_kernel<128> : append_int4_kernel<64>, dim3(static_cast<unsigned>(grid)),
                      dim3(kAppendThreads), 0, stream, 0, a, static_cast<uint32_t>(n_warps), static_cast<uint32_t>(n_pairs),
                      static_cast<uint32_t>(kv_warps), static_cast<uint32_t>(q_warps), table_rows(a.pg));
}

}  // namespace kvz
