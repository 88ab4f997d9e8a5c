// Writing and reading the paged 4-bit cache (layout and quantisation in
// kvz_cache4.cuh): kept rows into it (compaction), new rows behind them with
// the position rotation on the way (append), and rows back to bf16 (expand).
//
// All three move rows through registers, a warp per row pair (d = 128) or two
// pairs (d = 64), a lane per 8 dims: 16-byte loads and stores on the bf16
// side; on the 4-bit side a warp's stores of a pair cover its 128 bytes of K
// codes, 128 of V codes and its scale words whole.  HBM-bound: 4 d bytes of
// bf16 and 9/8 d bytes of the cache per row.
#include <cuda_runtime.h>

#include <cstdint>

#include "kvz.h"
#include "kvz_cache4.cuh"
#include "kvz_internal.h"
#include "kvz_rotary.cuh"
#include "kvz_sm100.cuh"

namespace kvz {

namespace {

constexpr int kC4Threads = 256;
constexpr int kC4Unroll = 4;                                  // units of a warp in flight

__device__ __forceinline__ uint4 ld_stream16(const void* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The pairs of all heads as one index space: head b's pairs start at
// pair_base(b) = offsets[b] / 2 + b, which leaves room for one more than half
// its rows (a run of n rows touches at most n / 2 + 1 pairs), so a unit finds
// its head by bisection and heads of any lengths share the grid evenly.
__device__ __forceinline__ int64_t pair_base(const int64_t* offsets, int64_t b) { return (offsets[b] >> 1) + b; }
__device__ __forceinline__ int64_t head_of(const int64_t* offsets, int64_t B, int64_t u) {
  int64_t lo = 0, hi = B - 1;                                 // largest b with pair_base(b) <= u
  while (lo < hi) {
    const int64_t mid = (lo + hi + 1) >> 1;
    if (pair_base(offsets, mid) <= u) lo = mid; else hi = mid - 1;
  }
  return lo;
}

template <int D>
__global__ void __launch_bounds__(kC4Threads)
    compact_int4_kernel(const uint16_t* __restrict__ K, const uint16_t* __restrict__ V, int64_t B, int64_t n_c,
                        const int32_t* __restrict__ idx, const int32_t* __restrict__ counts,
                        const int64_t* __restrict__ offsets, Pages4 pg, int64_t cap, int32_t* status) {
  using L = C4<D>;
  constexpr int PW = 16 / L::LPR;                             // pairs per warp step: 1 or 2
  const int lane = threadIdx.x & 31, l = lane % L::LPR;
  const int e = (lane / L::LPR) & 1, sub = lane / (2 * L::LPR);
  const int64_t total = pair_base(offsets, B);
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kC4Threads + threadIdx.x) >> 5;
  const int64_t n_warps = static_cast<int64_t>(gridDim.x) * (kC4Threads / 32);
  for (int64_t u0 = warp * (PW * kC4Unroll); u0 < total; u0 += n_warps * (PW * kC4Unroll)) {
    int64_t b = head_of(offsets, B, u0);
    uint4 kv[kC4Unroll], vv[kC4Unroll];
    uint8_t* blk[kC4Unroll];
    int row[kC4Unroll];
#pragma unroll
    for (int i = 0; i < kC4Unroll; ++i) {
      const int64_t u = u0 + i * PW + sub;
      blk[i] = nullptr;
      row[i] = e;
      kv[i] = vv[i] = make_uint4(0u, 0u, 0u, 0u);
      if (u >= total) continue;
      while (b + 1 < B && pair_base(offsets, b + 1) <= u) ++b;
      const int64_t n = counts[b], o = offsets[b];
      const int64_t p = 2 * (u - pair_base(offsets, b)) + e;  // slot of this lane's row
      if (n < 0 || n > offsets[b + 1] - o || n > cap) {
        if (p == 0 && l == 0) report(status, KVZ_ERR_INVALID_ARG);
        continue;
      }
      if (p >= n) continue;
      blk[i] = block_at<D>(pg, b, static_cast<uint32_t>(p >> 4), status);
      row[i] = static_cast<int>(p & 15);
      const int64_t j = idx[o + p];
      if (j >= 0 && j < n_c) {
        const int64_t at = (b * n_c + j) * D + 8 * l;
        kv[i] = ld_stream16(K + at);
        vv[i] = ld_stream16(V + at);
      } else if (l == 0) {
        report(status, KVZ_ERR_INVALID_ARG);                  // idx out of [0, n_c): a row of zeros
      }
    }
#pragma unroll
    for (int i = 0; i < kC4Unroll; ++i) {
      uint32_t code[8], sm;
      bool fine = quantise8(kv[i], code, sm);
      if (blk[i] != nullptr) store_k<D>(blk[i], row[i], l, code, fine, sm);
      fine = quantise8(vv[i], code, sm);
      store_v<D>(blk[i], row[i], l, code, fine, sm, blk[i] != nullptr);
    }
  }
}

// Rows first[b] .. counts[b] - 1 as bf16 rows offsets[b], offsets[b] + 1, ...
template <int D>
__global__ void __launch_bounds__(kC4Threads)
    expand_int4_kernel(Pages4 pg, const int32_t* __restrict__ counts, const int32_t* __restrict__ first,
                       const int64_t* __restrict__ offsets, int64_t B, int64_t cap, uint16_t* __restrict__ K_out,
                       uint16_t* __restrict__ V_out, int64_t n_rows, int32_t* status) {
  using L = C4<D>;
  constexpr int PW = 16 / L::LPR;
  const int lane = threadIdx.x & 31, l = lane % L::LPR;
  const int e = (lane / L::LPR) & 1, sub = lane / (2 * L::LPR);
  const int g = l / 8, c = (l % 8) / 2, uu = l % 2, r = l % 8;
  const int64_t total = pair_base(offsets, B);
  const int64_t warp = (static_cast<int64_t>(blockIdx.x) * kC4Threads + threadIdx.x) >> 5;
  const int64_t n_warps = static_cast<int64_t>(gridDim.x) * (kC4Threads / 32);
  for (int64_t u0 = warp * (PW * kC4Unroll); u0 < total; u0 += n_warps * (PW * kC4Unroll)) {
    int64_t b = head_of(offsets, B, u0);
    uint32_t kw[kC4Unroll], ks[kC4Unroll], vs[kC4Unroll];
    uint2 vw[kC4Unroll];
    int64_t dst[kC4Unroll];
#pragma unroll
    for (int i = 0; i < kC4Unroll; ++i) {
      const int64_t u = u0 + i * PW + sub;
      dst[i] = -1;
      if (u >= total) continue;
      while (b + 1 < B && pair_base(offsets, b + 1) <= u) ++b;
      const int64_t n = counts[b], f = first == nullptr ? 0 : first[b], o = offsets[b];
      const int64_t p = 2 * ((f >> 1) + u - pair_base(offsets, b)) + e;
      if (f < 0 || n < f || n > cap || n - f > offsets[b + 1] - o || o < 0 || o + (n - f) > n_rows) {
        if (u == pair_base(offsets, b) && l == 0) report(status, KVZ_ERR_INVALID_ARG);
        continue;
      }
      if (p < f || p >= n) continue;
      const uint8_t* blk = block_at<D>(pg, b, static_cast<uint32_t>(p >> 4), status);
      if (blk == nullptr) continue;
      const int row = static_cast<int>(p & 15);
      kw[i] = __ldg(reinterpret_cast<const uint32_t*>(blk + row * (D / 2) + (c * L::NG * 2 + g * 2 + uu) * 4));
      vw[i] = __ldg(reinterpret_cast<const uint2*>(blk + L::V_OFF + (row >> 1) * D + (r * L::NG + g) * 8));
      ks[i] = __ldg(reinterpret_cast<const uint32_t*>(blk + L::KS_OFF + (row * L::NG + g) * 4));
      vs[i] = __ldg(reinterpret_cast<const uint32_t*>(blk + L::VS_OFF + (row * L::NG + g) * 4));
      dst[i] = (o + p - f) * D + 8 * l;
    }
#pragma unroll
    for (int i = 0; i < kC4Unroll; ++i) {
      if (dst[i] < 0) continue;
      float s = bf_lo(ks[i]), m = bf_hi(ks[i]);
      const uint32_t w = __funnelshift_r(kw[i], kw[i], 3);
      uint4 y;
      y.x = pack_bf2(widen4(w, s, m), widen4(w >> 16, s, m));
      y.y = pack_bf2(widen4(w >> 4, s, m), widen4(w >> 20, s, m));
      y.z = pack_bf2(widen4(w >> 8, s, m), widen4(w >> 24, s, m));
      y.w = pack_bf2(widen4(w >> 12, s, m), widen4(w >> 28, s, m));
      *reinterpret_cast<uint4*>(K_out + dst[i]) = y;
      s = bf_lo(vs[i]), m = bf_hi(vs[i]);
      const uint32_t h = e ? 16u : 0u;
      const uint32_t a = vw[i].x >> h, z = vw[i].y >> h;
      y.x = pack_bf2(widen4(a, s, m), widen4(a >> 4, s, m));
      y.y = pack_bf2(widen4(a >> 8, s, m), widen4(a >> 12, s, m));
      y.z = pack_bf2(widen4(z, s, m), widen4(z >> 4, s, m));
      y.w = pack_bf2(widen4(z >> 8, s, m), widen4(z >> 12, s, m));
      *reinterpret_cast<uint4*>(V_out + dst[i]) = y;
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
      const float4 c = __ldg(reinterpret_cast<const float4*>(t));
      const float4 s = __ldg(reinterpret_cast<const float4*>(t + rot.rot / 2));
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

// Append.  Warps take, in this order: K row pairs, V row pairs, query rows,
// and one head each for the new counts.  Pair j of head b covers the slots
// 2 (counts[b] / 2 + j) and the next, of which those in [counts[b], counts[b]
// + n_new[b]) are written; a slot's other half and all later rows stay as
// they were.  A single token is latency (the count, the page and the row one
// after another), so K, V and queries go to warps of their own.
template <int D>
__global__ void __launch_bounds__(kC4Threads) append_int4_kernel(Append4Args a, int n_pairs, int64_t kv_warps,
                                                                 int64_t q_warps, int64_t cap) {
  using L = C4<D>;
  constexpr int PW = 16 / L::LPR;
  const int lane = threadIdx.x & 31, l = lane % L::LPR;
  int64_t w = (static_cast<int64_t>(blockIdx.x) * kC4Threads + threadIdx.x) >> 5;
  const bool turning = a.rot.pos != nullptr;

  if (w < 2 * kv_warps) {
    const bool is_k = w < kv_warps;
    if (!is_k) w -= kv_warps;
    const int e = (lane / L::LPR) & 1, sub = lane / (2 * L::LPR);
    const int64_t f = w * PW + sub, b = f / n_pairs;
    const int j = static_cast<int>(f - b * n_pairs);
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    uint8_t* blk = nullptr;
    int row = e;
    int64_t p = 0;
    if (b < a.B) {
      const int64_t base = a.counts[b], len = a.n_new == nullptr ? a.T : a.n_new[b];
      const bool head_ok = base >= 0 && len >= 0 && len <= a.T && base + len <= cap;
      if (!head_ok && is_k && j == 0 && e == 0 && l == 0) report(a.status, KVZ_ERR_INVALID_ARG);
      const int64_t slot = 2 * ((base >> 1) + j) + e, t = slot - base;
      if (head_ok && t >= 0 && t < len) {
        x = is_k ? *reinterpret_cast<const uint4*>(a.k + b * a.k_sb + t * a.k_st + 8 * l)
                 : *reinterpret_cast<const uint4*>(a.v + b * a.v_sb + t * a.v_st + 8 * l);
        blk = block_at<D>(a.pg, b, static_cast<uint32_t>(slot >> 4), a.status);
        row = static_cast<int>(slot & 15);
        if (turning) {
          p = a.rot.pos[b * a.rot.pos_sb + t];
          if (p < 0 || p >= a.rot.n_pos) {
            report(a.status, KVZ_ERR_INVALID_ARG);
            blk = nullptr;
          }
        }
      }
    }
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
    const int64_t f = w * (2 * PW) + lane / L::LPR;           // query row (b, g, t)
    uint4 x = make_uint4(0u, 0u, 0u, 0u);
    int64_t p = 0;
    bool on = false;
    if (f < a.B * a.G * a.T) {
      const int64_t t = f % a.T, bg = f / a.T, b = bg / a.G;
      const int g = static_cast<int>(bg - b * a.G);
      const int64_t len = a.n_new == nullptr ? a.T : a.n_new[b];
      if (t < len) {                                          // (a bad length is reported with the head's keys)
        x = *reinterpret_cast<const uint4*>(a.q + b * a.q_sb + g * a.q_sg + t * a.q_st + 8 * l);
        on = true;
        if (turning) {
          p = a.rot.pos[b * a.rot.pos_sb + t];
          on = p >= 0 && p < a.rot.n_pos;
        }
      }
    }
    if (turning) turn_row<D>(x, lane, l, a.rot, p, on);
    if (on) *reinterpret_cast<uint4*>(a.q_out + f * D + 8 * l) = x;
    return;
  }
  w -= q_warps;
  if (a.counts_out != nullptr && w < a.B) {
    // the new count, if every page and position of the head's new rows is valid
    const int64_t b = w, base = a.counts[b], len = a.n_new == nullptr ? a.T : a.n_new[b];
    bool ok = base >= 0 && len >= 0 && len <= a.T && base + len <= cap;
    if (ok && len > 0) {
      const int64_t p0 = page_of(a.pg, static_cast<uint32_t>(base >> 4));
      const int64_t p1 = page_of(a.pg, static_cast<uint32_t>((base + len - 1) >> 4));
      for (int64_t i = p0 + lane; i <= p1; i += 32) {
        const int32_t id = a.pg.pages[b * a.pg.max_pages + i];
        ok = ok && id >= 0 && id < a.pg.n_pages;
      }
      if (turning)
        for (int64_t t = lane; t < len; t += 32) {
          const int64_t p = a.rot.pos[b * a.rot.pos_sb + t];
          ok = ok && p >= 0 && p < a.rot.n_pos;
        }
    }
    ok = __all_sync(kFullMask, ok);
    if (lane == 0) a.counts_out[b] = static_cast<int32_t>(ok ? base + len : base);
  }
}

unsigned persistent_grid(int per_sm) { return 148u * static_cast<unsigned>(per_sm); }

int64_t table_rows(const Pages4& pg) { return pg.max_pages * pg.blocks * kC4Rows; }

}  // namespace

cudaError_t launch_compact_int4(const void* K, const void* V, int64_t B, int64_t n_c, int d, const int32_t* idx,
                                const int32_t* counts, const int64_t* offsets, const Pages4& pg, int32_t* status,
                                cudaStream_t stream) {
  const uint16_t *k = static_cast<const uint16_t*>(K), *v = static_cast<const uint16_t*>(V);
  if (d == 128)
    compact_int4_kernel<128><<<persistent_grid(4), kC4Threads, 0, stream>>>(k, v, B, n_c, idx, counts, offsets, pg,
                                                                            table_rows(pg), status);
  else
    compact_int4_kernel<64><<<persistent_grid(4), kC4Threads, 0, stream>>>(k, v, B, n_c, idx, counts, offsets, pg,
                                                                           table_rows(pg), status);
  return cudaGetLastError();
}

cudaError_t launch_expand_int4(const Pages4& pg, const int32_t* counts, const int32_t* first, const int64_t* offsets,
                               int64_t B, int d, void* K_out, void* V_out, int64_t n_rows, int32_t* status,
                               cudaStream_t stream) {
  uint16_t *k = static_cast<uint16_t*>(K_out), *v = static_cast<uint16_t*>(V_out);
  if (d == 128)
    expand_int4_kernel<128><<<persistent_grid(4), kC4Threads, 0, stream>>>(pg, counts, first, offsets, B,
                                                                           table_rows(pg), k, v, n_rows, status);
  else
    expand_int4_kernel<64><<<persistent_grid(4), kC4Threads, 0, stream>>>(pg, counts, first, offsets, B,
                                                                          table_rows(pg), k, v, n_rows, status);
  return cudaGetLastError();
}

cudaError_t launch_append_int4(int d, const Append4Args& a, cudaStream_t stream) {
  const int pw = 16 / (d / 8);                                // pairs per warp
  const int n_pairs = static_cast<int>(a.T / 2 + 1);          // a run of T slots touches at most this many
  const int64_t kv_warps = (a.B * n_pairs + pw - 1) / pw;
  const int64_t q_warps = a.q == nullptr ? 0 : (a.B * a.G * a.T + 2 * pw - 1) / (2 * pw);
  const int64_t warps = 2 * kv_warps + q_warps + (a.counts_out == nullptr ? 0 : a.B);
  const int64_t grid = (warps * 32 + kC4Threads - 1) / kC4Threads;
  if (grid > 0x7FFFFFFF) return cudaErrorInvalidValue;
  if (d == 128)
    append_int4_kernel<128><<<static_cast<unsigned>(grid), kC4Threads, 0, stream>>>(a, n_pairs, kv_warps, q_warps,
                                                                                    table_rows(a.pg));
  else
    append_int4_kernel<64><<<static_cast<unsigned>(grid), kC4Threads, 0, stream>>>(a, n_pairs, kv_warps, q_warps,
                                                                                   table_rows(a.pg));
  return cudaGetLastError();
}

}  // namespace kvz
