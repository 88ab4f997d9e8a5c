// Rotary positions (the queries and keys that scoring, the cache and the
// attention take are post-positional features).
//
// A pair (a, b) of a row at position p turns by theta = p * f_i:
//   a' = a cos - b sin,  b' = b cos + a sin
// The pairs are (x[i], x[i + rot/2]) or, interleaved, (x[2i], x[2i + 1]) of
// the first rot dims; the other dims pass through.  Every product and sum is
// one float32 operation, rounded to bf16 once, so the appended keys (which
// turn by the same steps) match rows turned here bit for bit.
#include <cuda_runtime.h>

#include <cstdint>

#include "kvz.h"
#include "kvz_internal.h"
#include "kvz_launch.cuh"
#include "kvz_rotary.cuh"
#include "kvz_sm100.cuh"

namespace kvz {

namespace {

constexpr int kRotThreads = 128;
constexpr int kRotUnroll = 4;                                 // rows in flight per thread
constexpr int kRotHeads = 8;                                  // rows a thread walks at most

// The angle of a far position needs more than 32 bits (131072 * f in float32
// is off by 2^-8 rad), so angle, cosine and sine are float64 and each entry is
// rounded once.  Run once per model, not on any hot path.
__global__ void __launch_bounds__(kRotThreads)
    rotary_table_kernel(const double* freqs, int64_t n, int half, double factor, float* table) {
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * kRotThreads + threadIdx.x; e < n;
       e += static_cast<int64_t>(gridDim.x) * kRotThreads) {
    const int64_t p = e / half;
    const int i = static_cast<int>(e % half);
    double s, c;
    sincos(static_cast<double>(p) * freqs[i], &s, &c);
    table[p * 2 * half + i] = static_cast<float>(c * factor);
    table[p * 2 * half + half + i] = static_cast<float>(s * factor);
  }
}

// HBM-bound: every row is read once and written once.  A thread owns 16 dims
// of one token, as two 16-byte vectors that hold whole pairs (so a row can be
// turned in place), keeps their cosines and sines in registers and walks
// `heads` rows of that token, four rows' loads in flight.  8 x 4 heads x 8,224
// tokens x 128 from a token-major projection: 24.1 us = 5.8 TB/s in a chain of
// calls; 2 to 16 heads a thread, 2 or 4 rows in flight and 128 or 256 threads
// all lie within 8% of it.
template <int D, bool IL>
__global__ void __launch_bounds__(kRotThreads) rotary_kernel(RotaryArgs a, int heads, int64_t n_threads) {
  constexpr int IT = D / 16;                                    // items of a row
  let_next_start();
  after_prior(a.x, a.y, a.rot.pos, a.rot.table);
  const int64_t f = static_cast<int64_t>(blockIdx.x) * kRotThreads + threadIdx.x;
  if (f >= n_threads) return;
  const int item = static_cast<int>(f % IT);
  const int64_t ft = f / IT;
  const int64_t t = ft % a.T, chunk = ft / a.T;
  const int rot = a.rot.rot, nrot = rot / 16;
  const bool turn = item < nrot;
  // the item's two vectors (first dims)
  const int d0 = turn ? (IL ? 16 * item : 8 * item) : rot + 16 * (item - nrot);
  const int d1 = turn && !IL ? d0 + rot / 2 : d0 + 8;
  const int64_t rows = a.B * a.G;
  const int64_t r0 = chunk * heads, r1 = r0 + heads < rows ? r0 + heads : rows;
  int64_t b = r0 / a.G;
  int g = static_cast<int>(r0 % a.G);
  float c[8], s[8];
  int64_t have = -1;                                            // head whose angles c, s hold
  bool ok = true;
  for (int64_t r = r0; r < r1; r += kRotUnroll) {
    uint4 v0[kRotUnroll], v1[kRotUnroll];
    int64_t yo[kRotUnroll];
    int64_t hb[kRotUnroll];
#pragma unroll
    for (int j = 0; j < kRotUnroll; ++j) {
      hb[j] = -1;
      if (r + j < r1) {
        const int64_t xo = b * a.x_sb + g * a.x_sg + t * a.x_st;
        v0[j] = *reinterpret_cast<const uint4*>(a.x + xo + d0);
        v1[j] = *reinterpret_cast<const uint4*>(a.x + xo + d1);
        yo[j] = b * a.y_sb + g * a.y_sg + t * a.y_st;
        hb[j] = b;
        if (++g == a.G) {
          g = 0;
          ++b;
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kRotUnroll; ++j) {
      if (hb[j] < 0) continue;
      const int64_t key = a.rot.pos_sb == 0 ? 0 : hb[j];
      if (key != have) {
        have = key;
        const int64_t p = a.rot.pos[key * a.rot.pos_sb + t];
        ok = p >= 0 && p < a.rot.n_pos;
        if (!ok) report(a.status, KVZ_ERR_INVALID_ARG);
        else if (turn) load_angles(a.rot.table + p * rot, rot / 2, 8 * item, a.rot.inverse, c, s);
      }
      if (!ok) continue;
      if (turn) {
        if (IL) turn_adjacent(v0[j], v1[j], c, s);
        else turn_halves(v0[j], v1[j], c, s);
      }
      *reinterpret_cast<uint4*>(a.y + yo[j] + d0) = v0[j];
      *reinterpret_cast<uint4*>(a.y + yo[j] + d1) = v1[j];
    }
  }
}

}  // namespace

cudaError_t launch_rotary_table(const double* freqs, int64_t n_pos, int rot, double factor, float* table,
                                cudaStream_t stream) {
  const int64_t n = n_pos * (rot / 2);
  const int64_t blocks = (n + kRotThreads - 1) / kRotThreads;
  rotary_table_kernel<<<static_cast<unsigned>(blocks < 148 * 8 ? blocks : 148 * 8), kRotThreads, 0, stream>>>(
      freqs, n, rot / 2, factor, table);
  return cudaGetLastError();
}

cudaError_t launch_rotary(int d, const RotaryArgs& a, cudaStream_t stream) {
  const int64_t rows = a.B * a.G, per_row = a.T * (d / 16);
  // rows a thread walks: as many as leave each SM about 1024 threads, 8 at most
  int64_t heads = rows * per_row / (148 * 1024);
  heads = heads < 1 ? 1 : (heads > kRotHeads ? kRotHeads : heads);
  const int64_t n = (rows + heads - 1) / heads * per_row;
  const int64_t blocks = (n + kRotThreads - 1) / kRotThreads;
  if (blocks > 0x7FFFFFFF) return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(blocks);
  const int h = static_cast<int>(heads);
  const auto kernel = d == 128 ? (a.rot.interleaved ? rotary_kernel<128, true> : rotary_kernel<128, false>)
                               : (a.rot.interleaved ? rotary_kernel<64, true> : rotary_kernel<64, false>);
  return launch_after(kernel, dim3(grid), dim3(kRotThreads), 0, stream, 0, a, h, n);
}

}  // namespace kvz
