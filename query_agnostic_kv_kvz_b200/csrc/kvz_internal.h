// Launchers shared between the C ABI (kvz_api.cu) and the kernel files.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

namespace kvz {

// Set a kernel's attribute once per device (the launch paths call this before
// every launch; the attribute call itself is a host round trip worth
// skipping).  `value` is a constant of the kernel.
template <auto Kernel, cudaFuncAttribute Attr>
cudaError_t attribute_once(int value) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev >= 0 && dev < 64 ? (uint64_t(1) << dev) : 0;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(Kernel, Attr, value);
  if (e == cudaSuccess && bit != 0) done.fetch_or(bit, std::memory_order_release);
  return e;
}
template <auto Kernel>
cudaError_t smem_limit_once(int bytes) {                      // dynamic shared memory
  return attribute_once<Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize>(bytes);
}
template <auto Kernel>
cudaError_t wide_clusters_once() {                            // clusters of more than 8 CTAs
  return attribute_once<Kernel, cudaFuncAttributeNonPortableClusterSizeAllowed>(1);
}

// Pass 1 (row log-sum-exp) arguments.  Rows i in [i_begin, i_end) are
// computed; rows_pad = roundup(i_end - i_begin, 256) entries per (b, g) are
// written at lse2[(b*G + g)*ld + (i - i_begin)], padding rows set to +inf.
// A call scores B independent problems (query groups against context keys).
// Problem p reads context-key block (p % T) of head (p / T): T = 1 for the
// plain score, T = chunks per head for chunked scoring (the context-key map
// is 4-D: columns, rows of a block, block, head).
// Grid: one CTA per (head, group, 256-row block) unit, longest first; the
// last r units (the partial last wave) may each be split into `nsplit`
// CTAs over consecutive key-tile ranges.  CTA x < n_full computes unit x
// whole; CTA n_full + t computes part t % nsplit of unit n_full + t / nsplit
// and writes its rows' partial (reference m, sum of 2^(c2 s - m)) to
// part[t * 256 + row]; a merge kernel then combines the parts of each unit
// in order.
struct LseArgs {
  int B, G, T;
  int64_t n_c, n_in;
  float c2;                 // scale * log2(e)
  int64_t i_begin, i_end, rows_pad, ld;
  float* lse2;
  int32_t* status;
  int n_full;               // CTAs that compute a whole unit (set by launch_lse)
  int nsplit;               // parts per split unit, 1 = none (set by launch_lse)
  float2* part;             // [split CTAs][256] partial (reference, sum); null = no split
  int head_major;           // unit order: 0 = row block, then (head, group); 1 = head, then row block, then
                            // group (set by launch_lse)
  int wave;                 // CTAs resident at once (the SM count; 0 = unknown) (set by launch_lse)
};
// Scratch for split units: at most this many split CTAs, 256 rows of
// (max, sum) each.
constexpr int kLseMaxSplitCtas = 256;
constexpr size_t kLsePartBytes = static_cast<size_t>(kLseMaxSplitCtas) * 256 * 8;

// Pass 2 (context-key column max) arguments; lse2 as pass 1 wrote it.
struct ColArgs {
  int B, G, T;
  int64_t n_c;
  float c2;
  int64_t i_begin, rows_pad, ld;
  const float* lse2;
  float* S;                 // problem p writes S[(p / T) * ldS + (p % T) * s_block + j], j < n_c
  int64_t ldS, s_block;
  int n_kblk;               // key blocks per head (set by launch_colmax)
  int nsplit;               // row-tile ranges per (head, key block) (set by launch_colmax)
  int tiles_per_split;      // (set by launch_colmax)
  int32_t* status;
};

cudaError_t launch_lse(int d, const CUtensorMap& tmQ, const CUtensorMap& tmKc, const CUtensorMap& tmKi,
                       const LseArgs& a, cudaStream_t stream);
cudaError_t launch_colmax(int d, const CUtensorMap& tmQ, const CUtensorMap& tmKc, const ColArgs& a,
                          cudaStream_t stream);
cudaError_t launch_fill_f32(float* x, int64_t n, float v, cudaStream_t stream);

// Decode attention over the pruned cache (a device-built work list of equal
// splits; split-KV partials merged by a two-level tree).
constexpr int kDecGMax = 8;                 // grouped queries per KV head
// One CTA of the decode kernel: split sp of head b, tiles t0 .. t0+n-1 of
// the head's 64-key tiles; its partial is written at the item's index, the
// head's nsp partials at indices (index - sp) .. (index - sp + nsp - 1).
struct __align__(16) DecItem {
  int b, sp, t0, n;                         // n == 0: nothing to do
  int count, nsp;                           // the head's kept rows and splits
  long long off;                            // the head's first row in K_out / V_out
};
static_assert(sizeof(DecItem) == 32, "two 16-byte loads");

struct DecArgs {
  int B, G;
  int64_t n_c;                              // upper bound of counts[b]
  float c2;                                 // scale * log2(e)
  const uint16_t* q;                        // bf16 [B][G][d]
  const int32_t* counts;
  const int64_t* offsets;
  int n_items;                              // decode CTAs (grid.x): kDecWave + B bounds the splits
  DecItem* items;                           // [n_items], written by the plan kernel
  float2* part_ml;                          // [n_items][G] (running max, sum), base 2
  float* part_o;                            // [n_items][G][d]
  unsigned* done;                           // [B] split groups merged per head (zeroed by the plan kernel)
  unsigned* gdone;                          // [n_items] splits finished per group, at the group's first item
  int32_t* status;
};
constexpr int kDecWave = 148 * 3;           // about 1.5 waves of two decode CTAs per SM (best of 2, 3, 4, 6 per SM)
inline int decode_items(int64_t B) { return static_cast<int>(kDecWave + B); }
cudaError_t launch_decode(int d, const CUtensorMap& tmK, const CUtensorMap& tmV, const DecArgs& a, float* out,
                          float* lse2, cudaStream_t stream);

// Head scores (segmented max of S) and the CSR form of a head-level selection.
cudaError_t launch_head_max(const float* S, int64_t B, int64_t n_c, float* S_head, int32_t* status,
                            cudaStream_t stream);
cudaError_t launch_head_expand(const int32_t* kept, int64_t k, int64_t B, int64_t n_c, int32_t* idx,
                               int32_t* counts, int64_t* offsets, cudaStream_t stream);

// Selection.  Workspace layout is computed by select_workspace().
struct SelWorkspace {
  size_t bytes;
  size_t off_state, off_hist, off_cg, off_ce, off_eqb, off_cbase, off_head_eq, off_head_base;
};
SelWorkspace select_workspace(int64_t B, int64_t n_c, int mode);
cudaError_t launch_select(const float* S, int64_t B, int64_t n_c, int64_t n_protect, int mode, int64_t k,
                          int32_t* idx, int32_t* counts, int64_t* offsets, void* ws, const SelWorkspace& lay,
                          int32_t* status, cudaStream_t stream);
cudaError_t launch_select_dist_begin(const float* S, int64_t B, int64_t n_c, int64_t k, uint32_t* hist, void* ws,
                                     const SelWorkspace& lay, int32_t* status, cudaStream_t stream);
cudaError_t launch_select_dist_step(const float* S, int64_t B, int64_t n_c, int pass, uint32_t* hist,
                                    unsigned long long* eq_total, void* ws, const SelWorkspace& lay,
                                    int32_t* status, cudaStream_t stream);
cudaError_t launch_select_dist_finish(const float* S, int64_t B, int64_t n_c, const unsigned long long* eq_ranks,
                                      int rank, int32_t* idx, int32_t* counts, int64_t* offsets, void* ws,
                                      const SelWorkspace& lay, cudaStream_t stream);

// Compaction.
cudaError_t launch_compact_gather(const void* K, const void* V, int64_t B, int64_t n_c, int d,
                                  const int32_t* idx, const int64_t* offsets, const int64_t* out_offsets,
                                  void* K_out, void* V_out, int32_t* status, cudaStream_t stream);
// In place: `ws` holds B + B*ceil(n_c/chunk) uint32 (per-head chunk claims and
// per-chunk "sources read" flags); the launcher zeroes it on `stream`.
// `wait_ns` bounds each ordering wait (kInplaceWaitNs normally); when hold_b
// and hold_c are both >= 0, chunk hold_c of head hold_b never publishes that
// its sources were read, so a chunk waiting on it times out (test use only).
constexpr uint64_t kInplaceWaitNs = 1000ull * 1000ull * 1000ull;   // 1 s: far beyond any legitimate wait
cudaError_t launch_compact_inplace(void* K, void* V, int64_t B, int64_t n_c, int d, const int32_t* idx,
                                   const int32_t* counts, const int64_t* offsets, uint32_t* ws, int32_t* status,
                                   cudaStream_t stream, uint64_t wait_ns = kInplaceWaitNs, int64_t hold_b = -1,
                                   int64_t hold_c = -1);
size_t compact_workspace_bytes(int64_t B, int64_t n_c);
// Out-of-place compaction into int8 codes with one fp32 scale per row.
cudaError_t launch_compact_int8(const void* K, const void* V, int64_t B, int64_t n_c, int d, const int32_t* idx,
                                const int32_t* counts, const int64_t* offsets, const int64_t* out_offsets,
                                int8_t* Kq, int8_t* Vq, float* K_scale, float* V_scale, int32_t* status,
                                cudaStream_t stream);

// The paged 4-bit cache (layout in kvz_cache4.cuh): `cache` is a pool of
// n_pages pages, pages[b][i] the page of rows [i * page_size, (i + 1) *
// page_size) of head b.
struct Pages4 {
  uint8_t* cache;
  int64_t n_pages;
  const int32_t* pages;                     // [B][max_pages]
  int64_t max_pages;
  uint32_t blocks;                          // 16-row blocks per page
  uint32_t inv;                             // floor(2^32 / blocks) + 1 (0 when blocks == 1)
};
// blk / blocks for blk < 2^26 and blocks <= 64: inv * blocks exceeds 2^32 by
// at most 64, so the product is off by less than 2^32 / blocks.
__host__ __device__ inline uint32_t page_of(const Pages4& p, uint32_t blk) {
  return p.inv == 0 ? blk : static_cast<uint32_t>((static_cast<uint64_t>(blk) * p.inv) >> 32);
}

// Kept rows of K, V [B][n_c][d] into the 4-bit cache.
cudaError_t launch_compact_int4(const void* K, const void* V, int64_t B, int64_t n_c, int d, const int32_t* idx,
                                const int32_t* counts, const int64_t* offsets, const Pages4& pg, int32_t* status,
                                cudaStream_t stream);
// Rows first[b] .. counts[b] of the 4-bit cache as bf16 rows from offsets[b] on.
cudaError_t launch_expand_int4(const Pages4& pg, const int32_t* counts, const int32_t* first, const int64_t* offsets,
                               int64_t B, int d, void* K_out, void* V_out, int64_t n_rows, int32_t* status,
                               cudaStream_t stream);

// Rotary positions.  Strides in elements; pos_sb is 0 for positions shared by all heads.
struct RotArgs {
  const int32_t* pos;                       // null: no rotation
  int64_t pos_sb;
  const float* table;                       // [n_pos][rot]: rot/2 cosines, rot/2 sines
  int64_t n_pos;
  int rot, interleaved, inverse;
};
struct RotaryArgs {
  const uint16_t* x;
  int64_t x_sb, x_sg, x_st;
  uint16_t* y;
  int64_t y_sb, y_sg, y_st;
  int64_t B, T;
  int G;
  RotArgs rot;
  int32_t* status;
};
cudaError_t launch_rotary(int d, const RotaryArgs& a, cudaStream_t stream);
cudaError_t launch_rotary_table(const double* freqs, int64_t n_pos, int rot, double factor, float* table,
                                cudaStream_t stream);

// New rows behind each head's counts[b] rows of the 4-bit cache.
struct Append4Args {
  const uint16_t *k, *v, *q;                // q may be null
  int64_t k_sb, k_st, v_sb, v_st, q_sb, q_sg, q_st;
  uint16_t* q_out;                          // [B][G][T][d]
  int64_t B, T;
  int G;
  RotArgs rot;
  Pages4 pg;
  const int32_t* counts;
  const int32_t* n_new;                     // null: T rows each
  int32_t* counts_out;                      // may be null
  int32_t* status;
};
cudaError_t launch_append_int4(int d, const Append4Args& a, cudaStream_t stream);

// Decode attention over the 4-bit cache: kD4Workers CTAs share the heads' 16-row
// blocks evenly; the heads that more than one CTA read are merged.
constexpr int kD4Workers = 148 * 2;         // two CTAs per SM
struct Dec4Args {
  Pages4 pg;
  int64_t B;
  int G;
  int64_t cap;                              // rows a head's page table can hold
  float c2;                                 // scale * log2(e)
  const uint16_t* q;                        // bf16 [B][G][d]
  const int32_t* counts;
  float* out;                               // [B][G][d]
  float* lse2;                              // [B][G], may be null
  int4* cont;                               // [kD4Workers] the head that runs past each CTA's range
  float2* part_ml;                          // [2 * kD4Workers][8] partial (reference, sum)
  float* part_o;                            // [2 * kD4Workers][G][d]
  int32_t* status;
  // the test entry point's only: its waits' limit, and the head and CTA (-1: any) whose first stage stays away
  uint64_t wait_ns = 0;
  int64_t hold_head = -1, hold_cta = -1;
  int max_cluster = 16;                     // and the widest cluster it may take
};
// The cluster form (decode4_kernels.cu): the CTAs that read a head whose page
// table holds `cap` rows, or 0 for shares of equal work; `alone`: each on an SM
// of its own.  us at d = 128, G = 4, clusters against shares:
//   1 head     2,000 rows 5.0 : 8.2    8,000 rows  7.3 :  8.7   16,000 rows 10.5 : 9.2
//   6 heads               5.5 : 9.0                7.8 : 11.4               11.0 : 12.9
//   12 heads              6.1 : 11.0              10.9 : 12.6               17.1 : 15.8
//   20 heads              7.5 : 11.5   4,000 rows 10.7 : 12.6    6,000 rows 13.9 : 13.6
//   32 heads             10.5 : 12.5   8,000 rows 18.6 : 18.4   12,000 rows 22.9 : 22.0
//   64 heads             10.2 : 15.0   4,000 rows 15.2 : 18.9    6,000 rows 19.7 : 22.9
//   96 heads             14.9 : 17.9   4,000 rows 24.1 : 23.7    6,000 rows 33.9 : 30.6
// So clusters take the shorter heads.  Lengths are on the device, so the
// table's width stands for the longest.  Few heads: the most CTAs up to 96
// that have an SM each (more clusters do not fit the GPU's GPCs side by side:
// 16 heads by 8 CTAs 8.7 us packed, 12.1 alone, by 4 alone 8.0 at 2,000 rows).
// Else the most up to 256 (37 heads by 8 CTAs, 296 in all, 15.0; by 4, 11.0).
// CTAs of 16 warps, which fill an SM: 7.1 against 6.7 for 8 heads of 2,457 rows.
struct Decode4Form {
  int cluster;
  bool alone;
};
inline Decode4Form decode4_form(int64_t B, int64_t cap) {
  for (int c = 16; c >= 4; c /= 2)
    if (c * B <= 96) return Decode4Form{cap <= c * 1280 ? c : 0, true};
  int c = 1;
  while (c < 8 && 2 * c * B <= 256) c *= 2;
  return Decode4Form{cap <= c * (c <= 4 && c * B >= 192 ? 2048 : 1280) ? c : 0, false};
}
cudaError_t launch_decode_int4(int d, const Dec4Args& a, cudaStream_t stream);

}  // namespace kvz
