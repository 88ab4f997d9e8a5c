// C ABI of the rotary positions and of the paged 4-bit cache: argument
// validation and workspace layout.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "kvz.h"
#include "kvz_internal.h"
#include "kvz_testing.h"

namespace {

constexpr int64_t kMaxCacheRows = int64_t(1) << 30;           // rows of one head's page table
constexpr int64_t kMaxStride = int64_t(1) << 40;              // elements

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// A stride that keeps 16-byte vectors aligned, and offsets inside 64 bits.
bool stride_ok(int64_t s) { return s >= 0 && s <= kMaxStride && s % 8 == 0; }

kvz_status check_pages(const void* cache, int64_t n_pages, int page_size, const int32_t* pages, int64_t max_pages,
                       int64_t B, int d, kvz::Pages4* pg) {
  if (cache == nullptr || pages == nullptr) return KVZ_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return KVZ_ERR_UNSUPPORTED;
  if (page_size < 16 || page_size > 1024 || page_size % 16 != 0) return KVZ_ERR_UNSUPPORTED;
  if (B < 1 || B > 65535 || n_pages < 1 || n_pages > 0x7FFFFFFF || max_pages < 1) return KVZ_ERR_INVALID_ARG;
  if (max_pages > kMaxCacheRows / page_size) return KVZ_ERR_INVALID_ARG;
  if (n_pages > 0x7FFFFFFF / (page_size / 16)) return KVZ_ERR_INVALID_ARG;   // a pool's blocks are numbered in 31 bits
  if (!aligned(cache, 16) || !aligned(pages, 4)) return KVZ_ERR_ALIGNMENT;
  pg->cache = static_cast<uint8_t*>(const_cast<void*>(cache));
  pg->n_pages = n_pages;
  pg->pages = pages;
  pg->max_pages = max_pages;
  pg->blocks = static_cast<uint32_t>(page_size / 16);
  pg->inv = pg->blocks == 1 ? 0u : static_cast<uint32_t>((uint64_t(1) << 32) / pg->blocks + 1);
  return KVZ_OK;
}

kvz_status check_rotation(const int32_t* positions, int64_t pos_sb, const float* table, int64_t n_pos, int rot, int d,
                          int interleaved, int inverse, kvz::RotArgs* r) {
  if (positions == nullptr || table == nullptr) return KVZ_ERR_INVALID_ARG;
  if (rot < 16 || rot > d || rot % 16 != 0) return KVZ_ERR_UNSUPPORTED;
  if (pos_sb < 0 || n_pos < 1 || n_pos > 0x7FFFFFFF) return KVZ_ERR_INVALID_ARG;
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1)) return KVZ_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(table, 16)) return KVZ_ERR_ALIGNMENT;
  *r = kvz::RotArgs{positions, pos_sb, table, n_pos, rot, interleaved, inverse};
  return KVZ_OK;
}

kvz_status decode_int4(const void* q, const void* cache, int64_t n_pages, int page_size, const int32_t* pages,
                       int64_t max_pages, const int32_t* counts, int64_t B, int G, int d, float scale, float* out,
                       float* lse2, void* workspace, size_t workspace_bytes, uint64_t wait_ns, int64_t hold_head,
                       int64_t hold_cta, int max_cluster, int32_t* d_status, cudaStream_t stream) {
  if (q == nullptr || counts == nullptr || out == nullptr) return KVZ_ERR_INVALID_ARG;
  kvz::Dec4Args a{};
  const kvz_status st = check_pages(cache, n_pages, page_size, pages, max_pages, B, d, &a.pg);
  if (st != KVZ_OK) return st;
  if (G < 1 || G > kvz::kDecGMax) return KVZ_ERR_UNSUPPORTED;
  if (!std::isfinite(scale) || !(scale > 0.0f)) return KVZ_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(counts, 4) || !aligned(lse2, 4)) return KVZ_ERR_ALIGNMENT;
  const size_t need = kvz_decode_int4_workspace_size(B, G, max_pages * page_size, d);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return KVZ_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return KVZ_ERR_ALIGNMENT;
  a.B = B, a.G = G;
  a.cap = max_pages * page_size;
  a.c2 = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  a.q = static_cast<const uint16_t*>(q);
  a.counts = counts;
  a.out = out, a.lse2 = lse2;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  a.cont = reinterpret_cast<int4*>(w);
  w += up256(kvz::kD4Workers * sizeof(int4));
  a.part_ml = reinterpret_cast<float2*>(w);
  w += up256(2 * kvz::kD4Workers * 8 * sizeof(float2));
  a.part_o = reinterpret_cast<float*>(w);
  a.status = d_status;
  a.wait_ns = wait_ns, a.hold_head = hold_head, a.hold_cta = hold_cta, a.max_cluster = max_cluster;
  return kvz::launch_decode_int4(d, a, stream) == cudaSuccess ? KVZ_OK : KVZ_ERR_CUDA;
}

}  // namespace

extern "C" {

kvz_status kvz_rotary_table(const double* freqs, int64_t n_pos, int rot, double factor, float* table,
                            cudaStream_t stream) {
  if (freqs == nullptr || table == nullptr) return KVZ_ERR_INVALID_ARG;
  if (rot < 16 || rot > 128 || rot % 16 != 0) return KVZ_ERR_UNSUPPORTED;
  if (n_pos < 1 || n_pos > 0x7FFFFFFF || !std::isfinite(factor)) return KVZ_ERR_INVALID_ARG;
  if (!aligned(freqs, 8) || !aligned(table, 16)) return KVZ_ERR_ALIGNMENT;
  return kvz::launch_rotary_table(freqs, n_pos, rot, factor, table, stream) == cudaSuccess ? KVZ_OK : KVZ_ERR_CUDA;
}

kvz_status kvz_rotary(const void* x, int64_t x_sb, int64_t x_sg, int64_t x_st, int64_t B, int G, int64_t n, int d,
                      const int32_t* positions, int64_t pos_sb, const float* table, int64_t n_pos, int rot,
                      int interleaved, int inverse, void* y, int64_t y_sb, int64_t y_sg, int64_t y_st,
                      int32_t* d_status, cudaStream_t stream) {
  if (x == nullptr || y == nullptr) return KVZ_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return KVZ_ERR_UNSUPPORTED;
  if (B < 1 || B > 65535 || G < 1 || G > 65535 || n < 1 || n > 0x7FFFFFFF) return KVZ_ERR_INVALID_ARG;
  kvz::RotaryArgs a{};
  const kvz_status st = check_rotation(positions, pos_sb, table, n_pos, rot, d, interleaved, inverse, &a.rot);
  if (st != KVZ_OK) return st;
  for (int64_t s : {x_sb, x_sg, x_st, y_sb, y_sg, y_st})
    if (!stride_ok(s)) return KVZ_ERR_ALIGNMENT;
  if (!aligned(x, 16) || !aligned(y, 16)) return KVZ_ERR_ALIGNMENT;
  // in place turns every row where it lies; anything between that and apart would read turned rows
  if (x == y && (x_sb != y_sb || x_sg != y_sg || x_st != y_st)) return KVZ_ERR_INVALID_ARG;
  a.x = static_cast<const uint16_t*>(x);
  a.x_sb = x_sb, a.x_sg = x_sg, a.x_st = x_st;
  a.y = static_cast<uint16_t*>(y);
  a.y_sb = y_sb, a.y_sg = y_sg, a.y_st = y_st;
  a.B = B, a.G = G, a.T = n;
  a.status = d_status;
  return kvz::launch_rotary(d, a, stream) == cudaSuccess ? KVZ_OK : KVZ_ERR_CUDA;
}

size_t kvz_cache4_page_bytes(int page_size, int d) {
  if ((d != 64 && d != 128) || page_size < 16 || page_size > 1024 || page_size % 16 != 0) return 0;
  return static_cast<size_t>(page_size) * d * 9 / 8;
}

kvz_status kvz_compact_int4(const void* K, const void* V, int64_t B, int64_t n_c, int d, const int32_t* idx,
                            const int32_t* counts, const int64_t* offsets, void* cache, int64_t n_pages,
                            int page_size, const int32_t* pages, int64_t max_pages, int32_t* d_status,
                            cudaStream_t stream) {
  if (K == nullptr || V == nullptr || idx == nullptr || counts == nullptr || offsets == nullptr)
    return KVZ_ERR_INVALID_ARG;
  kvz::Pages4 pg;
  const kvz_status st = check_pages(cache, n_pages, page_size, pages, max_pages, B, d, &pg);
  if (st != KVZ_OK) return st;
  if (n_c < 1 || n_c > 0x7FFFFFFF) return KVZ_ERR_INVALID_ARG;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(idx, 4) || !aligned(counts, 4) || !aligned(offsets, 8))
    return KVZ_ERR_ALIGNMENT;
  return kvz::launch_compact_int4(K, V, B, n_c, d, idx, counts, offsets, pg, d_status, stream) == cudaSuccess
             ? KVZ_OK
             : KVZ_ERR_CUDA;
}

kvz_status kvz_expand_int4(const void* cache, int64_t n_pages, int page_size, const int32_t* pages, int64_t max_pages,
                           const int32_t* counts, const int32_t* first, const int64_t* offsets, int64_t B, int d,
                           void* K_out, void* V_out, int64_t n_rows, int32_t* d_status, cudaStream_t stream) {
  if (counts == nullptr || offsets == nullptr) return KVZ_ERR_INVALID_ARG;
  kvz::Pages4 pg;
  const kvz_status st = check_pages(cache, n_pages, page_size, pages, max_pages, B, d, &pg);
  if (st != KVZ_OK) return st;
  if (n_rows < 0 || (n_rows > 0 && (K_out == nullptr || V_out == nullptr))) return KVZ_ERR_INVALID_ARG;
  if (n_rows > 0 && K_out == V_out) return KVZ_ERR_INVALID_ARG;
  if (!aligned(K_out, 16) || !aligned(V_out, 16) || !aligned(counts, 4) || !aligned(offsets, 8) ||
      (first != nullptr && !aligned(first, 4)))
    return KVZ_ERR_ALIGNMENT;
  return kvz::launch_expand_int4(pg, counts, first, offsets, B, d, K_out, V_out, n_rows, d_status, stream) ==
                 cudaSuccess
             ? KVZ_OK
             : KVZ_ERR_CUDA;
}

kvz_status kvz_append_int4(const void* k, int64_t k_sb, int64_t k_st, const void* v, int64_t v_sb, int64_t v_st,
                           const void* q, int64_t q_sb, int64_t q_sg, int64_t q_st, void* q_out, int64_t B, int G,
                           int64_t T, int d, const int32_t* positions, int64_t pos_sb, const float* table,
                           int64_t n_pos, int rot, int interleaved, void* cache, int64_t n_pages, int page_size,
                           const int32_t* pages, int64_t max_pages, const int32_t* counts, const int32_t* n_new,
                           int32_t* counts_out, int32_t* d_status, cudaStream_t stream) {
  if (k == nullptr || v == nullptr || counts == nullptr) return KVZ_ERR_INVALID_ARG;
  if ((q == nullptr) != (q_out == nullptr)) return KVZ_ERR_INVALID_ARG;
  kvz::Append4Args a{};
  kvz_status st = check_pages(cache, n_pages, page_size, pages, max_pages, B, d, &a.pg);
  if (st != KVZ_OK) return st;
  if (T < 1 || T > kMaxCacheRows || (q != nullptr && (G < 1 || G > 65535))) return KVZ_ERR_INVALID_ARG;
  // rows, and the warps that take them, are numbered in 32 bits
  if (B * (T + 2) > (int64_t(1) << 28) || (q != nullptr && B * G > 0x7FFFFFFF / T)) return KVZ_ERR_INVALID_ARG;
  if (positions != nullptr) {
    st = check_rotation(positions, pos_sb, table, n_pos, rot, d, interleaved, 0, &a.rot);
    if (st != KVZ_OK) return st;
  } else if (table != nullptr) {
    return KVZ_ERR_INVALID_ARG;
  }
  for (int64_t s : {k_sb, k_st, v_sb, v_st})
    if (!stride_ok(s)) return KVZ_ERR_ALIGNMENT;
  if (q != nullptr && (!stride_ok(q_sb) || !stride_ok(q_sg) || !stride_ok(q_st))) return KVZ_ERR_ALIGNMENT;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(q, 16) || !aligned(q_out, 16) || !aligned(counts, 4) ||
      !aligned(n_new, 4) || !aligned(counts_out, 4))
    return KVZ_ERR_ALIGNMENT;
  // every warp of a head reads its old count, its new rows' number and their positions
  if (counts_out != nullptr && (counts_out == counts || counts_out == n_new || counts_out == positions))
    return KVZ_ERR_INVALID_ARG;
  a.k = static_cast<const uint16_t*>(k), a.k_sb = k_sb, a.k_st = k_st;
  a.v = static_cast<const uint16_t*>(v), a.v_sb = v_sb, a.v_st = v_st;
  a.q = static_cast<const uint16_t*>(q), a.q_sb = q_sb, a.q_sg = q_sg, a.q_st = q_st;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.B = B, a.T = T, a.G = q != nullptr ? G : 1;
  a.counts = counts, a.n_new = n_new, a.counts_out = counts_out;
  a.status = d_status;
  return kvz::launch_append_int4(d, a, stream) == cudaSuccess ? KVZ_OK : KVZ_ERR_CUDA;
}

size_t kvz_decode_int4_workspace_size(int64_t B, int G, int64_t rows, int d) {
  if (B < 1 || B > 65535 || G < 1 || G > kvz::kDecGMax || (d != 64 && d != 128) || rows < 1) return 0;
  if (kvz::decode4_form(B, rows).cluster > 0) return 0;
  const size_t w = kvz::kD4Workers;
  return up256(w * sizeof(int4)) + up256(2 * w * 8 * sizeof(float2)) + up256(2 * w * G * d * sizeof(float));
}

kvz_status kvz_decode_int4(const void* q, const void* cache, int64_t n_pages, int page_size, const int32_t* pages,
                           int64_t max_pages, const int32_t* counts, int64_t B, int G, int d, float scale, float* out,
                           float* lse2, void* workspace, size_t workspace_bytes, int32_t* d_status,
                           cudaStream_t stream) {
  return decode_int4(q, cache, n_pages, page_size, pages, max_pages, counts, B, G, d, scale, out, lse2, workspace,
                     workspace_bytes, 0, -1, -1, 16, d_status, stream);
}

kvz_status kvz_testing_decode_int4_withhold(const void* q, const void* cache, int64_t n_pages, int page_size,
                                            const int32_t* pages, int64_t max_pages, const int32_t* counts, int64_t B,
                                            int G, int d, float scale, float* out, float* lse2, void* workspace,
                                            size_t workspace_bytes, int64_t wait_ns, int64_t hold_head,
                                            int64_t hold_cta, int max_cluster, int32_t* d_status,
                                            cudaStream_t stream) {
  if (wait_ns < 1000 || wait_ns > 1000000000 || hold_head < -1 || hold_head >= B || hold_cta < -1)
    return KVZ_ERR_INVALID_ARG;
  if (max_cluster < 1 || max_cluster > 16 || (max_cluster & (max_cluster - 1)) != 0) return KVZ_ERR_INVALID_ARG;
  return decode_int4(q, cache, n_pages, page_size, pages, max_pages, counts, B, G, d, scale, out, lse2, workspace,
                     workspace_bytes, static_cast<uint64_t>(wait_ns), hold_head, hold_cta, max_cluster, d_status, stream);
}

}  // extern "C"
