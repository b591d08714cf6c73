// The paged 4-bit key/value cache: layout helpers and the launchers of its
// kernels (write, read, attention, eviction). Format of include/vlm.h: a page
// of one key head holds 64 tokens as
//   key codes [64][D / 2] | value codes [64][D / 2] | key scales [64][D / 16] | value scales [64][D / 16]
// with E2M1 codes (the even column in the low nibble) and E4M3 scales of 16
// values, so a token costs 9/8 byte per column and head instead of 4.
#pragma once

#include "nvfp4.cuh"
#include "text_attention.cuh"

namespace vlm {

constexpr int kKv4Page = VLM_KV4_PAGE;  // tokens per page
static_assert(kKv4Page == 64, "the kernels split a page into four slices of 16 tokens");

template <int D>
struct Kv4Layout {
  static constexpr int kCodeRow = D / 2;   // bytes of codes per token
  static constexpr int kScaleRow = D / 16;  // bytes of scales per token
  static constexpr int kV = kKv4Page * kCodeRow;
  static constexpr int kKs = 2 * kV;
  static constexpr int kVs = kKs + kKv4Page * kScaleRow;
  static constexpr int kBytes = kVs + kKv4Page * kScaleRow;  // of one head's page
};

inline int64_t kv4_head_bytes(int head_dim) { return static_cast<int64_t>(kKv4Page) * (head_dim + head_dim / 8); }

// A cache and the tables of a batch of sequences (device pointers).
struct Kv4 {
  uint8_t* pages;
  int64_t n_pages;
  int kv_heads;
  int n_seqs;
  int max_pages;          // entries per row of table
  const int32_t* table;   // [n_seqs, max_pages]
  const int32_t* lens;    // [n_seqs]
  float k_sg, v_sg;
};

// The page of entry `e` of sequence s; a table entry that names no page is
// recorded in the status word and replaced by page 0, so the access stays
// inside the pool.
__device__ __forceinline__ int64_t kv4_page(const Kv4& c, int s, int e, int32_t* status) {
  const int32_t p = __ldg(c.table + static_cast<int64_t>(s) * c.max_pages + e);
  if (static_cast<uint32_t>(p) < static_cast<uint64_t>(c.n_pages)) return p;
  set_status(status, VLM_ERR_BAD_PAGE);
  return 0;
}
// Tokens of sequence s, held to the table's room.
__device__ __forceinline__ int kv4_len(const Kv4& c, int s, int32_t* status) {
  const int n = __ldg(c.lens + s);
  if (n >= 0 && n <= c.max_pages * kKv4Page) return n;
  set_status(status, VLM_ERR_BAD_PAGE);
  return n < 0 ? 0 : c.max_pages * kKv4Page;
}

// dtype: VLM_DTYPE_BF16 or VLM_DTYPE_F16. cu_new may be null (one new token per sequence).
int launch_kv4_append(const Kv4& c, int head_dim, const int32_t* cu_new, int64_t n_new, int dtype, const void* k,
                      int64_t k_stride, const void* v, int64_t v_stride, int32_t* status, cudaStream_t s);
int launch_kv4_read(const Kv4& c, int head_dim, const int32_t* cu, int64_t n_rows, int dtype, void* k, void* v,
                    int32_t* status, cudaStream_t s);
size_t kv4_attention_workspace(int n_seqs, int heads, int kv_heads, int head_dim, int q_len);
int launch_kv4_attention(const Kv4& c, int head_dim, int heads, int q_len, int dtype, const void* q, int64_t q_stride,
                         float scale, void* out, float* weights, void* ws, int32_t* status, cudaStream_t s);
size_t kv4_evict_workspace(int64_t n_pages, int n_seqs, int kv_heads, int budget);
int launch_kv4_evict(const Kv4& c, int head_dim, const float* weights, int budget, int sinks, int recent,
                     const int32_t* to_table, int to_max_pages, int32_t* to_lens, float* to_weights, int32_t* kept,
                     void* ws, int32_t* status, cudaStream_t s);

}  // namespace vlm
