// C-ABI layer of the text side's attention: prompt attention and the paged
// 4-bit cache (declared in include/vlm.h). Arguments are checked here, before
// anything is launched; what only the device knows (lengths, page tables) is
// checked in the kernels.
#include <climits>
#include <cmath>

#include "kv4.cuh"
#include "text_attention.cuh"

using namespace vlm;

namespace {

inline cudaStream_t as_stream(void* s) { return static_cast<cudaStream_t>(s); }
inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + nb && y < x + na;
}

#define VLM_TRY(expr)             \
  do {                            \
    const int rc_ = (expr);       \
    if (rc_ != VLM_OK) return rc_; \
  } while (0)

int check_heads(int heads, int kv_heads, int head_dim) {
  if (heads <= 0 || kv_heads <= 0) return VLM_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return VLM_ERR_UNSUPPORTED;
  if (heads % kv_heads != 0 || heads / kv_heads > 128 || heads > 65535) return VLM_ERR_UNSUPPORTED;
  return VLM_OK;
}

int check_rows(int dtype, const void* p, int64_t stride, int64_t width) {
  if (dtype != VLM_DTYPE_BF16 && dtype != VLM_DTYPE_F16) return VLM_ERR_UNSUPPORTED;
  if (p == nullptr || misaligned(p, 16)) return VLM_ERR_INVALID_ARG;
  if (stride < width) return VLM_ERR_BAD_SHAPE;
  if (stride % 8 != 0 || stride > (1LL << 38)) return VLM_ERR_UNSUPPORTED;
  return VLM_OK;
}

// Entries of a page table: places are 32-bit in the kernels, which step over them by up
// to 4,096 at a time, so the last place keeps that much room.
constexpr int kMaxPages = (INT_MAX - 8192) / kKv4Page;
constexpr int kMaxEntries = INT_MAX - 2 * 65536;  // and room for two more per sequence

// The cache and its tables as the kernels take them.
int make_kv4(const vlm_kv4_cache* c, const int32_t* table, int max_pages, int n_seqs, const int32_t* lens, Kv4* out) {
  if (c == nullptr || c->d_pages == nullptr || table == nullptr) return VLM_ERR_INVALID_ARG;
  if (misaligned(c->d_pages, 16) || misaligned(table, 4) || misaligned(lens, 4)) return VLM_ERR_INVALID_ARG;
  if (!(c->k_sg > 0.f) || !(c->v_sg > 0.f) || !std::isfinite(c->k_sg) || !std::isfinite(c->v_sg))
    return VLM_ERR_INVALID_ARG;
  VLM_TRY(check_heads(c->kv_heads, c->kv_heads, c->head_dim));
  if (c->n_pages <= 0 || c->n_pages > INT_MAX || n_seqs <= 0 || n_seqs > 65535 || max_pages <= 0 ||
      max_pages > kMaxPages || static_cast<int64_t>(max_pages) * n_seqs > kMaxEntries)
    return VLM_ERR_BAD_SHAPE;
  out->pages = static_cast<uint8_t*>(c->d_pages);
  out->n_pages = c->n_pages;
  out->kv_heads = c->kv_heads;
  out->n_seqs = n_seqs;
  out->max_pages = max_pages;
  out->table = table;
  out->lens = lens;
  out->k_sg = c->k_sg;
  out->v_sg = c->v_sg;
  return VLM_OK;
}

}  // namespace

extern "C" {

int vlm_prompt_attention(int dtype, int heads, int kv_heads, int head_dim, const int32_t* q_lens,
                         const int32_t* kv_lens, int n_seqs, const void* d_q, int64_t q_stride, const void* d_k,
                         int64_t k_stride, const void* d_v, int64_t v_stride, float scale, void* d_out,
                         int64_t out_stride, int32_t* d_status, void* stream) {
  if (q_lens == nullptr || kv_lens == nullptr || n_seqs <= 0) return VLM_ERR_INVALID_ARG;
  VLM_TRY(check_heads(heads, kv_heads, head_dim));
  if (!(scale > 0.f) || !std::isfinite(scale)) return VLM_ERR_INVALID_ARG;
  int64_t tq = 0, tk = 0;
  for (int i = 0; i < n_seqs; ++i) {
    if (q_lens[i] < 0 || kv_lens[i] < 0) return VLM_ERR_BAD_SHAPE;
    tq += q_lens[i];
    tk += kv_lens[i];
  }
  // places are 32-bit in the kernel, with room for a tile behind the last
  if (tq > INT_MAX - 512 || tk > INT_MAX - 512) return VLM_ERR_BAD_SHAPE;
  if (tq == 0) return VLM_OK;
  VLM_TRY(check_rows(dtype, d_q, q_stride, static_cast<int64_t>(heads) * head_dim));
  VLM_TRY(check_rows(dtype, d_out, out_stride, static_cast<int64_t>(heads) * head_dim));
  if (tk > 0) {
    VLM_TRY(check_rows(dtype, d_k, k_stride, static_cast<int64_t>(kv_heads) * head_dim));
    VLM_TRY(check_rows(dtype, d_v, v_stride, static_cast<int64_t>(kv_heads) * head_dim));
  }
  const PromptAttn p{dtype,    heads, kv_heads, head_dim, q_lens, kv_lens, n_seqs, d_q,        d_k,     d_v,
                     q_stride, k_stride, v_stride, scale,  d_out,  out_stride, d_status};
  try {
    return launch_prompt_attention(p, as_stream(stream));
  } catch (...) {  // host memory for the order of the sequences
    return VLM_ERR_CUDA;
  }
}

size_t vlm_kv4_page_bytes(int kv_heads, int head_dim) {
  if (check_heads(kv_heads, kv_heads, head_dim) != VLM_OK) return 0;
  return static_cast<size_t>(kv_heads) * kv4_head_bytes(head_dim);
}

int vlm_kv4_append(const vlm_kv4_cache* cache, const int32_t* d_table, int max_pages, int n_seqs,
                   const int32_t* d_lens, const int32_t* d_cu_new, int64_t n_new, int dtype, const void* d_k,
                   int64_t k_stride, const void* d_v, int64_t v_stride, int32_t* d_status, void* stream) {
  Kv4 c;
  VLM_TRY(make_kv4(cache, d_table, max_pages, n_seqs, d_lens, &c));
  if (misaligned(d_cu_new, 4)) return VLM_ERR_INVALID_ARG;
  if (n_new < 0 || n_new > INT_MAX || (d_cu_new == nullptr && n_new != n_seqs)) return VLM_ERR_BAD_SHAPE;
  if (n_new == 0) return VLM_OK;
  const int64_t width = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
  VLM_TRY(check_rows(dtype, d_k, k_stride, width));
  VLM_TRY(check_rows(dtype, d_v, v_stride, width));
  return launch_kv4_append(c, cache->head_dim, d_cu_new, n_new, dtype, d_k, k_stride, d_v, v_stride, d_status,
                           as_stream(stream));
}

int vlm_kv4_read(const vlm_kv4_cache* cache, const int32_t* d_table, int max_pages, int n_seqs,
                 const int32_t* d_start, const int32_t* d_cu, int64_t n_rows, int dtype, void* d_k, void* d_v,
                 int32_t* d_status, void* stream) {
  Kv4 c;
  VLM_TRY(make_kv4(cache, d_table, max_pages, n_seqs, d_start, &c));
  if (misaligned(d_cu, 4)) return VLM_ERR_INVALID_ARG;
  if (n_rows < 0 || n_rows > INT_MAX || (d_cu == nullptr && n_rows != n_seqs)) return VLM_ERR_BAD_SHAPE;
  if (n_rows == 0) return VLM_OK;
  const int64_t width = static_cast<int64_t>(cache->kv_heads) * cache->head_dim;
  VLM_TRY(check_rows(dtype, d_k, width, width));
  VLM_TRY(check_rows(dtype, d_v, width, width));
  return launch_kv4_read(c, cache->head_dim, d_cu, n_rows, dtype, d_k, d_v, d_status, as_stream(stream));
}

size_t vlm_kv4_attention_workspace_size(int n_seqs, int heads, int kv_heads, int head_dim, int q_len) {
  if (check_heads(heads, kv_heads, head_dim) != VLM_OK || n_seqs <= 0 || q_len <= 0) return 0;
  return kv4_attention_workspace(n_seqs, heads, kv_heads, head_dim, q_len);
}

int vlm_kv4_attention(const vlm_kv4_cache* cache, const int32_t* d_table, int max_pages, int n_seqs,
                      const int32_t* d_lens, int dtype, int heads, int q_len, const void* d_q, int64_t q_stride,
                      float scale, void* d_out, float* d_weights, void* d_workspace, size_t ws_bytes,
                      int32_t* d_status, void* stream) {
  Kv4 c;
  VLM_TRY(make_kv4(cache, d_table, max_pages, n_seqs, d_lens, &c));
  if (d_lens == nullptr || d_workspace == nullptr || misaligned(d_workspace, 256) || misaligned(d_weights, 4))
    return VLM_ERR_INVALID_ARG;
  VLM_TRY(check_heads(heads, cache->kv_heads, cache->head_dim));
  if (!(scale > 0.f) || !std::isfinite(scale)) return VLM_ERR_INVALID_ARG;
  if (q_len <= 0 || static_cast<int64_t>(q_len) * (heads / cache->kv_heads) > 65535 ||
      static_cast<int64_t>(q_len) * n_seqs > INT_MAX)
    return VLM_ERR_BAD_SHAPE;
  const int64_t width = static_cast<int64_t>(heads) * cache->head_dim;
  VLM_TRY(check_rows(dtype, d_q, q_stride, width));
  VLM_TRY(check_rows(dtype, d_out, width, width));
  if (ws_bytes < vlm_kv4_attention_workspace_size(n_seqs, heads, cache->kv_heads, cache->head_dim, q_len))
    return VLM_ERR_WORKSPACE;
  return launch_kv4_attention(c, cache->head_dim, heads, q_len, dtype, d_q, q_stride, scale, d_out, d_weights,
                              d_workspace, d_status, as_stream(stream));
}

size_t vlm_kv4_evict_workspace_size(int64_t n_pages, int n_seqs, int kv_heads, int budget) {
  if (n_pages <= 0 || n_pages > INT_MAX || n_seqs <= 0 || kv_heads <= 0 || budget <= 0) return 0;
  return kv4_evict_workspace(n_pages, n_seqs, kv_heads, budget);
}

int vlm_kv4_evict(const vlm_kv4_cache* cache, const int32_t* d_table, int max_pages, int n_seqs,
                  const int32_t* d_lens, const float* d_weights, int budget, int sinks, int recent,
                  const int32_t* d_to_table, int to_max_pages, int32_t* d_to_lens, float* d_to_weights,
                  int32_t* d_kept, void* d_workspace, size_t ws_bytes, int32_t* d_status, void* stream) {
  Kv4 c;
  VLM_TRY(make_kv4(cache, d_table, max_pages, n_seqs, d_lens, &c));
  if (d_lens == nullptr || d_weights == nullptr || d_to_table == nullptr || d_to_lens == nullptr ||
      d_to_weights == nullptr || d_workspace == nullptr)
    return VLM_ERR_INVALID_ARG;
  if (misaligned(d_weights, 4) || misaligned(d_to_table, 4) || misaligned(d_to_lens, 4) ||
      misaligned(d_to_weights, 4) || misaligned(d_kept, 4) || misaligned(d_workspace, 256))
    return VLM_ERR_INVALID_ARG;
  if (budget <= 0 || sinks < 0 || recent < 0 || static_cast<int64_t>(sinks) + recent > budget)
    return VLM_ERR_BAD_SHAPE;
  if (to_max_pages <= 0 || to_max_pages > kMaxPages || budget > to_max_pages * kKv4Page ||
      static_cast<int64_t>(to_max_pages) * n_seqs > INT_MAX)
    return VLM_ERR_BAD_SHAPE;
  // results over what other CTAs still read, or over one another
  const size_t units = static_cast<size_t>(n_seqs) * cache->kv_heads;
  const size_t need = vlm_kv4_evict_workspace_size(cache->n_pages, n_seqs, cache->kv_heads, budget);
  struct Span {
    const void* p;
    size_t n;
  };
  const Span results[] = {{d_to_lens, n_seqs * 4ull},
                          {d_to_weights, units * to_max_pages * kKv4Page * 4},
                          {d_kept, d_kept == nullptr ? 0 : units * budget * 4}};
  const Span others[] = {{d_lens, n_seqs * 4ull},
                         {d_weights, units * max_pages * kKv4Page * 4},
                         {d_table, static_cast<size_t>(n_seqs) * max_pages * 4},
                         {d_to_table, static_cast<size_t>(n_seqs) * to_max_pages * 4},
                         {c.pages, static_cast<size_t>(c.n_pages) * cache->kv_heads * kv4_head_bytes(cache->head_dim)},
                         {d_workspace, need},
                         {d_status, 4}};
  for (int i = 0; i < 3; ++i) {
    if (results[i].n == 0) continue;
    for (const Span& o : others)
      if (overlap(results[i].p, results[i].n, o.p, o.n)) return VLM_ERR_INVALID_ARG;
    for (int j = 0; j < i; ++j)
      if (overlap(results[i].p, results[i].n, results[j].p, results[j].n)) return VLM_ERR_INVALID_ARG;
  }
  if (ws_bytes < need) return VLM_ERR_WORKSPACE;
  return launch_kv4_evict(c, cache->head_dim, d_weights, budget, sinks, recent, d_to_table, to_max_pages, d_to_lens,
                          d_to_weights, d_kept, d_workspace, d_status, as_stream(stream));
}

}  // extern "C"
