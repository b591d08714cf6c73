// Eviction from the paged 4-bit cache by summed attention weight: per
// (sequence, key head) the `budget` places to keep -- the first `sinks`, the
// last `recent`, and of the others those with the largest weights, the lower
// place first among equals -- move in order of place to fresh pages, bit for
// bit, with their weights.
//
// kv4_select_kernel, one CTA per (sequence, key head): the weight of the last
//   place that still fits is found by a radix select over the weights' bits
//   (four passes of eight bits, a histogram in shared memory each), then one
//   ordered pass writes the kept places. The weights are 4 bytes per place and
//   are read five times, from L2 after the first.
// kv4_move_kernel, one CTA per destination page of a head: 16-byte copies of
//   the kept rows, 9/8 byte per column in and out: bound by HBM.
// Fresh pages have to be fresh: one more CTA per sequence marks its source and
// destination pages in two bit sets of the pool and compares them; on a
// destination page that is also a source page, or is named twice, no page is
// written and the status word says so. Marking before comparing lets the CTAs
// run in any order: of two that meet, the later one sees the earlier's mark.
#include <algorithm>

#include "kv4.cuh"

namespace vlm {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kPer = 4;  // places per thread and step of the ordered pass
constexpr int kMoveThreads = 128;

struct EvictArgs {
  Kv4 c;
  const float* weights;  // [n_seqs, kv_heads, max_pages * 64]
  int budget, sinks, recent;
  const int32_t* to_table;
  int to_max_pages;
  int32_t* to_lens;
  float* to_weights;  // [n_seqs, kv_heads, to_max_pages * 64]
  int32_t* kept;      // [n_seqs, kv_heads, budget]
  uint32_t *src_bits, *dst_bits;
  int32_t* clash;
  int32_t* status;
};

// Weights as unsigned keys of the same order; -0 is 0, a NaN is below all.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ void mark_pages(const EvictArgs& a, int s, int n, int n_new) {
  const int src = (n + kKv4Page - 1) / kKv4Page, dst = (n_new + kKv4Page - 1) / kKv4Page;
  bool bad = false;
  for (int e = threadIdx.x; e < src + dst; e += kSelThreads) {
    const bool is_dst = e >= src;
    const int32_t p = is_dst ? __ldg(a.to_table + static_cast<int64_t>(s) * a.to_max_pages + e - src)
                             : __ldg(a.c.table + static_cast<int64_t>(s) * a.c.max_pages + e);
    if (static_cast<uint32_t>(p) >= static_cast<uint64_t>(a.c.n_pages)) {
      bad = true;
      continue;
    }
    const uint32_t bit = 1u << (p & 31);
    const uint32_t old = atomicOr((is_dst ? a.dst_bits : a.src_bits) + (p >> 5), bit);
    __threadfence();
    const uint32_t other = atomicOr((is_dst ? a.src_bits : a.dst_bits) + (p >> 5), 0u);
    if ((other & bit) != 0 || (is_dst && (old & bit) != 0)) bad = true;
  }
  if (bad) {
    atomicExch(a.clash, 1);
    set_status(a.status, VLM_ERR_BAD_PAGE);
  }
}

__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(const EvictArgs a) {
  __shared__ uint32_t hist[256];
  __shared__ uint32_t found[2];  // the digit, and how many are still wanted below it
  __shared__ uint32_t warp_sum[kSelWarps];
  griddep_wait();
  griddep_launch_dependents();
  const int s = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
  const int n = kv4_len(a.c, s, h == 0 && tid == 0 ? a.status : nullptr);
  const int n_new = min(n, a.budget);
  if (h == a.c.kv_heads) {
    mark_pages(a, s, n, n_new);
    if (tid == 0) a.to_lens[s] = n_new;
    return;
  }
  const int64_t unit = static_cast<int64_t>(s) * a.c.kv_heads + h;
  const float* w = a.weights + unit * a.c.max_pages * kKv4Page;
  float* to_w = a.to_weights + unit * a.to_max_pages * kKv4Page;
  int32_t* kept = a.kept + unit * a.budget;
  for (int j = n_new + tid; j < a.to_max_pages * kKv4Page; j += kSelThreads) to_w[j] = 0.0f;
  for (int j = n_new + tid; j < a.budget; j += kSelThreads) kept[j] = -1;
  if (n <= a.budget) {
    for (int j = tid; j < n; j += kSelThreads) {
      kept[j] = j;
      to_w[j] = w[j];
    }
    return;
  }
  const int lo = a.sinks, hi = n - a.recent;  // the places that compete; more of them than are wanted
  uint32_t want = static_cast<uint32_t>(a.budget - a.sinks - a.recent);
  uint32_t prefix = 0;  // the digits found so far
  if (want > 0) {
#pragma unroll 1
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      const uint32_t mask = shift == 24 ? 0u : 0xFFFFFFFFu << (shift + 8);
#pragma unroll 4
      for (int j = lo + tid; j < hi; j += kSelThreads) {
        const uint32_t k = key_of(__ldg(w + j));
        if ((k & mask) == prefix) atomicAdd(&hist[(k >> shift) & 255u], 1u);
      }
      __syncthreads();
      // the largest digit with at least `want` keys at or above it
      if (tid < 32) {
        uint32_t cnt[8], sum = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          cnt[i] = hist[255 - (tid * 8 + i)];
          sum += cnt[i];
        }
        uint32_t inc = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
          if (tid >= o) inc += v;
        }
        uint32_t above = inc - sum;
        if (above < want && want <= inc) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (above < want && want <= above + cnt[i]) {
              found[0] = 255 - (tid * 8 + i);
              found[1] = want - above;
            }
            above += cnt[i];
          }
        }
      }
      __syncthreads();
      prefix |= found[0] << shift;
      want = found[1];
      __syncthreads();
    }
  }
  // `prefix` is the smallest kept key, `want` of its places are kept, the first ones.
  // With nothing wanted no key counts (want 0 and nothing above the top key).
  const uint32_t least = a.budget > a.sinks + a.recent ? prefix : 0xFFFFFFFFu;
  uint32_t base = 0;  // places above in the low half's count, equal ones in `eq`
  uint32_t base_eq = 0;
  for (int first = 0; first < n; first += kSelThreads * kPer) {
    const int j0 = first + tid * kPer;
    float x[kPer];
    uint32_t take = 0, equal = 0;  // bit masks over the thread's places
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int j = j0 + i;
      x[i] = j < n ? __ldg(w + j) : 0.0f;
      if (j < n) {
        if (j < lo || j >= hi) {
          take |= 1u << i;
        } else {
          const uint32_t k = key_of(x[i]);
          if (k > least) take |= 1u << i;
          if (k == least) equal |= 1u << i;
        }
      }
    }
    // both counts in one word: at most 4,096 each per step
    const uint32_t mine = __popc(take) | (__popc(equal) << 16);
    uint32_t inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
      if ((tid & 31) >= o) inc += v;
    }
    if ((tid & 31) == 31) warp_sum[tid >> 5] = inc;
    __syncthreads();
    uint32_t before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kSelWarps; ++i) {
      const uint32_t v = warp_sum[i];
      if (i < (tid >> 5)) before += v;
      total += v;
    }
    const uint32_t excl = before + inc - mine;
    uint32_t taken = base + (excl & 0xFFFFu), eq = base_eq + (excl >> 16);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool is_eq = (equal >> i) & 1;
      if (((take >> i) & 1) || (is_eq && eq < want)) {
        const uint32_t at = taken + min(eq, want);
        if (at < static_cast<uint32_t>(n_new)) {
          kept[at] = j0 + i;
          to_w[at] = x[i];
        }
      }
      taken += (take >> i) & 1;
      eq += is_eq;
    }
    base += total & 0xFFFFu;
    base_eq += total >> 16;
    __syncthreads();
  }
}

template <int D>
__global__ void __launch_bounds__(kMoveThreads) kv4_move_kernel(const EvictArgs a) {
  using L = Kv4Layout<D>;
  __shared__ int64_t from[kKv4Page];  // byte offset of the row's page of this head
  __shared__ int from_row[kKv4Page];
  griddep_wait();
  griddep_launch_dependents();
  if (*a.clash != 0) return;
  const int s = blockIdx.z, h = blockIdx.y, e = blockIdx.x, tid = threadIdx.x;
  const int n = kv4_len(a.c, s, nullptr);
  const int rows = min(min(n, a.budget) - e * kKv4Page, kKv4Page);
  if (rows <= 0) return;
  const int64_t to = __ldg(a.to_table + static_cast<int64_t>(s) * a.to_max_pages + e);
  if (tid < rows) {
    const int j = a.kept[(static_cast<int64_t>(s) * a.c.kv_heads + h) * a.budget + e * kKv4Page + tid];
    from[tid] = (kv4_page(a.c, s, j / kKv4Page, a.status) * a.c.kv_heads + h) * L::kBytes;
    from_row[tid] = j % kKv4Page;
  }
  __syncthreads();
  uint8_t* dst = a.c.pages + (to * a.c.kv_heads + h) * L::kBytes;
  constexpr int kCh = L::kCodeRow / 16;  // 16-byte chunks of a code row
#pragma unroll 4
  for (int i = tid; i < rows * kCh * 2; i += kMoveThreads) {
    const int part = i >= rows * kCh, x = i - part * rows * kCh, r = x / kCh, ch = x % kCh;
    const int64_t base = part * L::kV + ch * 16;
    *reinterpret_cast<uint4*>(dst + base + r * L::kCodeRow) =
        *reinterpret_cast<const uint4*>(a.c.pages + from[r] + base + from_row[r] * L::kCodeRow);
  }
  for (int i = tid; i < rows * 2; i += kMoveThreads) {
    const int part = i >= rows, r = i - part * rows;
    const int64_t base = L::kKs + part * (L::kVs - L::kKs);
    const uint8_t* src = a.c.pages + from[r] + base + from_row[r] * L::kScaleRow;
    if constexpr (D == 128)
      *reinterpret_cast<uint2*>(dst + base + r * L::kScaleRow) = *reinterpret_cast<const uint2*>(src);
    else
      *reinterpret_cast<uint32_t*>(dst + base + r * L::kScaleRow) = *reinterpret_cast<const uint32_t*>(src);
  }
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t kv4_evict_workspace(int64_t n_pages, int n_seqs, int kv_heads, int budget) {
  return 256 + 2 * up(static_cast<size_t>((n_pages + 31) / 32) * 4) +
         up(static_cast<size_t>(n_seqs) * kv_heads * budget * 4);
}

int launch_kv4_evict(const Kv4& c, int head_dim, const float* weights, int budget, int sinks, int recent,
                     const int32_t* to_table, int to_max_pages, int32_t* to_lens, float* to_weights, int32_t* kept,
                     void* ws, int32_t* status, cudaStream_t s) {
  const size_t bits = up(static_cast<size_t>((c.n_pages + 31) / 32) * 4);
  uint8_t* w = static_cast<uint8_t*>(ws);
  EvictArgs a{c, weights, budget, sinks, recent, to_table, to_max_pages, to_lens, to_weights, kept, nullptr, nullptr,
              nullptr, status};
  a.clash = reinterpret_cast<int32_t*>(w);
  a.src_bits = reinterpret_cast<uint32_t*>(w + 256);
  a.dst_bits = reinterpret_cast<uint32_t*>(w + 256 + bits);
  if (kept == nullptr) a.kept = reinterpret_cast<int32_t*>(w + 256 + 2 * bits);
  if (cudaMemsetAsync(w, 0, 256 + 2 * bits, s) != cudaSuccess) return VLM_ERR_CUDA;
  launch_begin(KC_KV4_EVICT, s);
  cudaError_t e = launch_pdl(kv4_select_kernel, dim3(c.kv_heads + 1, c.n_seqs), dim3(kSelThreads), 0, s, a);
  const dim3 grid((budget + kKv4Page - 1) / kKv4Page, c.kv_heads, c.n_seqs);
  if (e == cudaSuccess)
    e = head_dim == 128 ? launch_pdl(kv4_move_kernel<128>, grid, dim3(kMoveThreads), 0, s, a)
                        : launch_pdl(kv4_move_kernel<64>, grid, dim3(kMoveThreads), 0, s, a);
  launch_end(KC_KV4_EVICT, s);
  note_extra_launches(1);
  return e == cudaSuccess ? VLM_OK : VLM_ERR_CUDA;
}

}  // namespace vlm
