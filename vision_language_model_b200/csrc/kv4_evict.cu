// Eviction from the paged 4-bit cache by summed attention weight: per
// (sequence, key head) the `budget` places to keep -- the first `sinks`, the
// last `recent`, and of the others those with the largest weights, the lower
// place first among equals -- move in order of place to fresh pages, bit for
// bit, with their weights.
//
// kv4_select_kernel, one CTA per (sequence, key head): the weight of the last
//   place that still fits is found by a radix select over the weights' bits (11,
//   11 and 10), then one ordered pass writes the kept places. Up to 16,384
//   places the weights stay in registers and are read once. Softmax weights
//   share a few exponents, and what bounds the count of a digit is atomics on
//   one address: hence digits that reach into the mantissa, four copies of the
//   histogram, and places of weight 0 (many, as a rule) counted by ballots.
//   64 (sequence, head) pairs of up to 16,384 places, cold: 19 us (25 us with
//   four digits of 8 bits, one copy and the weights read again for each).
// kv4_move_kernel, one CTA per destination page of a head: 16-byte copies of
//   the kept rows, 9/8 byte per column in and out: bound by HBM, whose 64-byte
//   pieces a row's two 8-byte scale groups use by an eighth (29,000 scattered
//   rows of 8 heads: 58 MB read for 34, 17 us).
// Fresh pages have to be fresh: one more CTA marks all source and destination
// pages in two bit sets of the pool and compares them; on a destination page
// that is also a source page, or is named twice, no page is written and the
// status word says so. The bit sets lie in shared memory for pools of up to
// 262,144 pages; for larger ones in the workspace, cleared first, with one CTA
// per sequence: marking before comparing lets the CTAs run in any order, of two
// that meet the later one sees the earlier's mark.
#include <algorithm>
#include <type_traits>

#include "kv4.cuh"

namespace vlm {

namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kPer = 4;       // consecutive places per thread and step
constexpr int kCopies = 4;    // of a digit's histogram, side by side
constexpr int kDigits = 2048;
constexpr int kCached = 4;    // steps whose weights a thread keeps in registers
constexpr int kMoveThreads = 128;
constexpr int64_t kSharedPages = 262144;  // pools up to here are marked in shared memory
constexpr uint32_t kZeroKey = 0x80000000u;

struct EvictArgs {
  Kv4 c;
  const float* weights;  // [n_seqs, kv_heads, max_pages * 64]
  int budget, sinks, recent;
  const int32_t* to_table;
  int to_max_pages;
  int32_t* to_lens;
  float* to_weights;  // [n_seqs, kv_heads, to_max_pages * 64]
  int32_t* kept;      // [n_seqs, kv_heads, budget]
  uint32_t *src_bits, *dst_bits;  // null: in shared memory
  int32_t* clash;
  int32_t* status;
};

// Weights as unsigned keys of the same order; -0 is 0, a NaN is below all.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0u;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// Entry e of sequence s: the source pages, then the destination pages.
__device__ __forceinline__ int32_t page_entry(const EvictArgs& a, int s, int e, int src, bool& is_dst) {
  is_dst = e >= src;
  return is_dst ? __ldg(a.to_table + static_cast<int64_t>(s) * a.to_max_pages + e - src)
                : __ldg(a.c.table + static_cast<int64_t>(s) * a.c.max_pages + e);
}

__device__ void mark_shared(const EvictArgs& a, uint32_t* bits) {
  const int words = static_cast<int>((a.c.n_pages + 31) / 32);
  uint32_t* dst_bits = bits + words;
  for (int i = threadIdx.x; i < 2 * words; i += kSelThreads) bits[i] = 0;
  __syncthreads();
  // a warp takes 32 entries of a sequence at a time, so that many are looked up at once
  __shared__ int lens[kSelThreads];
  bool bad = false;
  const int chunks = (a.c.max_pages + a.to_max_pages + 31) / 32;
  for (int s0 = 0; s0 < a.c.n_seqs; s0 += kSelThreads) {
    const int count = min(kSelThreads, a.c.n_seqs - s0);
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < count) {
      const int n = kv4_len(a.c, s0 + threadIdx.x, a.status);
      lens[threadIdx.x] = n;
      a.to_lens[s0 + threadIdx.x] = min(n, a.budget);
    }
    __syncthreads();
#pragma unroll 4
    for (int task = threadIdx.x >> 5; task < count * chunks; task += kSelWarps) {
      const int s = task / chunks, e = (task - s * chunks) * 32 + (threadIdx.x & 31);
      const int n = lens[s], n_new = min(n, a.budget);
      const int src = (n + kKv4Page - 1) / kKv4Page, dst = (n_new + kKv4Page - 1) / kKv4Page;
      if (e >= src + dst) continue;
      bool is_dst;
      const int32_t p = page_entry(a, s0 + s, e, src, is_dst);
      if (static_cast<uint32_t>(p) >= static_cast<uint64_t>(a.c.n_pages)) {
        bad = true;
        continue;
      }
      const uint32_t bit = 1u << (p & 31);
      const uint32_t old = atomicOr((is_dst ? dst_bits : bits) + (p >> 5), bit);
      if (is_dst && (old & bit) != 0) bad = true;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < words; i += kSelThreads) bad |= (bits[i] & dst_bits[i]) != 0;
  const int any = __syncthreads_or(bad);
  if (threadIdx.x == 0) {
    *a.clash = any;
    if (any) set_status(a.status, VLM_ERR_BAD_PAGE);
  }
}

__device__ void mark_global(const EvictArgs& a, int s) {
  const int n = kv4_len(a.c, s, threadIdx.x == 0 ? a.status : nullptr), n_new = min(n, a.budget);
  if (threadIdx.x == 0) a.to_lens[s] = n_new;
  const int src = (n + kKv4Page - 1) / kKv4Page, dst = (n_new + kKv4Page - 1) / kKv4Page;
  bool bad = false;
  for (int e = threadIdx.x; e < src + dst; e += kSelThreads) {
    bool is_dst;
    const int32_t p = page_entry(a, s, e, src, is_dst);
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

// Inclusive sum over the CTA's threads in order; `total` their sum. Two barriers.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t* warp_sum, uint32_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) warp_sum[warp] = v;
  __syncthreads();
  uint32_t w = warp_sum[lane];  // one per warp: kSelWarps is 32
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += u;
  }
  total = __shfl_sync(0xffffffffu, w, 31);
  const uint32_t before = warp == 0 ? 0 : __shfl_sync(0xffffffffu, w, warp - 1);
  __syncthreads();
  return v + before;
}

__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(const EvictArgs a) {
  extern __shared__ __align__(16) uint32_t dyn[];  // the histogram's copies, or the pool's two bit sets
  __shared__ uint32_t warp_sum[kSelWarps];
  __shared__ uint32_t found[2];  // the digit, and how many of its places are still wanted
  static_assert(kSelWarps == 32, "block_scan");
  griddep_wait();
  griddep_launch_dependents();
  const int s = blockIdx.y, h = blockIdx.x, tid = threadIdx.x;
  if (h == a.c.kv_heads) {
    if (a.src_bits != nullptr)
      mark_global(a, s);
    else if (s == 0)
      mark_shared(a, dyn);
    return;
  }
  const int n = kv4_len(a.c, s, nullptr);
  const int n_new = min(n, a.budget);
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
  uint32_t least = 0xFFFFFFFFu;  // the smallest kept key; nothing wanted: above every key
  constexpr int kStep = kSelThreads * kPer;
  const int steps = (n + kStep - 1) / kStep;
  // a thread's places are kPer consecutive ones of every step
  auto load = [&](int step, float (&x)[kPer]) {
    const int j = step * kStep + tid * kPer;
    if (j + kPer <= n) {  // rows of weights are whole pages: 16-byte aligned as long as the array is
      if ((reinterpret_cast<uintptr_t>(w) & 15) == 0) {
        const float4 f = __ldg(reinterpret_cast<const float4*>(w + j));
        x[0] = f.x; x[1] = f.y; x[2] = f.z; x[3] = f.w;
        return;
      }
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) x[i] = j + i < n ? __ldg(w + j + i) : 0.0f;
  };
  // keys, and which places compete (bit kPer step + i), of the first steps
  uint32_t cache[kCached][kPer], competes = 0;
  auto range = [&](int step) {
    const int j = step * kStep + tid * kPer;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) m |= (j + i >= lo && j + i < hi ? 1u : 0u) << i;
    return m;
  };
  {
    float x[kCached][kPer];
#pragma unroll
    for (int c = 0; c < kCached; ++c)
      if (c < steps) load(c, x[c]);
#pragma unroll
    for (int c = 0; c < kCached; ++c) {
      if (c < steps) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) cache[c][i] = key_of(x[c][i]);
        competes |= range(c) << (kPer * c);
      }
    }
  }
  if (want > 0) {
    uint32_t prefix = 0;  // the digits found so far
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digit = pass == 2 ? 1023u : 2047u;
      const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xFFE00000u : 0xFFFFFC00u;
      for (int i = tid; i < kCopies * kDigits / 4; i += kSelThreads) reinterpret_cast<uint4*>(dyn)[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      uint32_t* mine = dyn + tid % kCopies;  // neighbouring lanes count in different copies, in different banks
      uint32_t zeros = 0;
      const bool with_zeros = (kZeroKey & mask) == prefix;
      auto count = [&](uint32_t in, const uint32_t (&k)[kPer]) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
          const bool counts = ((in >> i) & 1) && (k[i] & mask) == prefix;
          if (with_zeros) zeros += __popc(__ballot_sync(0xffffffffu, counts && k[i] == kZeroKey));
          if (counts && k[i] != kZeroKey) atomicAdd(mine + ((k[i] >> shift) & digit) * kCopies, 1u);
        }
      };
#pragma unroll
      for (int c = 0; c < kCached; ++c)
        if (c < steps) count(competes >> (kPer * c), cache[c]);
      for (int c = kCached; c < steps; ++c) {
        float x[kPer];
        uint32_t k[kPer];
        load(c, x);
#pragma unroll
        for (int i = 0; i < kPer; ++i) k[i] = key_of(x[i]);
        count(range(c), k);
      }
      if ((tid & 31) == 0 && zeros > 0) atomicAdd(mine + ((kZeroKey >> shift) & digit) * kCopies, zeros);
      __syncthreads();
      // digits from the top, two per thread: the largest with `want` keys at or above it
      uint32_t cnt[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 c = reinterpret_cast<const uint4*>(dyn)[kDigits - 1 - (2 * tid + i)];
        cnt[i] = c.x + c.y + c.z + c.w;
      }
      uint32_t total;
      const uint32_t inc = block_scan(cnt[0] + cnt[1], warp_sum, total);
      const uint32_t above = inc - cnt[0] - cnt[1];
      if (above < want && want <= inc) {
        const int second = want > above + cnt[0];
        found[0] = kDigits - 1 - (2 * tid + second);
        found[1] = want - above - (second ? cnt[0] : 0);
      }
      __syncthreads();
      prefix |= found[0] << shift;
      want = found[1];
    }
    least = prefix;
  }
  // every key above `least`, and the first `want` places of it
  uint32_t base = 0, base_eq = 0;
  auto emit = [&](int step, uint32_t in, const uint32_t (&k)[kPer]) {
    const int j0 = step * kStep + tid * kPer;
    uint32_t take = 0, equal = 0;  // bit masks over the thread's places
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool competing = (in >> i) & 1;
      if (competing ? k[i] > least : j0 + i < n) take |= 1u << i;
      if (competing && k[i] == least) equal |= 1u << i;
    }
    // both counts in one word: at most 4,096 each per step
    const uint32_t mine = __popc(take) | (__popc(equal) << 16);
    uint32_t total;
    const uint32_t excl = block_scan(mine, warp_sum, total) - mine;
    uint32_t taken = base + (excl & 0xFFFFu), eq = base_eq + (excl >> 16);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const bool is_eq = (equal >> i) & 1;
      if (((take >> i) & 1) || (is_eq && eq < want)) {
        const uint32_t at = taken + min(eq, want);
        if (at < static_cast<uint32_t>(n_new)) {
          kept[at] = j0 + i;
          to_w[at] = __ldg(w + j0 + i);
        }
      }
      taken += (take >> i) & 1;
      eq += is_eq;
    }
    base += total & 0xFFFFu;
    base_eq += total >> 16;
  };
#pragma unroll
  for (int c = 0; c < kCached; ++c)
    if (c < steps) emit(c, competes >> (kPer * c), cache[c]);
  for (int c = kCached; c < steps; ++c) {
    float x[kPer];
    uint32_t k[kPer];
    load(c, x);
#pragma unroll
    for (int i = 0; i < kPer; ++i) k[i] = key_of(x[i]);
    emit(c, range(c), k);
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
  // all of a thread's loads before its stores: source and destination are one
  // buffer, so the compiler would keep each load behind the store before it
  constexpr int kCh = L::kCodeRow / 16;  // 16-byte chunks of a code row
  constexpr int kEach = kKv4Page * kCh * 2 / kMoveThreads;
  using Scale = std::conditional_t<D == 128, uint2, uint32_t>;  // a row's scales of keys or values
  uint4 codes[kEach];
  Scale scales;
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = tid + k * kMoveThreads, part = i / (kKv4Page * kCh), x = i % (kKv4Page * kCh), r = x / kCh, ch = x % kCh;
    if (r < rows)
      codes[k] = *reinterpret_cast<const uint4*>(a.c.pages + from[r] + part * L::kV + from_row[r] * L::kCodeRow + ch * 16);
  }
  static_assert(kMoveThreads == 2 * kKv4Page, "one scale group per thread");
  const int s_part = tid / kKv4Page, s_row = tid % kKv4Page;
  const int64_t s_base = L::kKs + s_part * (L::kVs - L::kKs);
  if (s_row < rows)
    scales = *reinterpret_cast<const Scale*>(a.c.pages + from[s_row] + s_base + from_row[s_row] * L::kScaleRow);
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    const int i = tid + k * kMoveThreads, part = i / (kKv4Page * kCh), x = i % (kKv4Page * kCh), r = x / kCh, ch = x % kCh;
    if (r < rows) *reinterpret_cast<uint4*>(dst + part * L::kV + r * L::kCodeRow + ch * 16) = codes[k];
  }
  if (s_row < rows) *reinterpret_cast<Scale*>(dst + s_base + s_row * L::kScaleRow) = scales;
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t kv4_evict_workspace(int64_t n_pages, int n_seqs, int kv_heads, int budget) {
  const size_t bits = n_pages <= kSharedPages ? 0 : 2 * up(static_cast<size_t>((n_pages + 31) / 32) * 4);
  return 256 + bits +
         up(static_cast<size_t>(n_seqs) * kv_heads * budget * 4);
}

int launch_kv4_evict(const Kv4& c, int head_dim, const float* weights, int budget, int sinks, int recent,
                     const int32_t* to_table, int to_max_pages, int32_t* to_lens, float* to_weights, int32_t* kept,
                     void* ws, int32_t* status, cudaStream_t s) {
  const bool shared = c.n_pages <= kSharedPages;
  const size_t bits = shared ? 0 : up(static_cast<size_t>((c.n_pages + 31) / 32) * 4);
  uint8_t* w = static_cast<uint8_t*>(ws);
  EvictArgs a{c, weights, budget, sinks, recent, to_table, to_max_pages, to_lens, to_weights, kept, nullptr, nullptr,
              nullptr, status};
  a.clash = reinterpret_cast<int32_t*>(w);
  if (kept == nullptr) a.kept = reinterpret_cast<int32_t*>(w + 256 + 2 * bits);
  size_t smem = kCopies * kDigits * 4;
  if (shared) {
    smem = std::max(smem, static_cast<size_t>((c.n_pages + 31) / 32) * 8);
  } else {
    a.src_bits = reinterpret_cast<uint32_t*>(w + 256);
    a.dst_bits = reinterpret_cast<uint32_t*>(w + 256 + bits);
    if (cudaMemsetAsync(w, 0, 256 + 2 * bits, s) != cudaSuccess) return VLM_ERR_CUDA;
  }
  static bool ready[64] = {};  // 64 KB of shared memory, once per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return VLM_ERR_CUDA;
  if (dev >= 64 || !ready[dev]) {
    if (cudaFuncSetAttribute(kv4_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kSharedPages / 32 * 8)) != cudaSuccess)
      return VLM_ERR_CUDA;
    if (dev < 64) ready[dev] = true;
  }
  launch_begin(KC_KV4_EVICT, s);
  cudaError_t e = launch_pdl(kv4_select_kernel, dim3(c.kv_heads + 1, c.n_seqs), dim3(kSelThreads), smem, s, a);
  const dim3 grid((budget + kKv4Page - 1) / kKv4Page, c.kv_heads, c.n_seqs);
  if (e == cudaSuccess)
    e = head_dim == 128 ? launch_pdl(kv4_move_kernel<128>, grid, dim3(kMoveThreads), 0, s, a)
                        : launch_pdl(kv4_move_kernel<64>, grid, dim3(kMoveThreads), 0, s, a);
  launch_end(KC_KV4_EVICT, s);
  note_extra_launches(1);
  return e == cudaSuccess ? VLM_OK : VLM_ERR_CUDA;
}

}  // namespace vlm
