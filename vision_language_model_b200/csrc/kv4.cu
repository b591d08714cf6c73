// Rows into the paged 4-bit cache and back (layout in kv4.cuh).
//   write: per block of 16 columns s = e4m3(amax / fp32(6 s_g)),
//          r = 1 / fp32(s s_g) (0 if s is 0), codes e2m1(x r) -- the NVFP4
//          recipe of nvfp4.cuh, every step one fp32 operation;
//   read:  fp32(code * s * s_g) rounded once to the output type (code * s has
//          at most 6 significant bits, so only the last product rounds).
// Both are bound by the bytes they move. A thread takes one block of a row, 32
// bytes of 16-bit values against 8 bytes of codes and one scale byte, for
// several heads: where a row lives (its sequence, place and page: a chain of
// dependent loads) is looked up once, and the heads' loads then run together.
// With a lookup per head the chain was the bound: 25,600 rows of 8 heads of 128
// read in 37 us, 3.6 TB/s; now 27 us, 5.6. The D / 16 blocks of a row and four consecutive
// tokens make up neighbouring threads (a whole warp at D = 128), so codes go to
// memory as runs of 4 * D / 2 bytes and scales as whole 32-byte sectors where
// the tokens share a page.
#include "kv4.cuh"

namespace vlm {

namespace {

constexpr int kThreads = 128;

// Largest s with cu[s] <= t: the sequence of packed row t.
__device__ __forceinline__ int seq_of(const int32_t* cu, int n_seqs, int64_t t) {
  int lo = 0, hi = n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(cu + mid) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Where packed row t lives: its page and the row inside it, or false (and the
// status word set) when it lies behind the table's room or outside cu.
__device__ __forceinline__ bool locate(const Kv4& c, const int32_t* cu, int64_t t, int64_t& page, int& row,
                                       int32_t* status) {
  int s;
  int64_t first = 0;
  if (cu == nullptr) {
    s = static_cast<int>(t);
    first = t;
  } else {
    s = seq_of(cu, c.n_seqs, t);
    first = __ldg(cu + s);
    if (t < first || t >= __ldg(cu + s + 1)) {
      set_status(status, VLM_ERR_BAD_PAGE);
      return false;
    }
  }
  const int64_t pos = (c.lens == nullptr ? 0 : static_cast<int64_t>(__ldg(c.lens + s))) + (t - first);
  if (pos < 0 || pos >= static_cast<int64_t>(c.max_pages) * kKv4Page) {
    set_status(status, VLM_ERR_BAD_PAGE);
    return false;
  }
  const int32_t p = __ldg(c.table + static_cast<int64_t>(s) * c.max_pages + pos / kKv4Page);
  if (static_cast<uint32_t>(p) >= static_cast<uint64_t>(c.n_pages)) {
    set_status(status, VLM_ERR_BAD_PAGE);
    return false;
  }
  page = p;
  row = static_cast<int>(pos % kKv4Page);
  return true;
}

// Thread i: blocks fastest, then tokens.
template <int NB>
__device__ __forceinline__ void split_item(int64_t i, int64_t& t, int& b) {
  b = static_cast<int>(i % NB);
  t = i / NB;
}

// 32 bytes, in one access where they are aligned to it.
__device__ __forceinline__ void load32(const void* p, bool wide, uint32_t (&w)[8]) {
  if (wide) {
    asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(p));
  } else {
    const uint4 u0 = __ldg(static_cast<const uint4*>(p)), u1 = __ldg(static_cast<const uint4*>(p) + 1);
    w[0] = u0.x; w[1] = u0.y; w[2] = u0.z; w[3] = u0.w;
    w[4] = u1.x; w[5] = u1.y; w[6] = u1.z; w[7] = u1.w;
  }
}

constexpr int kBatch = 4;  // heads whose loads are issued together

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    kv4_append_kernel(const Kv4 c, const int32_t* __restrict__ cu, int64_t n_new, const T* __restrict__ k,
                      int64_t k_stride, const T* __restrict__ v, int64_t v_stride, int heads_per, int32_t* status) {
  using L = Kv4Layout<D>;
  constexpr int NB = D / 16;
  griddep_wait();
  griddep_launch_dependents();
  int64_t t;
  int b;
  split_item<NB>(static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, t, b);
  if (t >= n_new) return;
  const bool is_v = blockIdx.y != 0;
  const T* src = (is_v ? v + t * v_stride : k + t * k_stride) + b * 16;
  const bool wide = ((reinterpret_cast<uintptr_t>(is_v ? v : k) | ((is_v ? v_stride : k_stride) * 2)) & 31) == 0;
  int64_t page;
  int row;
  if (!locate(c, cu, t, page, row, status)) return;
  const float sg = is_v ? c.v_sg : c.k_sg, six_sg = 6.0f * sg;
  uint8_t* dst = c.pages + page * c.kv_heads * L::kBytes;
  const int code_at = (is_v ? L::kV : 0) + row * L::kCodeRow + b * 8;
  const int scale_at = (is_v ? L::kVs : L::kKs) + row * L::kScaleRow + b;
  const int h0 = blockIdx.z * heads_per, h1 = min(c.kv_heads, h0 + heads_per);
  for (int h = h0; h < h1; h += kBatch) {
    uint32_t w[kBatch][8];
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
      if (h + i < h1) load32(src + (h + i) * D, wide, w[i]);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (h + i >= h1) break;
      float x[16], amax = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 f = unpack16<T>(w[i][j]);
        x[2 * j] = f.x;
        x[2 * j + 1] = f.y;
        amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
      }
      uint2 codes;
      const uint32_t sb = nvfp4_quant16(x, amax, sg, six_sg, codes);
      uint8_t* at = dst + static_cast<int64_t>(h + i) * L::kBytes;
      *reinterpret_cast<uint2*>(at + code_at) = codes;
      at[scale_at] = static_cast<uint8_t>(sb);
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    kv4_read_kernel(const Kv4 c, const int32_t* __restrict__ cu, int64_t n_rows, T* __restrict__ k,
                    T* __restrict__ v, int heads_per, int32_t* status) {
  using L = Kv4Layout<D>;
  constexpr int NB = D / 16;
  griddep_wait();
  griddep_launch_dependents();
  int64_t t;
  int b;
  split_item<NB>(static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x, t, b);
  if (t >= n_rows) return;
  const bool is_v = blockIdx.y != 0;
  int64_t page;
  int row;
  if (!locate(c, cu, t, page, row, status)) return;
  const uint8_t* src = c.pages + page * c.kv_heads * L::kBytes;
  const int code_at = (is_v ? L::kV : 0) + row * L::kCodeRow + b * 8;
  const int scale_at = (is_v ? L::kVs : L::kKs) + row * L::kScaleRow + b;
  const float sg = is_v ? c.v_sg : c.k_sg;
  T* dst = (is_v ? v : k) + t * c.kv_heads * D + b * 16;
  const bool wide = (reinterpret_cast<uintptr_t>(is_v ? v : k) & 31) == 0;
  const int h0 = blockIdx.z * heads_per, h1 = min(c.kv_heads, h0 + heads_per);
  for (int h = h0; h < h1; h += kBatch) {
    uint2 codes[kBatch];
    uint32_t sb[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (h + i < h1) {
        const uint8_t* at = src + static_cast<int64_t>(h + i) * L::kBytes;
        codes[i] = __ldg(reinterpret_cast<const uint2*>(at + code_at));
        sb[i] = __ldg(at + scale_at);
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      if (h + i >= h1) break;
      const float scale = e4m3_value(sb[i]);
      uint32_t w[8];
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        uint32_t p[4];
        e2m1x8_f16(half ? codes[i].y : codes[i].x, p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = unpack16<__half>(p[j]);
          w[4 * half + j] = pack16<T>(__fmul_rn(f.x * scale, sg), __fmul_rn(f.y * scale, sg));
        }
      }
      store32(dst + (h + i) * D, w, wide);
    }
  }
}

// Threads of one head over all rows and both operands, and how many heads a
// thread takes: all that fit a few batches once the rows alone fill the SMs.
int grid_of(int64_t rows, int heads, int nb, dim3& grid, int& heads_per) {
  const int64_t g = (rows * nb + kThreads - 1) / kThreads;
  if (g > 0x7FFFFFFFLL) return VLM_ERR_BAD_SHAPE;
  const int64_t want = 4LL * num_sms() / (2 * g) + 1;  // CTAs along the heads that fill the SMs' slots
  int per = static_cast<int>((heads + want - 1) / want);
  per = per < 8 ? per : 8;
  per = per < (heads + 65534) / 65535 ? (heads + 65534) / 65535 : per;
  heads_per = per;
  grid = dim3(static_cast<unsigned>(g), 2, static_cast<unsigned>((heads + per - 1) / per));
  return VLM_OK;
}

}  // namespace

int launch_kv4_append(const Kv4& c, int head_dim, const int32_t* cu_new, int64_t n_new, int dtype, const void* k,
                      int64_t k_stride, const void* v, int64_t v_stride, int32_t* status, cudaStream_t s) {
  dim3 grid;
  int heads_per;
  const int rc = grid_of(n_new, c.kv_heads, head_dim / 16, grid, heads_per);
  if (rc != VLM_OK) return rc;
  launch_begin(KC_KV4_ROWS, s);
  auto go = [&](auto kern, auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    return launch_pdl(kern, grid, dim3(kThreads), 0, s, c, cu_new, n_new, static_cast<const T*>(k), k_stride,
                      static_cast<const T*>(v), v_stride, heads_per, status);
  };
  __nv_bfloat16* bf = nullptr;
  __half* hf = nullptr;
  const cudaError_t e = dtype == VLM_DTYPE_F16
                            ? (head_dim == 128 ? go(kv4_append_kernel<__half, 128>, hf) : go(kv4_append_kernel<__half, 64>, hf))
                            : (head_dim == 128 ? go(kv4_append_kernel<__nv_bfloat16, 128>, bf)
                                               : go(kv4_append_kernel<__nv_bfloat16, 64>, bf));
  launch_end(KC_KV4_ROWS, s);
  return e == cudaSuccess ? VLM_OK : VLM_ERR_CUDA;
}

int launch_kv4_read(const Kv4& c, int head_dim, const int32_t* cu, int64_t n_rows, int dtype, void* k, void* v,
                    int32_t* status, cudaStream_t s) {
  dim3 grid;
  int heads_per;
  const int rc = grid_of(n_rows, c.kv_heads, head_dim / 16, grid, heads_per);
  if (rc != VLM_OK) return rc;
  launch_begin(KC_KV4_ROWS, s);
  auto go = [&](auto kern, auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    return launch_pdl(kern, grid, dim3(kThreads), 0, s, c, cu, n_rows, static_cast<T*>(k), static_cast<T*>(v),
                      heads_per, status);
  };
  __nv_bfloat16* bf = nullptr;
  __half* hf = nullptr;
  const cudaError_t e = dtype == VLM_DTYPE_F16
                            ? (head_dim == 128 ? go(kv4_read_kernel<__half, 128>, hf) : go(kv4_read_kernel<__half, 64>, hf))
                            : (head_dim == 128 ? go(kv4_read_kernel<__nv_bfloat16, 128>, bf)
                                               : go(kv4_read_kernel<__nv_bfloat16, 64>, bf));
  launch_end(KC_KV4_ROWS, s);
  return e == cudaSuccess ? VLM_OK : VLM_ERR_CUDA;
}

}  // namespace vlm
