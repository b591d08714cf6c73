// Rows into the paged 4-bit cache and back (layout in kv4.cuh).
//   write: per block of 16 columns s = e4m3(amax / fp32(6 s_g)),
//          r = 1 / fp32(s s_g) (0 if s is 0), codes e2m1(x r) -- the NVFP4
//          recipe of nvfp4.cuh, every step one fp32 operation;
//   read:  fp32(code * s * s_g) rounded once to the output type (code * s has
//          at most 6 significant bits, so only the last product rounds).
// Both are bound by the bytes they move. A thread takes one block: 32 bytes of
// 16-bit values against 8 bytes of codes and one scale byte. The D / 16 blocks
// of a row and four consecutive tokens of one head make up the neighbouring
// threads (a whole warp at D = 128), so codes go to memory as runs of
// 4 * D / 2 bytes and scales as whole 32-byte sectors where the tokens share
// a page.
#include "kv4.cuh"

namespace vlm {

namespace {

constexpr int kThreads = 256;

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

// Item i of a (rows x heads x blocks) grid: blocks fastest, then four tokens,
// then heads, then groups of four tokens.
template <int NB>
__device__ __forceinline__ void split_item(int64_t i, int heads, int64_t& t, int& h, int& b) {
  b = static_cast<int>(i % NB);
  const int64_t j = i / (NB * 4);
  h = static_cast<int>(j % heads);
  t = j / heads * 4 + (i / NB) % 4;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    kv4_append_kernel(const Kv4 c, const int32_t* __restrict__ cu, int64_t n_new, const T* __restrict__ k,
                      int64_t k_stride, const T* __restrict__ v, int64_t v_stride, int32_t* status) {
  using L = Kv4Layout<D>;
  constexpr int NB = D / 16;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  int64_t t;
  int h, b;
  split_item<NB>(i, c.kv_heads, t, h, b);
  if (t >= n_new) return;
  const bool is_v = blockIdx.y != 0;
  const uint4* src = reinterpret_cast<const uint4*>((is_v ? v + t * v_stride : k + t * k_stride) + h * D + b * 16);
  const uint4 u0 = __ldg(src), u1 = __ldg(src + 1);
  int64_t page;
  int row;
  if (!locate(c, cu, t, page, row, status)) return;
  const uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
  float x[16], amax = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 f = unpack16<T>(w[j]);
    x[2 * j] = f.x;
    x[2 * j + 1] = f.y;
    amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  const float sg = is_v ? c.v_sg : c.k_sg;
  uint2 codes;
  const uint32_t sb = nvfp4_quant16(x, amax, sg, 6.0f * sg, codes);
  uint8_t* dst = c.pages + (page * c.kv_heads + h) * L::kBytes;
  *reinterpret_cast<uint2*>(dst + (is_v ? L::kV : 0) + row * L::kCodeRow + b * 8) = codes;
  dst[(is_v ? L::kVs : L::kKs) + row * L::kScaleRow + b] = static_cast<uint8_t>(sb);
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads)
    kv4_read_kernel(const Kv4 c, const int32_t* __restrict__ cu, int64_t n_rows, T* __restrict__ k,
                    T* __restrict__ v, int32_t* status) {
  using L = Kv4Layout<D>;
  constexpr int NB = D / 16;
  griddep_wait();
  griddep_launch_dependents();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  int64_t t;
  int h, b;
  split_item<NB>(i, c.kv_heads, t, h, b);
  if (t >= n_rows) return;
  const bool is_v = blockIdx.y != 0;
  int64_t page;
  int row;
  if (!locate(c, cu, t, page, row, status)) return;
  const uint8_t* src = c.pages + (page * c.kv_heads + h) * L::kBytes;
  const uint2 codes = __ldg(reinterpret_cast<const uint2*>(src + (is_v ? L::kV : 0) + row * L::kCodeRow + b * 8));
  const float sb = e4m3_value(__ldg(src + (is_v ? L::kVs : L::kKs) + row * L::kScaleRow + b));
  const float sg = is_v ? c.v_sg : c.k_sg;
  uint32_t w[8];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t p[4];
    e2m1x8_f16(half ? codes.y : codes.x, p);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = unpack16<__half>(p[j]);
      w[4 * half + j] = pack16<T>(__fmul_rn(f.x * sb, sg), __fmul_rn(f.y * sb, sg));
    }
  }
  uint4* dst = reinterpret_cast<uint4*>((is_v ? v : k) + (t * c.kv_heads + h) * D + b * 16);
  dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
  dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

int grid_of(int64_t rows, int heads, int nb, unsigned& grid) {
  const int64_t items = (rows + 3) / 4 * 4 * heads * nb;
  const int64_t g = (items + kThreads - 1) / kThreads;
  if (g > 0x7FFFFFFFLL) return VLM_ERR_BAD_SHAPE;
  grid = static_cast<unsigned>(g);
  return VLM_OK;
}

}  // namespace

int launch_kv4_append(const Kv4& c, int head_dim, const int32_t* cu_new, int64_t n_new, int dtype, const void* k,
                      int64_t k_stride, const void* v, int64_t v_stride, int32_t* status, cudaStream_t s) {
  unsigned grid;
  const int rc = grid_of(n_new, c.kv_heads, head_dim / 16, grid);
  if (rc != VLM_OK) return rc;
  launch_begin(KC_KV4_ROWS, s);
  auto go = [&](auto kern, auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    return launch_pdl(kern, dim3(grid, 2), dim3(kThreads), 0, s, c, cu_new, n_new, static_cast<const T*>(k), k_stride,
                      static_cast<const T*>(v), v_stride, status);
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
  unsigned grid;
  const int rc = grid_of(n_rows, c.kv_heads, head_dim / 16, grid);
  if (rc != VLM_OK) return rc;
  launch_begin(KC_KV4_ROWS, s);
  auto go = [&](auto kern, auto* p) {
    using T = std::remove_pointer_t<decltype(p)>;
    return launch_pdl(kern, dim3(grid, 2), dim3(kThreads), 0, s, c, cu, n_rows, static_cast<T*>(k), static_cast<T*>(v),
                      status);
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
