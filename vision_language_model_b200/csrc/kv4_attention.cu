// Attention of a few new tokens over the paged 4-bit cache (layout in kv4.cuh).
// Sequence s has len tokens in the cache, its m new ones last; new token i
// sees the places j <= len - m + i:
//   o_i = sum_j p_ij v_j,  p_ij = softmax_j(scale q_i . k_j)
// for the G = heads / kv_heads query heads of every key head.
//
// Bound: the codes are read once, 9/8 byte per column and head, so the floor
// is HBM; what competes with it is the issue rate of turning codes into
// operands. The layout of the work:
//   - The G * m query rows of one (sequence, key head) are the 16 rows of
//     mma.m16n8k16 (fp16 operands, fp32 sums; more rows: further row tiles).
//     At one to sixteen rows the product is far from the tensor cores' rate,
//     and its operands can be made in registers, which tcgen05 cannot take.
//   - A warp takes 16 tokens of a page. Its bytes come by cp.async into a ring
//     of its own in shared memory, so no warp waits for another.
//   - Code times block scale has at most 6 significant bits, so fp16 holds it
//     exactly: one cvt and one multiply per two values, no rounding. A query
//     row is scaled by a power of two so that its largest value lies in [1, 2)
//     and rounded to fp16: bf16 has 8 significant bits, so only values below
//     2^-14 of the row's largest lose bits, 2^-25 of the largest at most --
//     what an fp32 sum loses as well. The global scales, 1 / that power and
//     log2(e) are one fp32 factor of the logit.
//   - P is rounded to fp16 for the second product (half a step, 2^-11); the
//     sum of a row's weights, its maximum and both products' sums stay in fp32.
//   - Work is cut into equal runs of pages over the flattened (sequence, key
//     head, row tile, page) list, whatever the lengths, computed on the device
//     from the lengths there, so a captured graph replays with other lengths.
//     A unit (sequence, key head, row tile) cut by a border leaves partial sums
//     that kv4_combine_kernel joins in the order of the runs: the result does
//     not depend on timing.
// Places behind what a row sees get logit -inf; value scales of places behind
// the sequence's end are taken as 0, so stale bytes (NaN scales among them)
// reach no sum. A row that sees nothing is 0.
#include <algorithm>

#include "kv4.cuh"
#include "softmax.cuh"

namespace vlm {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSlice = 16;   // tokens of a page per warp
constexpr int kStages = 4;   // ring of slices per warp
constexpr int kMaxSeqs = 4096;  // sequences per launch (their page offsets are held in shared memory)
constexpr int kCtasPerSm = 3;
constexpr int kMinPages = 4;  // a run shorter than this costs more to join than it gains
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescale = 8.0f;  // log2 units; P stays below 2^8

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
struct Args {
  Kv4 c;
  const void* q;
  int64_t q_stride;  // elements between tokens
  int heads, group, q_len, rows, row_tiles;
  float scale;
  void* out;         // [n_seqs * q_len, heads, D]
  int32_t* prefix;   // [n_seqs + 1] page offsets, written by the first kernel's CTA 0
  float* part_o;     // [2 * grid][16][D]
  float2* part_ml;   // [2 * grid][16] maximum (log2 units) and sum
  float* lse;        // [n_seqs, kv_heads, rows] log2 of a row's sum (null: not wanted)
  float* weights;    // [n_seqs, kv_heads, max_pages * 64]
  int grid;          // CTAs of the first kernel
  int32_t* status;
};

// Fragment maps. Lane = 4 g + c. The 16 tokens of a slice are the two 8-wide
// column tiles i of S; column 2 c + e of tile i is token 8 i + 4 e + (c ^ x e).
// x (1 for D = 128, 2 for D = 64) spreads the rows that one load touches over
// the banks. A lane's k elements of a query or key row, and its columns of O,
// are the D / 4 columns from c D / 4 on.
template <int D>
struct Map {
  static constexpr int kX = D == 128 ? 1 : 2;
  static constexpr int kSteps = D / 16;                // mma steps of a logit
  static constexpr int kCols = D / 4;                  // columns per lane
  static constexpr int kKOff = 0, kVOff = kSlice * D / 2;
  static constexpr int kKsOff = kSlice * D, kVsOff = kKsOff + kSlice * D / 16;
  static constexpr int kBytes = kVsOff + kSlice * D / 16;  // one slice
  static __device__ __forceinline__ int token(int i, int c, int e) { return 8 * i + 4 * e + (c ^ (kX * e)); }
};

struct Plan {
  int64_t total, chunk;
};

// The page offsets of all sequences into shared memory (prefix[n_seqs + 1]) and the cut.
__device__ __forceinline__ Plan make_plan(const Kv4& c, int units_per_seq, int grid, int* prefix, int* warp_sum,
                                          int32_t* status) {
  const int n = c.n_seqs, per = (n + kThreads - 1) / kThreads;
  const int lo = min(n, static_cast<int>(threadIdx.x) * per), hi = min(n, lo + per);
  int sum = 0;
  for (int s = lo; s < hi; ++s) sum += (kv4_len(c, s, status) + kKv4Page - 1) / kKv4Page;
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, inc, o);
    if ((threadIdx.x & 31) >= o) inc += v;
  }
  if ((threadIdx.x & 31) == 31) warp_sum[threadIdx.x >> 5] = inc;
  __syncthreads();
  int base = inc - sum;
  for (int w = 0; w < static_cast<int>(threadIdx.x >> 5); ++w) base += warp_sum[w];
  for (int s = lo; s < hi; ++s) {
    prefix[s] = base;
    base += (kv4_len(c, s, nullptr) + kKv4Page - 1) / kKv4Page;
  }
  if (hi == n && lo < n) prefix[n] = base;
  __syncthreads();
  Plan p;
  p.total = static_cast<int64_t>(prefix[n]) * units_per_seq;
  p.chunk = max(static_cast<int64_t>(kMinPages), (p.total + grid - 1) / grid);
  return p;
}

// A lane's part of the 16 query rows [first, first + 16) of (sequence, key
// head) as mma A fragments, and the factor of its two rows' logits.
template <typename T, int D>
__device__ __forceinline__ void load_q(const Args& a, int s, int kvh, int first, uint32_t (&qf)[D / 16][4],
                                       float (&factor)[2]) {
  using M = Map<D>;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int r = first + g + 8 * half;
    uint32_t w[M::kCols / 2];
#pragma unroll
    for (int j = 0; j < M::kCols / 2; ++j) w[j] = 0;
    if (r < a.rows) {
      const int tok = r / a.group, h = kvh * a.group + r % a.group;
      const uint4* src = reinterpret_cast<const uint4*>(
          static_cast<const T*>(a.q) + (static_cast<int64_t>(s) * a.q_len + tok) * a.q_stride + h * D + c * M::kCols);
#pragma unroll
      for (int j = 0; j < M::kCols / 8; ++j) {
        const uint4 u = __ldg(src + j);
        w[4 * j] = u.x; w[4 * j + 1] = u.y; w[4 * j + 2] = u.z; w[4 * j + 3] = u.w;
      }
    }
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < M::kCols / 2; ++j) {
      const float2 f = unpack16<T>(w[j]);
      amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // 2^-floor(log2 amax); 1 where amax is 0, subnormal or infinite
    const int e = static_cast<int>(__float_as_uint(amax) >> 23);
    const float mul = e == 0 || e == 255 ? 1.0f : __uint_as_float(static_cast<uint32_t>(max(254 - e, 1)) << 23);
    factor[half] = a.scale * a.c.k_sg * kLog2e / mul;
#pragma unroll
    for (int k = 0; k < M::kSteps; ++k) {
      const float2 f0 = unpack16<T>(w[2 * k]), f1 = unpack16<T>(w[2 * k + 1]);
      qf[k][half] = pack_f16x2(f0.x * mul, f0.y * mul);
      qf[k][2 + half] = pack_f16x2(f1.x * mul, f1.y * mul);
    }
  }
}

// A warp's 16 tokens of one page into its ring slot (keys only: kValues false).
template <int D, bool kValues>
__device__ __forceinline__ void fetch(uint32_t dst, const uint8_t* page, int warp) {
  using L = Kv4Layout<D>;
  using M = Map<D>;
  const int lane = threadIdx.x & 31;
  const uint8_t* k = page + warp * kSlice * L::kCodeRow;
  const uint8_t* v = page + L::kV + warp * kSlice * L::kCodeRow;
  constexpr int kPerRow = D / 32;  // 16-byte chunks of a code row
#pragma unroll
  for (int j = 0; j < kSlice * kPerRow / 32; ++j) {
    const int x = j * 32 + lane, row = x / kPerRow, ch = x % kPerRow;
    cp_async16(dst + M::kKOff + x * 16, k + x * 16);
    // the value rows' chunks are exchanged by row so that four rows' halves lie in different banks (D = 128)
    if (kValues) cp_async16(dst + M::kVOff + (row * kPerRow + (D == 128 ? ch ^ (row & 2) : ch)) * 16, v + x * 16);
  }
  constexpr int kSc = kSlice * D / 256;  // 16-byte chunks of a slice's scales
  if (lane < kSc)
    cp_async16(dst + M::kKsOff + lane * 16, page + L::kKs + warp * kSlice * L::kScaleRow + lane * 16);
  else if (kValues && lane < 2 * kSc)
    cp_async16(dst + M::kVsOff + (lane - kSc) * 16,
               page + L::kVs + warp * kSlice * L::kScaleRow + (lane - kSc) * 16);
}

// S = q . (code * scale) for the 16 tokens of a slice.
template <int D>
__device__ __forceinline__ void logits(const uint8_t* st, const uint32_t (&qf)[D / 16][4], float (&s)[2][4]) {
  using M = Map<D>;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
    const int row = M::token(i, g >> 1, g & 1);
    uint32_t w[D / 32];
    uint32_t sc[2];
    if constexpr (D == 128) {
      const uint4 u = *reinterpret_cast<const uint4*>(st + M::kKOff + row * 64 + c * 16);
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
      const uint32_t h2 = e4m3x2_f16(*reinterpret_cast<const uint16_t*>(st + M::kKsOff + row * 8 + 2 * c));
      sc[0] = __byte_perm(h2, 0, 0x1010);
      sc[1] = __byte_perm(h2, 0, 0x3232);
    } else {
      const uint2 u = *reinterpret_cast<const uint2*>(st + M::kKOff + row * 32 + c * 8);
      w[0] = u.x; w[1] = u.y;
      const uint32_t h2 = e4m3x2_f16(st[M::kKsOff + row * 4 + c]);
      sc[0] = sc[1] = __byte_perm(h2, 0, 0x1010);
    }
#pragma unroll
    for (int x = 0; x < D / 32; ++x) {
      uint32_t p[4];
      e2m1x8_f16(w[x], p);
      const uint32_t f = sc[D == 128 ? x >> 1 : 0];
      mma16816(s[i], qf[2 * x], hmul2(p[0], f), hmul2(p[1], f));
      mma16816(s[i], qf[2 * x + 1], hmul2(p[2], f), hmul2(p[3], f));
    }
  }
}

// Where run position x lies: sequence, key head, row tile, first page.
struct Place {
  int s, kvh, tile, page, pages;
};
__device__ __forceinline__ Place place_of(const int* prefix, int n_seqs, int kv_heads, int row_tiles, int64_t x) {
  const int per_seq = kv_heads * row_tiles;
  int lo = 0, hi = n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<int64_t>(prefix[mid]) * per_seq <= x) lo = mid; else hi = mid - 1;
  }
  Place p;
  p.s = lo;
  p.pages = prefix[lo + 1] - prefix[lo];
  const int64_t r = x - static_cast<int64_t>(prefix[lo]) * per_seq;
  const int unit = static_cast<int>(r / p.pages);
  p.page = static_cast<int>(r - static_cast<int64_t>(unit) * p.pages);
  p.kvh = unit / row_tiles;
  p.tile = unit % row_tiles;
  return p;
}

// Element (row, column quad) of the O tile a warp leaves in its ring, in
// floats; the exchange spreads the quads of a column group over the banks.
template <int D>
__device__ __forceinline__ int o_at(int row, int quad) {
  constexpr int kPer = D / 16;  // quads per lane's column run
  return row * D + ((quad ^ ((quad / kPer) * 2) ^ (row & 1)) * 4);
}

template <typename T>
__device__ __forceinline__ void store4(T* dst, float x, float y, float z, float w) {
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack16<T>(x, y), pack16<T>(z, w));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv4_attn_kernel(const Args a) {
  using M = Map<D>;
  using L = Kv4Layout<D>;
  static_assert(kStages * M::kBytes >= 16 * D * 4, "a warp's O tile fits its ring");
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int warp_sum[kWarps];
  __shared__ float sm_m[kWarps][16], sm_l[kWarps][16];
  uint8_t* ring_base = smem;
  int* prefix = reinterpret_cast<int*>(smem + kWarps * kStages * M::kBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  uint8_t* ring = ring_base + warp * kStages * M::kBytes;
  const uint32_t ring_s = smem_u32(ring);

  griddep_wait();
  griddep_launch_dependents();
  const int per_seq = a.c.kv_heads * a.row_tiles;
  const Plan plan = make_plan(a.c, per_seq, a.grid, prefix, warp_sum, blockIdx.x == 0 ? a.status : nullptr);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= a.c.n_seqs; i += kThreads) a.prefix[i] = prefix[i];

  // sequences without a token: their rows are 0
  for (int s = blockIdx.x; s < a.c.n_seqs; s += a.grid) {
    if (prefix[s + 1] != prefix[s]) continue;
    uint2* dst = reinterpret_cast<uint2*>(static_cast<T*>(a.out) + static_cast<int64_t>(s) * a.q_len * a.heads * D);
    for (int i = threadIdx.x; i < a.q_len * a.heads * D / 4; i += kThreads) dst[i] = make_uint2(0, 0);
  }

  const int64_t begin = blockIdx.x * plan.chunk;
  const int64_t end = min(plan.total, begin + plan.chunk);
  for (int64_t x = begin; x < end;) {
    const Place at = place_of(prefix, a.c.n_seqs, a.c.kv_heads, a.row_tiles, x);
    const int p0 = at.page;
    const int p1 = static_cast<int>(min(static_cast<int64_t>(at.pages), p0 + (end - x)));
    const int len = kv4_len(a.c, at.s, nullptr);
    // the places below `open` are seen by every row
    const int open = len - a.q_len + 1;
    uint32_t qf[D / 16][4];
    float factor[2];
    load_q<T, D>(a, at.s, at.kvh, at.tile * 16, qf, factor);
    int seen[2];  // one past the last place each of the lane's rows sees
#pragma unroll
    for (int half = 0; half < 2; ++half) seen[half] = open + (at.tile * 16 + g + 8 * half) / a.group;

    float o[D / 8][4];
#pragma unroll
    for (int j = 0; j < D / 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] = 0.0f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};

    int ids = 0, ids_at = p0;  // page offsets of 32 entries from ids_at on, one per lane
    auto issue = [&](int p) {
      if (p < p1) {
        if (p >= ids_at + 32 || p == p0) {
          ids_at = p;
          ids = p + lane < p1 ? static_cast<int>(kv4_page(a.c, at.s, p + lane, a.status)) : 0;
        }
        const int id = __shfl_sync(0xffffffffu, ids, p - ids_at);
        if (p * kKv4Page + warp * kSlice < len)
          fetch<D, true>(ring_s + (p - p0) % kStages * M::kBytes,
                         a.c.pages + (static_cast<int64_t>(id) * a.c.kv_heads + at.kvh) * L::kBytes, warp);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int j = 0; j < kStages - 1; ++j) issue(p0 + j);

    for (int p = p0; p < p1; ++p) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const uint8_t* st = ring + (p - p0) % kStages * M::kBytes;
      issue(p + kStages - 1);
      const int first = p * kKv4Page + warp * kSlice;
      if (first >= len) continue;
      float s[2][4];
      logits<D>(st, qf, s);
      float mx[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[i][e] *= factor[e >> 1];
      const bool edge = first + kSlice > open;
      if (edge) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (first + M::token(i, c, e & 1) >= seen[e >> 1]) s[i][e] = -INFINITY;
      }
#pragma unroll
      for (int half = 0; half < 2; ++half)
        mx[half] = fmaxf(fmaxf(s[0][2 * half], s[0][2 * half + 1]), fmaxf(s[1][2 * half], s[1][2 * half + 1]));
      if (__any_sync(0xffffffffu, mx[0] > m[0] + kRescale || mx[1] > m[1] + kRescale)) {
        float corr[2];
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float v = fmaxf(mx[half], __shfl_xor_sync(0xffffffffu, mx[half], 1));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
          v = fmaxf(v, m[half]);
          corr[half] = v == m[half] ? 1.0f : ex2(m[half] - v);
          m[half] = v;
          l[half] *= corr[half];
        }
#pragma unroll
        for (int j = 0; j < D / 8; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[j][e] *= corr[e >> 1];
      }
      uint32_t pf[4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const float ref = m[half] == -INFINITY ? 0.0f : m[half];
          const float x0 = ex2(s[i][2 * half] - ref), x1 = ex2(s[i][2 * half + 1] - ref);
          l[half] += x0 + x1;
          pf[2 * i + half] = pack_f16x2(x0, x1);
        }
      // values: token pairs (2 c, 2 c + 1) of each column tile, columns g D / 8 + j
      uint32_t vsc[2], v[2][2][D / 64];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t by[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int row = M::token(i, c, e);
          by[e] = D == 128 ? st[M::kVsOff + row * 8 + g] : st[M::kVsOff + row * 4 + (g >> 1)];
          if (edge && first + row >= len) by[e] = 0;
          if constexpr (D == 128) {
            const uint2 u = *reinterpret_cast<const uint2*>(st + M::kVOff + row * 64 + ((8 * g) ^ ((row & 2) * 16)));
            v[i][e][0] = u.x;
            v[i][e][1] = u.y;
          } else {
            v[i][e][0] = *reinterpret_cast<const uint32_t*>(st + M::kVOff + row * 32 + 4 * g);
          }
        }
        vsc[i] = e4m3x2_f16(by[0] | by[1] << 8);
      }
#pragma unroll
      for (int w = 0; w < D / 64; ++w) {
        uint32_t x[2][2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) e2m1x8_f16(v[i][e][w], x[i][e]);
#pragma unroll
        for (int b = 0; b < 4; ++b) {
          mma16816(o[8 * w + 2 * b], pf, hmul2(__byte_perm(x[0][0][b], x[0][1][b], 0x5410), vsc[0]),
                   hmul2(__byte_perm(x[1][0][b], x[1][1][b], 0x5410), vsc[1]));
          mma16816(o[8 * w + 2 * b + 1], pf, hmul2(__byte_perm(x[0][0][b], x[0][1][b], 0x7632), vsc[0]),
                   hmul2(__byte_perm(x[1][0][b], x[1][1][b], 0x7632), vsc[1]));
        }
      }
    }
    cp_async_wait<0>();

    // join the four warps: a common maximum per row, each warp's O in its ring
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 1);
      l[half] += __shfl_xor_sync(0xffffffffu, l[half], 2);
      if (c == 0) {
        sm_m[warp][g + 8 * half] = m[half];
        sm_l[warp][g + 8 * half] = l[half];
      }
    }
    __syncthreads();
    float* own = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int r = g + 8 * half;
      float top = sm_m[0][r];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm_m[w][r]);
      const float f = m[half] == top ? 1.0f : ex2(m[half] - top);
      // column c D / 4 + y is element 2 (y / (D / 8)) + ... : tile y % (D / 8), pair member y / (D / 8)
#pragma unroll
      for (int y = 0; y < D / 4; y += 4) {
        const int e = 2 * half + y / (D / 8), j = y % (D / 8);
        *reinterpret_cast<float4*>(own + o_at<D>(r, c * (D / 16) + y / 4)) =
            make_float4(o[j][e] * f, o[j + 1][e] * f, o[j + 2][e] * f, o[j + 3][e] * f);
      }
    }
    __syncthreads();
    const bool whole = p0 == 0 && p1 == at.pages;
    const int slot = 2 * blockIdx.x + (x == begin ? 0 : 1);
    {
      const int r = threadIdx.x >> 3, part = threadIdx.x & 7;  // 16 rows, 8 threads each
      const int row = at.tile * 16 + r;
      if (row < a.rows) {
        float top = sm_m[0][r], sum = 0.0f;
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm_m[w][r]);
#pragma unroll
        for (int w = 0; w < kWarps; ++w) sum += sm_l[w][r] * (sm_m[w][r] == top ? 1.0f : ex2(sm_m[w][r] - top));
        const float inv = sum == 0.0f ? 0.0f : a.c.v_sg / sum;
        T* dst = static_cast<T*>(a.out) +
                 ((static_cast<int64_t>(at.s) * a.q_len + row / a.group) * a.heads + at.kvh * a.group + row % a.group) * D;
#pragma unroll
        for (int k = 0; k < D / 32; ++k) {
          const int quad = part + 8 * k;
          float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 u = *reinterpret_cast<const float4*>(
                reinterpret_cast<const float*>(ring_base + w * kStages * M::kBytes) + o_at<D>(r, quad));
            t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
          }
          if (whole)
            store4<T>(dst + quad * 4, t.x * inv, t.y * inv, t.z * inv, t.w * inv);
          else
            *reinterpret_cast<float4*>(a.part_o + (static_cast<int64_t>(slot) * 16 + r) * D + quad * 4) = t;
        }
        if (part == 0) {
          if (!whole) a.part_ml[slot * 16 + r] = make_float2(top, sum);
          if (whole && a.lse != nullptr)
            a.lse[(static_cast<int64_t>(at.s) * a.c.kv_heads + at.kvh) * a.rows + row] =
                sum == 0.0f ? INFINITY : top + log2f(sum);
        }
      }
    }
    __syncthreads();
    x += p1 - p0;
  }
}

// Joins the partial sums of one row of a unit that was cut: a CTA per row,
// the runs strided over its warps, each lane four columns.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_combine_kernel(const Args a) {
  griddep_wait();
  griddep_launch_dependents();
  __shared__ float sm_o[kWarps][D];
  __shared__ float2 sm_ml[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.y, tile = row / 16, r = row % 16;
  const int s = blockIdx.x / a.c.kv_heads, kvh = blockIdx.x % a.c.kv_heads;
  const int per_seq = a.c.kv_heads * a.row_tiles;
  const int64_t total = static_cast<int64_t>(a.prefix[a.c.n_seqs]) * per_seq;
  const int64_t chunk = max(static_cast<int64_t>(kMinPages), (total + a.grid - 1) / a.grid);
  const int pages = a.prefix[s + 1] - a.prefix[s];
  const int64_t lo = static_cast<int64_t>(a.prefix[s]) * per_seq + static_cast<int64_t>(kvh * a.row_tiles + tile) * pages;
  const int64_t i0 = lo / chunk, i1 = (lo + pages - 1) / chunk;
  float* lse = a.lse == nullptr ? nullptr : a.lse + (static_cast<int64_t>(s) * a.c.kv_heads + kvh) * a.rows + row;
  if (pages == 0) {
    if (lse != nullptr && threadIdx.x == 0) *lse = INFINITY;
    return;
  }
  if (i0 == i1) return;  // one run held the unit: done there
  auto slot = [&](int64_t i) { return 2 * i + (i * chunk >= lo ? 0 : 1); };
  float top = -INFINITY;
  for (int64_t i = i0 + lane; i <= i1; i += 32) top = fmaxf(top, a.part_ml[slot(i) * 16 + r].x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.0f;
  const bool mine = lane * 4 < D;
#pragma unroll 4
  for (int64_t i = i0 + warp; i <= i1; i += kWarps) {
    const float2 ml = a.part_ml[slot(i) * 16 + r];
    const float f = ml.x == top ? 1.0f : ex2(ml.x - top);
    sum += ml.y * f;
    if (mine) {
      const float4 u = *reinterpret_cast<const float4*>(a.part_o + (slot(i) * 16 + r) * D + lane * 4);
      t.x += u.x * f; t.y += u.y * f; t.z += u.z * f; t.w += u.w * f;
    }
  }
  if (mine) *reinterpret_cast<float4*>(&sm_o[warp][lane * 4]) = t;
  if (lane == 0) sm_ml[warp].y = sum;
  __syncthreads();
  if (warp != 0) return;
  sum = 0.0f;
  t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    sum += sm_ml[w].y;
    if (mine) {
      const float4 u = *reinterpret_cast<const float4*>(&sm_o[w][lane * 4]);
      t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
    }
  }
  const float inv = sum == 0.0f ? 0.0f : a.c.v_sg / sum;
  if (mine)
    store4<T>(static_cast<T*>(a.out) +
                     ((static_cast<int64_t>(s) * a.q_len + row / a.group) * a.heads + kvh * a.group + row % a.group) * D +
                     lane * 4,
                 t.x * inv, t.y * inv, t.z * inv, t.w * inv);
  if (lse != nullptr && lane == 0) *lse = sum == 0.0f ? INFINITY : top + log2f(sum);
}

// weights[s, kvh, j] += sum over the rows of 2^(logit - lse): the logits once
// more from the keys alone (half the cache's bytes; storing them in the first
// kernel would cost 8 bytes per row and token). One warp owns a slice and sums
// its rows in a fixed order, so no atomics.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv4_weights_kernel(const Args a) {
  using M = Map<D>;
  using L = Kv4Layout<D>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int warp_sum[kWarps];
  int* prefix = reinterpret_cast<int*>(smem + kWarps * kStages * M::kBytes);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * kStages * M::kBytes;
  const uint32_t ring_s = smem_u32(ring);
  griddep_wait();
  griddep_launch_dependents();
  const Plan plan = make_plan(a.c, a.c.kv_heads, gridDim.x, prefix, warp_sum, nullptr);
  const int64_t begin = blockIdx.x * plan.chunk;
  const int64_t end = min(plan.total, begin + plan.chunk);
  for (int64_t x = begin; x < end;) {
    const Place at = place_of(prefix, a.c.n_seqs, a.c.kv_heads, 1, x);
    const int p0 = at.page;
    const int p1 = static_cast<int>(min(static_cast<int64_t>(at.pages), p0 + (end - x)));
    const int len = kv4_len(a.c, at.s, nullptr);
    const int open = len - a.q_len + 1;
    const float* lse = a.lse + (static_cast<int64_t>(at.s) * a.c.kv_heads + at.kvh) * a.rows;
    float* dst = a.weights + (static_cast<int64_t>(at.s) * a.c.kv_heads + at.kvh) * a.c.max_pages * kKv4Page;
    uint32_t qf[D / 16][4];
    float factor[2], norm[2];
    auto rows_of = [&](int tile) {
      load_q<T, D>(a, at.s, at.kvh, tile * 16, qf, factor);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int row = tile * 16 + g + 8 * half;
        norm[half] = row < a.rows ? lse[row] : INFINITY;
      }
    };
    rows_of(0);
    int ids = 0, ids_at = p0;
    auto issue = [&](int p) {
      if (p < p1) {
        if (p >= ids_at + 32 || p == p0) {
          ids_at = p;
          ids = p + lane < p1 ? static_cast<int>(kv4_page(a.c, at.s, p + lane, a.status)) : 0;
        }
        const int id = __shfl_sync(0xffffffffu, ids, p - ids_at);
        if (p * kKv4Page + warp * kSlice < len)
          fetch<D, false>(ring_s + (p - p0) % kStages * M::kBytes,
                          a.c.pages + (static_cast<int64_t>(id) * a.c.kv_heads + at.kvh) * L::kBytes, warp);
      }
      cp_async_commit();
    };
#pragma unroll
    for (int j = 0; j < kStages - 1; ++j) issue(p0 + j);
    for (int p = p0; p < p1; ++p) {
      cp_async_wait<kStages - 2>();
      __syncwarp();
      const uint8_t* st = ring + (p - p0) % kStages * M::kBytes;
      issue(p + kStages - 1);
      const int first = p * kKv4Page + warp * kSlice;
      if (first >= len) continue;
      float w[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};  // [column tile][pair member]
      for (int tile = 0; tile < a.row_tiles; ++tile) {
        if (a.row_tiles > 1) rows_of(tile);
        float s[2][4];
        logits<D>(st, qf, s);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int half = e >> 1;
            const int row = tile * 16 + g + 8 * half;
            const bool sees = first + M::token(i, c, e & 1) < open + row / a.group;
            const float p2 = ex2(s[i][e] * factor[half] - norm[half]);
            w[i][e & 1] += sees && row < a.rows ? p2 : 0.0f;
          }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float v = w[i][e];
          v += __shfl_xor_sync(0xffffffffu, v, 4);
          v += __shfl_xor_sync(0xffffffffu, v, 8);
          v += __shfl_xor_sync(0xffffffffu, v, 16);
          const int j = first + M::token(i, c, e);
          if (g == 0 && j < len) dst[j] += v;
        }
    }
    cp_async_wait<0>();
    __syncwarp();
    x += p1 - p0;
  }
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

}  // namespace

size_t kv4_attention_workspace(int n_seqs, int heads, int kv_heads, int head_dim, int q_len) {
  (void)kv_heads;
  const size_t n = std::min(n_seqs, kMaxSeqs);
  const size_t slots = 2 * static_cast<size_t>(kCtasPerSm) * 256;  // 256: above any SM count
  return up((n + 1) * 4) + up(slots * 16 * head_dim * 4) + up(slots * 16 * 8) + up(n * heads * q_len * 4);
}

int launch_kv4_attention(const Kv4& c0, int head_dim, int heads, int q_len, int dtype, const void* q, int64_t q_stride,
                         float scale, void* out, float* weights, void* ws, int32_t* status, cudaStream_t s) {
  Args a;
  a.q_stride = q_stride;
  a.heads = heads;
  a.group = heads / c0.kv_heads;
  a.q_len = q_len;
  a.rows = a.group * q_len;
  a.row_tiles = (a.rows + 15) / 16;
  a.scale = scale;
  a.grid = kCtasPerSm * std::min(num_sms(), 256);
  a.status = status;
  const size_t slots = 2 * static_cast<size_t>(kCtasPerSm) * 256;
  const int n_max = std::min(c0.n_seqs, kMaxSeqs);
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.prefix = reinterpret_cast<int32_t*>(w);
  w += up((static_cast<size_t>(n_max) + 1) * 4);
  a.part_o = reinterpret_cast<float*>(w);
  w += up(slots * 16 * head_dim * 4);
  a.part_ml = reinterpret_cast<float2*>(w);
  w += up(slots * 16 * 8);
  a.lse = weights == nullptr ? nullptr : reinterpret_cast<float*>(w);
  const size_t smem = kWarps * kStages * (head_dim == 128 ? Map<128>::kBytes : Map<64>::kBytes) +
                      (static_cast<size_t>(n_max) + 1) * 4;
  auto run = [&](auto attn, auto combine, auto weigh, int elem) -> int {
    if (smem > 48 * 1024) {
      if (cudaFuncSetAttribute(attn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess ||
          cudaFuncSetAttribute(weigh, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem)) != cudaSuccess)
        return VLM_ERR_CUDA;
    }
    for (int first = 0; first < c0.n_seqs; first += kMaxSeqs) {
      a.c = c0;
      a.c.n_seqs = std::min(kMaxSeqs, c0.n_seqs - first);
      a.c.table += static_cast<int64_t>(first) * c0.max_pages;
      a.c.lens += first;
      a.q = static_cast<const uint8_t*>(q) + static_cast<int64_t>(first) * q_len * q_stride * elem;
      a.out = static_cast<uint8_t*>(out) + static_cast<int64_t>(first) * q_len * heads * head_dim * elem;
      a.weights = weights == nullptr
                      ? nullptr
                      : weights + static_cast<int64_t>(first) * c0.kv_heads * c0.max_pages * kKv4Page;
      cudaError_t e = launch_pdl(attn, dim3(a.grid), dim3(kThreads), smem, s, a);
      if (e == cudaSuccess)
        e = launch_pdl(combine, dim3(a.c.n_seqs * a.c.kv_heads, a.rows), dim3(kThreads), 0, s, a);
      if (e == cudaSuccess && weights != nullptr) e = launch_pdl(weigh, dim3(a.grid), dim3(kThreads), smem, s, a);
      if (e != cudaSuccess) return VLM_ERR_CUDA;
    }
    return VLM_OK;
  };
  launch_begin(KC_KV4_ATTN, s);
  int rc;
  if (dtype == VLM_DTYPE_F16)
    rc = head_dim == 128 ? run(kv4_attn_kernel<__half, 128>, kv4_combine_kernel<__half, 128>, kv4_weights_kernel<__half, 128>, 2)
                         : run(kv4_attn_kernel<__half, 64>, kv4_combine_kernel<__half, 64>, kv4_weights_kernel<__half, 64>, 2);
  else
    rc = head_dim == 128 ? run(kv4_attn_kernel<__nv_bfloat16, 128>, kv4_combine_kernel<__nv_bfloat16, 128>,
                               kv4_weights_kernel<__nv_bfloat16, 128>, 2)
                         : run(kv4_attn_kernel<__nv_bfloat16, 64>, kv4_combine_kernel<__nv_bfloat16, 64>,
                               kv4_weights_kernel<__nv_bfloat16, 64>, 2);
  launch_end(KC_KV4_ATTN, s);
  note_extra_launches(((c0.n_seqs + kMaxSeqs - 1) / kMaxSeqs) * (weights != nullptr ? 3 : 2) - 1);
  return rc;
}

}  // namespace vlm
