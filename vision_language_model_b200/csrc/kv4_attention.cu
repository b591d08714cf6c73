// Attention of a few new tokens over the paged 4-bit cache (layout in kv4.cuh).
// Sequence s has len tokens in the cache, its m new ones last; new token i
// sees the places j <= len - m + i:
//   o_i = sum_j p_ij v_j,  p_ij = softmax_j(scale q_i . k_j)
// for the G = heads / kv_heads query heads of every key head.
//
// Bound: the codes are read once, 9/8 byte per column and head, so the floor
// is HBM; what competes with it is the issue rate of turning codes into
// operands. The layout of the work:
//   - The products run as mma.m16n8k16 (fp16 operands, fp32 sums) with the
//     tokens (S^T = K q^T) and the value columns (O^T = V^T P^T) as the 16 rows
//     and the G * m query rows of one (sequence, key head) as the 8 columns, two
//     such tiles for more than 8 rows, further row tiles for more than 16. So
//     what is made from codes is the big operand, made once in registers, which
//     tcgen05 cannot take; at these few rows the product is far from its rate.
//   - A warp takes half pages, 32 tokens, by bulk copies into a ring of its own
//     in shared memory, so no warp waits for another.
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
#include <cfloat>

#include <algorithm>

#include "kv4.cuh"
#include "softmax.cuh"

namespace vlm {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kPart = 32;  // tokens of a page that a warp takes at a time
constexpr int kMaxSeqs = 4096;  // sequences per launch (their page offsets are held in shared memory)
constexpr int kMaxCtasPerSm = 4;
// registers: O and q take 48 per lane for one 8-row tile, 96 for two
template <int NT>
constexpr int kCtasPerSm = NT == 1 ? 4 : 3;
constexpr int kMinPages = 4;  // a run shorter than this costs more to join than it gains
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNoMax = -3.0e38f;  // a row's maximum before it sees a place; finite, so that -inf minus it is no NaN
constexpr float kRescale = 8.0f;  // log2 units; P stays below 2^8

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// The transpose of an 8 x 8 tile of 16-bit values (row g in lanes 4 g .. 4 g + 3, two columns each).
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
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
  int heads, group, q_len, rows, tile_rows, row_tiles;
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

// Fragment maps. Lane = 4 g + c. Row 8 i + 2 c + e of the 16 tokens of an mma
// tile is token 8 i + 4 e + (c ^ x e): x (1 for D = 128, 2 for D = 64) spreads
// the rows that one shared-memory load touches over the banks (the value rows
// at D = 128 still meet two at a time). As S^T's rows a lane has tokens g and
// g + 8 (numbered so), as V^T's columns tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9.
// A lane's elements of key and query rows are the D / 4 columns from c D / 4 on,
// its value columns (rows of O^T) the D / 8 from g D / 8 on, its query rows (the
// mma columns of S^T and O^T) 2 c and 2 c + 1 of each 8-row tile.
template <int D>
struct Map {
  static constexpr int kX = D == 128 ? 1 : 2;
  static constexpr int kSteps = D / 16;  // mma steps of a logit
  static constexpr int kCols = D / 4;    // columns per lane
  // a ring slot: 32 tokens as key codes, value codes, key scales, value scales
  static constexpr int kV = kPart * D / 2, kKs = 2 * kV, kVs = kKs + kPart * D / 16;
  static constexpr int kBytes = kVs + kPart * D / 16;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr int kRing = kStages * kBytes;  // bytes per warp
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

// The query rows [first, first + 8 NT) of (sequence, key head) as mma B
// fragments, and the factors of the logits of the lane's rows 2 c, 2 c + 1.
template <typename T, int D, int NT>
__device__ __forceinline__ void load_q(const Args& a, int s, int kvh, int first, uint32_t (&qf)[NT][D / 16][2],
                                       float (&factor)[NT][2]) {
  using M = Map<D>;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int r = first + 8 * n + g;
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
    const float mine = fmaxf(a.scale * a.c.k_sg * kLog2e / mul, FLT_MIN);  // not 0: it multiplies -inf
    factor[n][0] = __shfl_sync(0xffffffffu, mine, 8 * c);
    factor[n][1] = __shfl_sync(0xffffffffu, mine, 8 * c + 4);
#pragma unroll
    for (int k = 0; k < M::kSteps; ++k) {
      const float2 f0 = unpack16<T>(w[2 * k]), f1 = unpack16<T>(w[2 * k + 1]);
      qf[n][k][0] = pack_f16x2(f0.x * mul, f0.y * mul);
      qf[n][k][1] = pack_f16x2(f1.x * mul, f1.y * mul);
    }
  }
}

// The halves of a run's pages that a warp takes, every kWarps-th, through its
// ring: four bulk copies each, one by each of the lanes 0..3, counted on one
// barrier. All lanes call together. kWarps is even, so a warp takes the same
// half of every page and a copy's place inside the page never changes.
template <int D>
struct PartRing {
  static_assert(kWarps % 2 == 0, "one half per warp");
  uint32_t bars;        // shared-memory address of the barriers
  uint32_t dst, bytes;  // this lane's copy: into slot 0, its size
  uint32_t src;         // its offset in a page
  uint32_t issued = 0, taken = 0;
  __device__ __forceinline__ PartRing(uint32_t ring, uint32_t bars_, int half, int lane) : bars(bars_) {
    using M = Map<D>;
    using L = Kv4Layout<D>;
    const int which = lane & 1;
    const bool codes = (lane & 2) == 0;
    bytes = codes ? M::kV : M::kVs - M::kKs;
    src = codes ? which * L::kV + half * M::kV : L::kKs + which * (L::kVs - L::kKs) + half * (M::kVs - M::kKs);
    dst = ring + (codes ? which * M::kV : M::kKs + which * (M::kVs - M::kKs));
  }
  __device__ __forceinline__ void issue(const uint8_t* page, int lane) {
    using M = Map<D>;
    const uint32_t st = issued % M::kStages, bar = bars + st * 8;
    if (lane == 0) mbar_arrive_expect_tx(bar, M::kBytes);
    __syncwarp();
    if (lane < 4)
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                       dst + st * M::kBytes),
                   "l"(page + src), "r"(bytes), "r"(bar)
                   : "memory");
    ++issued;
  }
  __device__ __forceinline__ bool wait(volatile int* abort, int32_t* status) const {
    constexpr uint32_t n = Map<D>::kStages;
    return mbar_wait_warp(bars + taken % n * 8, (taken / n) & 1, abort, status);
  }
};

// S^T = (code * scale) . q for the 32 tokens of a ring slot: s[x][n] is 16
// tokens by 8 query rows.
template <int D, int NT>
__device__ __forceinline__ void logits(const uint8_t* part, const uint32_t (&qf)[NT][D / 16][2], float (&s)[2][NT][4]) {
  using M = Map<D>;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    uint32_t w[2][D / 32], sc[2][D == 128 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 16 * x + M::token(i, g >> 1, g & 1);
      if constexpr (D == 128) {
        const uint4 u = *reinterpret_cast<const uint4*>(part + row * 64 + c * 16);
        w[i][0] = u.x; w[i][1] = u.y; w[i][2] = u.z; w[i][3] = u.w;
        const uint32_t h2 = e4m3x2_f16(*reinterpret_cast<const uint16_t*>(part + M::kKs + row * 8 + 2 * c));
        sc[i][0] = __byte_perm(h2, 0, 0x1010);
        sc[i][1] = __byte_perm(h2, 0, 0x3232);
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(part + row * 32 + c * 8);
        w[i][0] = u.x; w[i][1] = u.y;
        const uint32_t h2 = e4m3x2_f16(part[M::kKs + row * 4 + c]);
        sc[i][0] = __byte_perm(h2, 0, 0x1010);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[x][n][j] = 0.0f;
#pragma unroll
    for (int y = 0; y < D / 32; ++y) {
      uint32_t p[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        e2m1x8_f16(w[i][y], p[i]);
        const uint32_t f = sc[i][D == 128 ? y >> 1 : 0];
#pragma unroll
        for (int j = 0; j < 4; ++j) p[i][j] = hmul2(p[i][j], f);
      }
      const uint32_t a0[4] = {p[0][0], p[1][0], p[0][1], p[1][1]}, a1[4] = {p[0][2], p[1][2], p[0][3], p[1][3]};
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        mma16816(s[x][n], a0, qf[n][2 * y][0], qf[n][2 * y][1]);
        mma16816(s[x][n], a1, qf[n][2 * y + 1][0], qf[n][2 * y + 1][1]);
      }
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
// floats; the exchange spreads the rows that one store touches over the banks.
template <int D>
__device__ __forceinline__ int o_at(int row, int quad) {
  const int c = row >> 1;
  return row * D + ((quad ^ (D == 128 ? c & 3 : (c & 1) | ((c & 2) << 1))) * 4);
}

template <typename T>
__device__ __forceinline__ void store4(T* dst, float x, float y, float z, float w) {
  *reinterpret_cast<uint2*>(dst) = make_uint2(pack16<T>(x, y), pack16<T>(z, w));
}

// A lane's running state of its query rows 2 c and 2 c + 1 of each tile: O, the
// rows' maxima (of the products, before `factor`: a rounded product would not do
// for large ones) and its part of their sums.
template <int D, int NT>
struct State {
  float o[NT][D / 16][4];
  float m[NT][2], grow[NT][2];  // the maximum moves when a product passes `grow`, kRescale above it in log2 units
  uint64_t l[NT];
};

// The 32 tokens of a ring slot, from place `first` on, into the state.
template <int D, int NT, bool kEdge>
__device__ __forceinline__ void take32(const uint8_t* part, int first, int len, const int (&seen)[NT][2],
                                       const uint32_t (&qf)[NT][D / 16][2], const float (&factor)[NT][2],
                                       State<D, NT>& z) {
  using M = Map<D>;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  float s[2][NT][4];
  logits<D, NT>(part, qf, s);
  if (kEdge) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = first + 16 * x + M::token(e >> 1, g >> 1, g & 1);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (j >= seen[n][e & 1]) s[x][n][e] = -INFINITY;
      }
  }
  bool grows = false;
  float mx[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      mx[n][r] = fmaxf(max3f(s[0][n][r], s[0][n][2 + r], s[1][n][r]), s[1][n][2 + r]);
      grows |= mx[n][r] > z.grow[n][r];
    }
  if (__any_sync(0xffffffffu, grows)) {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float corr[2];
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float v = mx[n][r];
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
        v = fmaxf(v, z.m[n][r]);
        corr[r] = ex2((z.m[n][r] - v) * factor[n][r]);
        z.m[n][r] = v;
        z.grow[n][r] = v + kRescale / factor[n][r];
      }
      z.l[n] = mul2(z.l[n], pack2(__float_as_uint(corr[0]), __float_as_uint(corr[1])));
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) z.o[n][j][e] *= corr[e & 1];
    }
  }
  uint32_t pf[2][NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint64_t f2 = pack2(__float_as_uint(factor[n][0]), __float_as_uint(factor[n][1]));
    const uint64_t negm = pack2(__float_as_uint(-z.m[n][0]), __float_as_uint(-z.m[n][1]));
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x0, x1;
        unpack2(mul2(add2(pack2(__float_as_uint(s[x][n][2 * i]), __float_as_uint(s[x][n][2 * i + 1])), negm), f2), x0, x1);
        x0 = ex2(x0);
        x1 = ex2(x1);
        z.l[n] = add2(z.l[n], pack2(__float_as_uint(x0), __float_as_uint(x1)));
        pf[x][n][i] = transpose8(pack_f16x2(x0, x1));
      }
  }
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    uint32_t vsc[2], v[2][2][D / 64];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t by[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 16 * x + M::token(i, c, e);
        by[e] = D == 128 ? part[M::kVs + row * 8 + g] : part[M::kVs + row * 4 + (g >> 1)];
        if (kEdge && first + row >= len) by[e] = 0;
        if constexpr (D == 128) {
          const uint2 u = *reinterpret_cast<const uint2*>(part + M::kV + row * 64 + 8 * g);
          v[i][e][0] = u.x;
          v[i][e][1] = u.y;
        } else {
          v[i][e][0] = *reinterpret_cast<const uint32_t*>(part + M::kV + row * 32 + 4 * g);
        }
      }
      vsc[i] = e4m3x2_f16(by[0] | by[1] << 8);
    }
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {
      // the two tokens' codes of one column side by side before they are converted:
      // even columns in y[i][0], odd ones in y[i][1]
      uint32_t y[2][2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        constexpr uint32_t m = 0x0F0F0F0Fu;
        e2m1x8_f16((v[i][0][w] & m) | ((v[i][1][w] << 4) & ~m), y[i][0]);
        e2m1x8_f16(((v[i][0][w] >> 4) & m) | (v[i][1][w] & ~m), y[i][1]);
      }
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        // columns g D / 8 + 8 w + 2 b (rows g of the tile) and + 1 (rows g + 8)
        const uint32_t at[4] = {hmul2(y[0][0][b], vsc[0]), hmul2(y[0][1][b], vsc[0]), hmul2(y[1][0][b], vsc[1]),
                                hmul2(y[1][1][b], vsc[1])};
#pragma unroll
        for (int n = 0; n < NT; ++n) mma16816(z.o[n][4 * w + b], at, pf[x][n][0], pf[x][n][1]);
      }
    }
  }
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<NT>) kv4_attn_kernel(const Args a) {
  using M = Map<D>;
  using L = Kv4Layout<D>;
  constexpr int kTileRows = 8 * NT;
  static_assert(M::kRing >= kTileRows * D * 4, "a warp's O tile fits its ring");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int warp_sum[kWarps];
  __shared__ float sm_m[kWarps][kTileRows], sm_l[kWarps][kTileRows];
  __shared__ uint64_t bars[kWarps][M::kStages];
  __shared__ int abort_flag;
  int* prefix = reinterpret_cast<int*>(smem + kWarps * M::kRing);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * M::kRing;
  PartRing<D> pr(smem_u32(ring), smem_u32(bars[warp]), warp & 1, lane);
  if (lane == 0) {
    for (int i = 0; i < M::kStages; ++i) mbar_init(smem_u32(&bars[warp][i]), 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) abort_flag = 0;
  volatile int* abort_v = &abort_flag;

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

  bool ok = true;
  const int64_t begin = blockIdx.x * plan.chunk;
  const int64_t end = min(plan.total, begin + plan.chunk);
  for (int64_t x = begin; x < end;) {
    const Place at = place_of(prefix, a.c.n_seqs, a.c.kv_heads, a.row_tiles, x);
    const int p0 = at.page;
    const int p1 = static_cast<int>(min(static_cast<int64_t>(at.pages), p0 + (end - x)));
    const int len = kv4_len(a.c, at.s, nullptr);

    // this warp's half pages 2 p0 + warp, + kWarps, ...: two of kWarps = 4 pages' eight;
    // the page numbers of the next 32 of them, one per lane
    const int mine = (2 * (p1 - p0) - warp + kWarps - 1) / kWarps;
    int ids = 0;
    auto issue = [&](int k) {  // k in order, all lanes together
      if (k % 32 == 0) {
        const int e = p0 + (warp + (k + lane) * kWarps) / 2;
        ids = e < p1 ? static_cast<int>(kv4_page(a.c, at.s, e, a.status)) : 0;
      }
      pr.issue(a.c.pages + (static_cast<int64_t>(__shfl_sync(0xffffffffu, ids, k % 32)) * a.c.kv_heads + at.kvh) * L::kBytes,
               lane);
    };
    int next = 0;
    for (; next < min(mine, M::kStages); ++next) issue(next);

    // the places below `open` are seen by every row
    const int open = len - a.q_len + 1;
    uint32_t qf[NT][M::kSteps][2];
    float factor[NT][2];
    load_q<T, D, NT>(a, at.s, at.kvh, at.tile * kTileRows, qf, factor);
    int seen[NT][2];  // one past the last place each of the lane's rows sees
    State<D, NT> z;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        seen[n][r] = open + (at.tile * kTileRows + 8 * n + 2 * c + r) / a.group;
        z.m[n][r] = z.grow[n][r] = kNoMax;
      }
      z.l[n] = 0;
#pragma unroll
      for (int j = 0; j < D / 16; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) z.o[n][j][e] = 0.0f;
    }

    for (int k = 0; k < mine; ++k) {
      if (ok) ok = pr.wait(abort_v, a.status);
      const uint8_t* part = ring + pr.taken % M::kStages * M::kBytes;
      const int first = p0 * kKv4Page + (warp + k * kWarps) * kPart;
      if (ok) {
        if (first + kPart <= open)
          take32<D, NT, false>(part, first, len, seen, qf, factor, z);
        else
          take32<D, NT, true>(part, first, len, seen, qf, factor, z);
      }
      ++pr.taken;
      __syncwarp();
      if (ok && next < mine) {
        issue(next);
        ++next;
      }
    }
    // join the four warps: a common maximum per row (in log2 units), each warp's O in its ring
    float m[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float l[2];
      unpack2(z.l[n], l[0], l[1]);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
        m[n][r] = z.m[n][r] == kNoMax ? -INFINITY : z.m[n][r] * factor[n][r];
        if (g == 0) {
          sm_m[warp][8 * n + 2 * c + r] = m[n][r];
          sm_l[warp][8 * n + 2 * c + r] = l[r];
        }
      }
    }
    __syncthreads();
    float* own = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = 8 * n + 2 * c + r;
        float top = sm_m[0][row];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) top = fmaxf(top, sm_m[w][row]);
        const float f = m[n][r] == top ? 1.0f : ex2(m[n][r] - top);
        // columns g D / 8 + 2 j (elements r) and + 1 (elements 2 + r) of tile j
#pragma unroll
        for (int j = 0; j < D / 16; j += 2)
          *reinterpret_cast<float4*>(own + o_at<D>(row, g * (D / 32) + j / 2)) =
              make_float4(z.o[n][j][r] * f, z.o[n][j][2 + r] * f, z.o[n][j + 1][r] * f, z.o[n][j + 1][2 + r] * f);
      }
    __syncthreads();
    const bool whole = p0 == 0 && p1 == at.pages;
    const int slot = 2 * blockIdx.x + (x == begin ? 0 : 1);
    {
      constexpr int kPer = kThreads / kTileRows;  // threads per row
      const int r = threadIdx.x / kPer, part = threadIdx.x % kPer;
      const int row = at.tile * kTileRows + r;
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
        for (int k = 0; k < D / 4 / kPer; ++k) {
          const int quad = part + kPer * k;
          float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < kWarps; ++w) {
            const float4 u = *reinterpret_cast<const float4*>(
                reinterpret_cast<const float*>(smem + w * M::kRing) + o_at<D>(r, quad));
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
    fence_proxy_async_smem();  // the O tiles were written where the next pages will be copied
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
  const int row = blockIdx.y, tile = row / a.tile_rows, r = row % a.tile_rows;
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
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<NT>) kv4_weights_kernel(const Args a) {
  using M = Map<D>;
  using L = Kv4Layout<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int warp_sum[kWarps];
  __shared__ uint64_t bars[kWarps][M::kStages];
  __shared__ int abort_flag;
  int* prefix = reinterpret_cast<int*>(smem + kWarps * M::kRing);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * M::kRing;
  PartRing<D> pr(smem_u32(ring), smem_u32(bars[warp]), warp & 1, lane);
  if (lane == 0) {
    for (int i = 0; i < M::kStages; ++i) mbar_init(smem_u32(&bars[warp][i]), 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) abort_flag = 0;
  volatile int* abort_v = &abort_flag;
  bool ok = true;
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
    uint32_t qf[NT][M::kSteps][2];
    float factor[NT][2], norm[NT][2];
    int seen[NT][2];
    auto rows_of = [&](int tile) {
      load_q<T, D, NT>(a, at.s, at.kvh, tile * 8 * NT, qf, factor);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = tile * 8 * NT + 8 * n + 2 * c + r;
          norm[n][r] = row < a.rows ? lse[row] : INFINITY;
          seen[n][r] = row < a.rows ? open + row / a.group : 0;
        }
    };
    rows_of(0);
    const int mine = (2 * (p1 - p0) - warp + kWarps - 1) / kWarps;
    int ids = 0;
    auto issue = [&](int k) {
      if (k % 32 == 0) {
        const int e = p0 + (warp + (k + lane) * kWarps) / 2;
        ids = e < p1 ? static_cast<int>(kv4_page(a.c, at.s, e, a.status)) : 0;
      }
      pr.issue(a.c.pages + (static_cast<int64_t>(__shfl_sync(0xffffffffu, ids, k % 32)) * a.c.kv_heads + at.kvh) * L::kBytes,
               lane);
    };
    int next = 0;
    for (; next < min(mine, M::kStages); ++next) issue(next);
    for (int k = 0; k < mine; ++k) {
      if (ok) ok = pr.wait(abort_v, a.status);
      const uint8_t* part = ring + pr.taken % M::kStages * M::kBytes;
      const int first = p0 * kKv4Page + (warp + k * kWarps) * kPart;
      if (ok && first < len) {
        float w[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};  // tokens g and g + 8 of both tiles
        for (int tile = 0; tile < a.row_tiles; ++tile) {
          if (a.row_tiles > 1) rows_of(tile);
          float s[2][NT][4];
          logits<D, NT>(part, qf, s);
#pragma unroll
          for (int x = 0; x < 2; ++x)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int j = first + 16 * x + M::token(e >> 1, g >> 1, g & 1);
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const float p2 = ex2(__fmul_rn(s[x][n][e], factor[n][e & 1]) - norm[n][e & 1]);
                w[x][e >> 1] += j < seen[n][e & 1] ? p2 : 0.0f;
              }
            }
        }
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float v = w[x][i];
            v += __shfl_xor_sync(0xffffffffu, v, 1);
            v += __shfl_xor_sync(0xffffffffu, v, 2);
            const int j = first + 16 * x + M::token(i, g >> 1, g & 1);
            if (c == 2 * x + i && j < len) dst[j] += v;
          }
      }
      ++pr.taken;
      __syncwarp();
      if (ok && next < mine) {
        issue(next);
        ++next;
      }
    }
    x += p1 - p0;
  }
}

size_t up(size_t x) { return (x + 255) / 256 * 256; }

// Opts the kernels in to their shared memory (static parts included, more than
// 48 KB), once per device.
template <typename T, int D, int NT>
bool smem_ready() {
  static bool done[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev < 64 && done[dev]) return true;
  constexpr int most = kWarps * Map<D>::kRing + (kMaxSeqs + 1) * 4;
  if (cudaFuncSetAttribute(kv4_attn_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
      cudaFuncSetAttribute(kv4_weights_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
    return false;
  if (dev < 64) done[dev] = true;
  return true;
}

}  // namespace

size_t kv4_attention_workspace(int n_seqs, int heads, int kv_heads, int head_dim, int q_len) {
  (void)kv_heads;
  const size_t n = std::min(n_seqs, kMaxSeqs);
  const size_t slots = 2 * static_cast<size_t>(kMaxCtasPerSm) * 256;  // 256: above any SM count
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
  // one 8-row tile holds the rows, or tiles of 16 (two of 8 that share the operand made from codes)
  const bool one = a.rows <= 8;
  a.tile_rows = one ? 8 : 16;
  a.row_tiles = (a.rows + a.tile_rows - 1) / a.tile_rows;
  a.scale = scale;
  a.grid = (one ? kCtasPerSm<1> : kCtasPerSm<2>) * std::min(num_sms(), 256);
  a.status = status;
  const size_t slots = 2 * static_cast<size_t>(kMaxCtasPerSm) * 256;
  const int n_max = std::min(c0.n_seqs, kMaxSeqs);
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.prefix = reinterpret_cast<int32_t*>(w);
  w += up((static_cast<size_t>(n_max) + 1) * 4);
  a.part_o = reinterpret_cast<float*>(w);
  w += up(slots * 16 * head_dim * 4);
  a.part_ml = reinterpret_cast<float2*>(w);
  w += up(slots * 16 * 8);
  a.lse = weights == nullptr ? nullptr : reinterpret_cast<float*>(w);
  const size_t smem = kWarps * (head_dim == 128 ? Map<128>::kRing : Map<64>::kRing) +
                      (static_cast<size_t>(n_max) + 1) * 4;
  auto run = [&](auto attn, auto combine, auto weigh, int elem, bool ready) -> int {
    if (!ready) return VLM_ERR_CUDA;
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
  auto pick = [&](auto type, auto dim, auto nt) {
    using T = decltype(type);
    constexpr int D = decltype(dim)::value, NT = decltype(nt)::value;
    return run(kv4_attn_kernel<T, D, NT>, kv4_combine_kernel<T, D>, kv4_weights_kernel<T, D, NT>, 2, smem_ready<T, D, NT>());
  };
  auto by_rows = [&](auto type, auto dim) {
    return one ? pick(type, dim, std::integral_constant<int, 1>()) : pick(type, dim, std::integral_constant<int, 2>());
  };
  auto by_dim = [&](auto type) {
    return head_dim == 128 ? by_rows(type, std::integral_constant<int, 128>()) : by_rows(type, std::integral_constant<int, 64>());
  };
  const int rc = dtype == VLM_DTYPE_F16 ? by_dim(__half()) : by_dim(__nv_bfloat16());
  launch_end(KC_KV4_ATTN, s);
  note_extra_launches(((c0.n_seqs + kMaxSeqs - 1) / kMaxSeqs) * (weights != nullptr ? 3 : 2) - 1);
  return rc;
}

}  // namespace vlm
