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
//   - A warp works on its own run of pages, one bulk copy each into a ring of its
//     own in shared memory: no warp waits for another, at the ends of runs neither.
//     With one 8-row tile it takes a page's 64 tokens at once, which gives four
//     independent chains of products to fill the pipes with.
//   - Code times block scale has at most 6 significant bits, so fp16 holds it
//     exactly: one cvt and one multiply per two values, no rounding. A query
//     row is scaled by a power of two so that its largest value lies in [1, 2)
//     and rounded to fp16: bf16 has 8 significant bits, so only values below
//     2^-14 of the row's largest lose bits, 2^-25 of the largest at most --
//     what an fp32 sum loses as well. The global scales, 1 / that power and
//     log2(e) are one fp32 factor of the logit.
//   - P is rounded to fp16 for the second product. It is made 2^7 times as large,
//     up to fp16's largest powers of two: half a step, 2^-11, down to 2^-21 of the
//     row's largest weight so far, and 2^-32 of that below, so that a long tail of
//     small weights beside a large one keeps its sum (made as it is, everything
//     under 2^-25 became 0). The sum of a row's weights, its maximum and both
//     products' sums stay in fp32.
//   - Work is cut into equal runs of pages, one per warp, over the flattened
//     (sequence, key head, row tile, page) list, whatever the lengths (a unit's
//     start counts as two pages more), computed on the device from the lengths
//     there, so a captured graph replays with other lengths.
//     A unit (sequence, key head, row tile) cut by a border leaves partial sums
//     that kv4_combine_kernel joins in the order of the runs: the result does
//     not depend on timing (its last bits do on where the batch was cut).
// Measured (a graph of the call replayed), 32/8 heads of 128: 31 sequences of up to
// 16,000 tokens (378 MB) 74 us, of which the join is 4 to 5; 131,072, 131,071, 98,304
// and 77 (415 MB) 80 us, 5.2 TB/s (0.79 of the copy rate). What it lacks is issue
// slots, 58% used, 430 instructions per 32 tokens of a head of which 256 convert and
// scale. As 16-row tiles of S and O it took 104 us. For the weights, logits stored in
// fp32 would cost 8 bytes per row and token; they are made again from the keys.
// Places behind what a row sees get logit -inf; value scales of places behind
// the sequence's end are taken as 0, so stale bytes (NaN scales among them)
// reach no sum. A row that sees nothing is 0, one whose logits are all -inf NaN.
#include <cfloat>

#include <algorithm>

#include "kv4.cuh"
#include "softmax.cuh"

namespace vlm {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxSeqs = 4096;  // sequences per launch (their page offsets are held in shared memory)
// 168 registers; four CTAs would have to spill. Three also have room for the offsets of some
// 740 sequences in their shared memory (by clusters of 90); with more in a launch two are
// resident, and the last third of the grid follows them.
constexpr int kCtasPerSm = 3;
constexpr int kCluster = 8;       // CTAs that share a unit of a small batch
constexpr int kClusterPages = 128;  // and the pages a sequence may then have: four per warp
constexpr int kMinPages = 1;  // of a run: a page takes a warp about 1 us, joining a run less
constexpr int kUnitPages = 2;  // pages that starting a unit counts as where the work is cut
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kNoMax = -3.0e38f;  // a row's maximum before it sees a place; finite, so that -inf minus it is no NaN
constexpr float kRescale = 8.0f;  // log2 units; weights stay below 2^8 of their maximum
constexpr float kLift = 7.0f;     // log2 units that P, O and the sums are larger by: P stays below 2^15

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
  int32_t* prefix;   // [n_seqs + 1] sequences' offsets in the cut, written by the first kernel's CTA 0
  float* part_o;     // [2 * runs][tile_rows][D]
  float4* part_ml;   // [2 * runs][tile_rows] maximum of the products (-inf: none seen), sum, the row's factor
  float2* stats;     // [n_seqs, kv_heads, rows] a row's maximum and 1 / its sum of weights (null: not wanted)
  float* weights;    // [n_seqs, kv_heads, max_pages * 64]
  int runs;          // warps of the first kernel
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
  static constexpr int kStages = D == 128 ? 2 : 4;              // pages in a warp's ring
  static constexpr int kRing = kStages * Kv4Layout<D>::kBytes;  // bytes per warp
  static __device__ __forceinline__ int token(int i, int c, int e) { return 8 * i + 4 * e + (c ^ (kX * e)); }
};

struct Plan {
  int64_t total, chunk;
};

// A unit's length in the cut: its pages behind kUnitPages without work, which stand for
// what it costs to start one. (Without them the warp that got a short sequence's eight
// units, two pages each, finished last: 131,072, 131,071, 77 and 98,304 places 104 us, with
// one page 87, with two 80, with three 80; 31 ragged sequences 79, 77, 76, 76.)
__device__ __forceinline__ int cut_length(int len) {
  return len == 0 ? 0 : (len + kKv4Page - 1) / kKv4Page + kUnitPages;
}

// The sequences' offsets into shared memory (prefix[n_seqs + 1], units_per_seq to be
// multiplied) and the cut.
__device__ __forceinline__ Plan make_plan(const Kv4& c, int units_per_seq, int runs, int* prefix, int* warp_sum,
                                          int32_t* status) {
  const int n = c.n_seqs, per = (n + kThreads - 1) / kThreads;
  const int lo = min(n, static_cast<int>(threadIdx.x) * per), hi = min(n, lo + per);
  int sum = 0;
  for (int s = lo; s < hi; ++s) sum += cut_length(kv4_len(c, s, status));
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
    base += cut_length(kv4_len(c, s, nullptr));
  }
  if (hi == n && lo < n) prefix[n] = base;
  __syncthreads();
  Plan p;
  p.total = static_cast<int64_t>(prefix[n]) * units_per_seq;
  p.chunk = max(static_cast<int64_t>(kMinPages), (p.total + runs - 1) / runs);
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
    // not 0 and not infinite: it multiplies -inf and differences of 0
    const float mine = fminf(fmaxf(a.scale * a.c.k_sg * kLog2e / mul, FLT_MIN), FLT_MAX);
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

// The pages of a warp's run through its ring, one bulk copy each. All lanes call
// together, lane 0 issues.
template <int D>
struct PageRing {
  uint32_t ring, bars;  // shared-memory addresses
  uint32_t issued = 0, taken = 0;
  __device__ __forceinline__ void issue(const uint8_t* page, int lane) {
    constexpr uint32_t n = Map<D>::kStages, bytes = Kv4Layout<D>::kBytes;
    const uint32_t st = issued % n, bar = bars + st * 8;
    if (lane == 0) {
      mbar_arrive_expect_tx(bar, bytes);
      asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                       ring + st * bytes),
                   "l"(page), "r"(bytes), "r"(bar)
                   : "memory");
    }
    ++issued;
  }
  __device__ __forceinline__ bool wait(volatile int* abort, int32_t* status) const {
    constexpr uint32_t n = Map<D>::kStages;
    return mbar_wait_warp(bars + taken % n * 8, (taken / n) & 1, abort, status);
  }
  // After a wait gave up: the copies still under way land, or are given up as well,
  // before the warp puts the ring to other use or ends.
  __device__ __forceinline__ void drain() {
    constexpr uint32_t n = Map<D>::kStages;
    for (; taken != issued; ++taken) mbar_wait_landed(bars + taken % n * 8, (taken / n) & 1);
    __syncwarp();
  }
};

// S^T = (code * scale) . q for tokens [16 x0, 16 (x0 + X)) of a page in shared
// memory: s[x][n] is 16 tokens by 8 query rows.
template <int D, int NT, int X>
__device__ __forceinline__ void logits(const uint8_t* page, int x0, const uint32_t (&qf)[NT][D / 16][2],
                                       float (&s)[X][NT][4]) {
  using M = Map<D>;
  using L = Kv4Layout<D>;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int x = 0; x < X; ++x) {
    uint32_t w[2][D / 32], sc[2][D == 128 ? 2 : 1];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 16 * (x0 + x) + M::token(i, g >> 1, g & 1);
      if constexpr (D == 128) {
        const uint4 u = *reinterpret_cast<const uint4*>(page + row * 64 + c * 16);
        w[i][0] = u.x; w[i][1] = u.y; w[i][2] = u.z; w[i][3] = u.w;
        const uint32_t h2 = e4m3x2_f16(*reinterpret_cast<const uint16_t*>(page + L::kKs + row * 8 + 2 * c));
        sc[i][0] = __byte_perm(h2, 0, 0x1010);
        sc[i][1] = __byte_perm(h2, 0, 0x3232);
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(page + row * 32 + c * 8);
        w[i][0] = u.x; w[i][1] = u.y;
        const uint32_t h2 = e4m3x2_f16(page[L::kKs + row * 4 + c]);
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

// The part of a run from position x on that lies in one unit: sequence, key head, row
// tile, the pages [p0, p1) of `pages` (none where it ends before the first), its length
// in the cut.
struct Place {
  int s, kvh, tile, p0, p1, pages;
  int64_t length;
};
__device__ __forceinline__ Place place_of(const int* prefix, int n_seqs, int kv_heads, int row_tiles, int64_t x,
                                          int64_t end) {
  const int per_seq = kv_heads * row_tiles;
  int lo = 0, hi = n_seqs - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (static_cast<int64_t>(prefix[mid]) * per_seq <= x) lo = mid; else hi = mid - 1;
  }
  Place p;
  p.s = lo;
  const int span = prefix[lo + 1] - prefix[lo];
  p.pages = span - kUnitPages;
  const int64_t r = x - static_cast<int64_t>(prefix[lo]) * per_seq;
  const int unit = r < 0x80000000LL ? static_cast<int>(static_cast<uint32_t>(r) / static_cast<uint32_t>(span))
                                    : static_cast<int>(r / span);
  const int at = static_cast<int>(r - static_cast<int64_t>(unit) * span);
  p.length = min(static_cast<int64_t>(span - at), end - x);
  p.p0 = max(0, at - kUnitPages);
  p.p1 = max(0, at + static_cast<int>(p.length) - kUnitPages);
  p.kvh = unit / row_tiles;
  p.tile = unit % row_tiles;
  return p;
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

// Tokens [16 x0, 16 (x0 + X)) of a page whose first place is `first` into the state.
template <int D, int NT, int X, bool kEdge>
__device__ __forceinline__ void take(const uint8_t* page, int x0, int first, int len, const int (&seen)[NT][2],
                                     const uint32_t (&qf)[NT][D / 16][2], const float (&factor)[NT][2],
                                     State<D, NT>& z) {
  using M = Map<D>;
  using L = Kv4Layout<D>;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  float s[X][NT][4];
  logits<D, NT, X>(page, x0, qf, s);
  if (kEdge) {
#pragma unroll
    for (int x = 0; x < X; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int j = first + 16 * (x0 + x) + M::token(e >> 1, g >> 1, g & 1);
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
      mx[n][r] = fmaxf(s[0][n][r], s[0][n][2 + r]);
#pragma unroll
      for (int x = 1; x < X; ++x) mx[n][r] = max3f(mx[n][r], s[x][n][r], s[x][n][2 + r]);
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
  uint32_t pf[X][NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint64_t f2 = pack2(__float_as_uint(factor[n][0]), __float_as_uint(factor[n][1]));
    const uint64_t negm = pack2(__float_as_uint(-z.m[n][0]), __float_as_uint(-z.m[n][1])), lift = pair_f32(kLift);
#pragma unroll
    for (int x = 0; x < X; ++x)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float p0, p1;
        unpack2(fma2(add2(pack2(__float_as_uint(s[x][n][2 * i]), __float_as_uint(s[x][n][2 * i + 1])), negm), f2, lift),
                p0, p1);
        p0 = ex2(p0);
        p1 = ex2(p1);
        z.l[n] = add2(z.l[n], pack2(__float_as_uint(p0), __float_as_uint(p1)));
        pf[x][n][i] = transpose8(pack_f16x2(p0, p1));
      }
  }
#pragma unroll
  for (int x = 0; x < X; ++x) {
    uint32_t vsc[2], v[2][2][D / 64];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t by[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 16 * (x0 + x) + M::token(i, c, e);
        by[e] = D == 128 ? page[L::kVs + row * 8 + g] : page[L::kVs + row * 4 + (g >> 1)];
        if (kEdge && first + row >= len) by[e] = 0;
        if constexpr (D == 128) {
          const uint2 u = *reinterpret_cast<const uint2*>(page + L::kV + row * 64 + 8 * g);
          v[i][e][0] = u.x;
          v[i][e][1] = u.y;
        } else {
          v[i][e][0] = *reinterpret_cast<const uint32_t*>(page + L::kV + row * 32 + 4 * g);
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

// A warp's ring, its barriers and the CTA's page offsets, in shared memory.
template <int D>
struct Smem {
  uint64_t bars[kWarps][Map<D>::kStages];
  int warp_sum[kWarps];
  int abort_flag;
};
template <int D>
__device__ __forceinline__ void init_smem(Smem<D>& sm, int warp, int lane) {
  if (lane == 0) {
    for (int i = 0; i < Map<D>::kStages; ++i) mbar_init(smem_u32(&sm.bars[warp][i]), 1);
    fence_mbar_init();
  }
  if (threadIdx.x == 0) sm.abort_flag = 0;
}

// What a weight is made of again: 2^((product - maximum) factor) / sum, with the sum's lift. Maxima are
// joined and kept as products: a rounded maximum in log2 units would be off by
// 2^-24 of itself, and the log of the sum lost beside it, which counts from logits
// of some 10^3 on and makes equal places of large ones weigh 1 each.
__device__ __forceinline__ float2 row_stats(float top, float sum) {
  return make_float2(top, static_cast<float>(1 << static_cast<int>(kLift)) / sum);
}
// What O is multiplied by. A sum of 0: no place seen, or logits that are all -inf, whose
// softmax is 0 / 0 (and so are the weights).
__device__ __forceinline__ float row_scale(float v_sg, float sum, int seen) {
  return sum != 0.0f ? v_sg / sum : seen > 0 ? NAN : 0.0f;
}

template <int D, int NT>
__device__ __forceinline__ void clear(State<D, NT>& z) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
#pragma unroll
    for (int r = 0; r < 2; ++r) z.m[n][r] = z.grow[n][r] = kNoMax;
    z.l[n] = 0;
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) z.o[n][j][e] = 0.0f;
  }
}

// A page whose first place is `first` into the state; the places below `open` are seen by every row.
template <int D, int NT>
__device__ __forceinline__ void take_page(const uint8_t* page, int first, int open, int len, const int (&seen)[NT][2],
                                          const uint32_t (&qf)[NT][D / 16][2], const float (&factor)[NT][2],
                                          State<D, NT>& z) {
  // a whole page at once, or halves where the state of two row tiles takes the registers
  constexpr int X = NT == 1 || D == 64 ? 4 : 2;
#pragma unroll 1
  for (int x0 = 0; x0 < 4; x0 += X) {
    if (first + kKv4Page <= open)
      take<D, NT, X, false>(page, x0, first, len, seen, qf, factor, z);
    else if (first + 16 * x0 < len)
      take<D, NT, X, true>(page, x0, first, len, seen, qf, factor, z);
  }
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv4_attn_kernel(const Args a) {
  using M = Map<D>;
  using L = Kv4Layout<D>;
  constexpr int kTileRows = 8 * NT;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Smem<D> sm;
  int* prefix = reinterpret_cast<int*>(smem + kWarps * M::kRing);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const uint8_t* ring = smem + warp * M::kRing;
  PageRing<D> pr{smem_u32(ring), smem_u32(sm.bars[warp])};
  init_smem(sm, warp, lane);
  volatile int* abort_v = &sm.abort_flag;

  griddep_wait();
  griddep_launch_dependents();
  const int per_seq = a.c.kv_heads * a.row_tiles;
  const Plan plan = make_plan(a.c, per_seq, a.runs, prefix, sm.warp_sum, blockIdx.x == 0 ? a.status : nullptr);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= a.c.n_seqs; i += kThreads) a.prefix[i] = prefix[i];

  // sequences without a token: their rows are 0
  for (int s = blockIdx.x; s < a.c.n_seqs; s += gridDim.x) {
    if (prefix[s + 1] != prefix[s]) continue;
    uint2* dst = reinterpret_cast<uint2*>(static_cast<T*>(a.out) + static_cast<int64_t>(s) * a.q_len * a.heads * D);
    const int64_t n = static_cast<int64_t>(a.q_len) * a.heads * (D / 4);
    for (int64_t i = threadIdx.x; i < n; i += kThreads) dst[i] = make_uint2(0, 0);
  }

  // runs go to CTAs in turn, so that few runs spread over the SMs
  const int run = warp * gridDim.x + blockIdx.x;
  const int64_t begin = run * plan.chunk;
  const int64_t end = min(plan.total, begin + plan.chunk);
  int64_t x = begin;
  while (x < end) {
    const Place at = place_of(prefix, a.c.n_seqs, a.c.kv_heads, a.row_tiles, x, end);
    const int64_t from = x;
    x += at.length;
    const int p0 = at.p0, p1 = at.p1;
    if (p0 == p1) continue;
    const int len = kv4_len(a.c, at.s, nullptr);
    const int mine = p1 - p0;
    int ids = 0;  // the numbers of the next 32 pages, one per lane
    auto issue = [&](int k) {  // k in order, all lanes together
      if (k % 32 == 0) ids = p0 + k + lane < p1 ? static_cast<int>(kv4_page(a.c, at.s, p0 + k + lane, a.status)) : 0;
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
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int r = 0; r < 2; ++r) seen[n][r] = open + (at.tile * kTileRows + 8 * n + 2 * c + r) / a.group;
    State<D, NT> z;
    clear(z);

    bool ok = true;
    for (int k = 0; k < mine && ok; ++k) {
      ok = pr.wait(abort_v, a.status);
      if (!ok) break;
      take_page<D, NT>(ring + pr.taken % M::kStages * L::kBytes, (p0 + k) * kKv4Page, open, len, seen, qf, factor, z);
      ++pr.taken;
      __syncwarp();
      if (next < mine) {
        issue(next);
        ++next;
      }
    }
    if (!ok) {  // a copy that never arrived: the status word says so
      pr.drain();
      break;
    }

    // the rows' results, or partial sums where the unit goes on in other runs
    const bool whole = p0 == 0 && p1 == at.pages;
    const int64_t slot = 2 * static_cast<int64_t>(run) + (from == begin ? 0 : 1);
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      float l[2];
      unpack2(z.l[n], l[0], l[1]);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
        const int tr = 8 * n + 2 * c + r, row = at.tile * kTileRows + tr;
        if (row >= a.rows) continue;
        // columns g D / 8 + 2 j (elements r) and + 1 (elements 2 + r) of tile j
        if (whole) {
          const float inv = row_scale(a.c.v_sg, l[r], seen[n][r]);
          T* dst = static_cast<T*>(a.out) +
                   ((static_cast<int64_t>(at.s) * a.q_len + row / a.group) * a.heads + at.kvh * a.group + row % a.group) * D +
                   g * (D / 8);
#pragma unroll
          for (int j = 0; j < D / 16; j += 4)
            *reinterpret_cast<uint4*>(dst + 2 * j) =
                make_uint4(pack16<T>(z.o[n][j][r] * inv, z.o[n][j][2 + r] * inv),
                           pack16<T>(z.o[n][j + 1][r] * inv, z.o[n][j + 1][2 + r] * inv),
                           pack16<T>(z.o[n][j + 2][r] * inv, z.o[n][j + 2][2 + r] * inv),
                           pack16<T>(z.o[n][j + 3][r] * inv, z.o[n][j + 3][2 + r] * inv));
          if (g == 0 && a.stats != nullptr)
            a.stats[(static_cast<int64_t>(at.s) * a.c.kv_heads + at.kvh) * a.rows + row] = row_stats(z.m[n][r], l[r]);
        } else {
          float* dst = a.part_o + (slot * kTileRows + tr) * D + g * (D / 8);
#pragma unroll
          for (int j = 0; j < D / 16; j += 2)
            *reinterpret_cast<float4*>(dst + 2 * j) =
                make_float4(z.o[n][j][r], z.o[n][j][2 + r], z.o[n][j + 1][r], z.o[n][j + 1][2 + r]);
          if (g == 0)
            a.part_ml[slot * kTileRows + tr] =
                make_float4(z.m[n][r] == kNoMax ? -INFINITY : z.m[n][r], l[r], factor[n][r], 0.0f);
        }
      }
    }
  }
}

// The two of a page's 64 places that a lane adds to: tokens g and g + 8 (by c & 1) of
// tiles c >> 1 and 2 + (c >> 1).
template <int D>
__device__ __forceinline__ int own_place(int first, int h) {
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  return first + 32 * h + 16 * (c >> 1) + Map<D>::token(c & 1, g >> 1, g & 1);
}
template <int D>
__device__ __forceinline__ void weights_before(const float* dst, int first, int len, float (&before)[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) before[h] = own_place<D>(first, h) < len ? dst[own_place<D>(first, h)] : 0.0f;
}

// dst[j] = before + the sum over the rows of 2^((product - top) factor) inv for the places
// of a page: the products once more from its keys. rows_of(tile) sets the rows of a row
// tile, where there are several.
template <int D, int NT, typename Rows>
__device__ __forceinline__ void weigh_page(const uint8_t* page, int first, int len, int row_tiles, Rows rows_of,
                                           const uint32_t (&qf)[NT][D / 16][2], const float (&factor)[NT][2],
                                           const float2 (&stats)[NT][2], const int (&seen)[NT][2],
                                           const float (&before)[2], float* dst) {
  using M = Map<D>;
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (first + 32 * h >= len) continue;
    float w[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};  // tokens g and g + 8 of both tiles
    for (int tile = 0; tile < row_tiles; ++tile) {
      if (row_tiles > 1) rows_of(tile);
      float s[2][NT][4];
      logits<D, NT, 2>(page, 2 * h, qf, s);
#pragma unroll
      for (int y = 0; y < 2; ++y)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int j = first + 32 * h + 16 * y + M::token(e >> 1, g >> 1, g & 1);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float p2 = ex2((s[y][n][e] - stats[n][e & 1].x) * factor[n][e & 1]);
            w[y][e >> 1] += j < seen[n][e & 1] ? p2 * stats[n][e & 1].y : 0.0f;
          }
        }
    }
    float own = 0.0f;
#pragma unroll
    for (int y = 0; y < 2; ++y)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float v = w[y][i];
        v += __shfl_xor_sync(0xffffffffu, v, 1);
        v += __shfl_xor_sync(0xffffffffu, v, 2);
        if (c == 2 * y + i) own = v;
      }
    if (own_place<D>(first, h) < len) dst[own_place<D>(first, h)] = before[h] + own;
  }
}

// Few and short sequences: a cluster of eight CTAs holds a unit. Its 32 warps
// take every 32nd page each and join their sums through distributed shared
// memory, CTA r the rows r (and r + 8): one launch, nothing through memory. Weights,
// where they are wanted and one row tile holds the unit, follow in the same launch.
__device__ __forceinline__ float4 ld_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}
__device__ __forceinline__ uint32_t ld_cluster1(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ float2 ld_cluster2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

template <typename T, int D, int NT>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, kCtasPerSm)
    kv4_cluster_attn_kernel(const Args a) {
  using M = Map<D>;
  using L = Kv4Layout<D>;
  constexpr int kTileRows = 8 * NT;
  static_assert(L::kBytes >= kTileRows * D * 4, "a warp's O tile fits a stage of its ring");
  static_assert(kCluster * kWarps == 32, "a lane per warp of the cluster");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Smem<D> sm;
  __shared__ float2 ml[kWarps][kTileRows];
  __shared__ uint32_t sums_at[kWarps];
  __shared__ float4 join[kWarps][D / 4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  uint8_t* ring = smem + warp * M::kRing;
  PageRing<D> pr{smem_u32(ring), smem_u32(sm.bars[warp])};
  init_smem(sm, warp, lane);
  volatile int* abort_v = &sm.abort_flag;
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();

  const int rank = static_cast<int>(cluster_ctarank());
  const int per_seq = a.c.kv_heads * a.row_tiles, unit = blockIdx.x / kCluster;
  const int s = unit / per_seq, kvh = unit % per_seq / a.row_tiles, tile = unit % a.row_tiles;
  const int len = kv4_len(a.c, s, threadIdx.x == 0 ? a.status : nullptr);
  const int pages = (len + kKv4Page - 1) / kKv4Page;
  const int w0 = rank * kWarps + warp;
  const int mine = (pages - w0 + 31) / 32;  // pages w0, w0 + 32, ...
  int ids = 0;
  auto issue = [&](int k) {  // k in order, all lanes together
    if (k % 32 == 0) {
      const int e = w0 + (k + lane) * 32;
      ids = e < pages ? static_cast<int>(kv4_page(a.c, s, e, a.status)) : 0;
    }
    pr.issue(a.c.pages + (static_cast<int64_t>(__shfl_sync(0xffffffffu, ids, k % 32)) * a.c.kv_heads + kvh) * L::kBytes, lane);
  };
  int next = 0;
  for (; next < min(mine, M::kStages); ++next) issue(next);

  const int open = len - a.q_len + 1;
  uint32_t qf[NT][M::kSteps][2];
  float factor[NT][2];
  load_q<T, D, NT>(a, s, kvh, tile * kTileRows, qf, factor);
  int seen[NT][2];
  State<D, NT> z;
  clear(z);
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r) seen[n][r] = open + (tile * kTileRows + 8 * n + 2 * c + r) / a.group;

  // a copy that never arrives: the status word says so, the cluster goes on to its barriers
  for (int k = 0; k < mine; ++k) {
    if (!pr.wait(abort_v, a.status)) break;
    take_page<D, NT>(ring + pr.taken % M::kStages * L::kBytes, (w0 + k * 32) * kKv4Page, open, len, seen, qf, factor, z);
    ++pr.taken;
    __syncwarp();
    if (next < mine) {
      issue(next);
      ++next;
    }
  }
  pr.drain();

  // each warp's sums into the last stage that it read; the stages before it take the
  // first pages again where the weights are wanted
  const bool weigh = a.weights != nullptr && a.row_tiles == 1;
  const uint32_t last = (pr.issued + M::kStages - 1) % M::kStages * L::kBytes;
  if (lane == 0) sums_at[warp] = last;
  float* own = reinterpret_cast<float*>(ring + last);
  next = 0;
  if (weigh)
    for (; next < min(mine, M::kStages - 1); ++next) issue(next);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    float l[2];
    unpack2(z.l[n], l[0], l[1]);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
      const int tr = 8 * n + 2 * c + r;
      if (g == 0) ml[warp][tr] = make_float2(z.m[n][r] == kNoMax ? -INFINITY : z.m[n][r], l[r]);
#pragma unroll
      for (int j = 0; j < D / 16; j += 2)
        *reinterpret_cast<float4*>(own + tr * D + g * (D / 8) + 2 * j) =
            make_float4(z.o[n][j][r], z.o[n][j][2 + r], z.o[n][j + 1][r], z.o[n][j + 1][2 + r]);
    }
  }
  cluster_sync_all();
  const uint32_t ml0 = smem_u32(&ml[0][0]), ring0 = smem_u32(smem);
  // lane i: where warp i of the cluster left its sums
  const uint32_t part_at = mapa_shared(ring0 + lane % kWarps * M::kRing, lane / kWarps) +
                           ld_cluster1(mapa_shared(smem_u32(&sums_at[lane % kWarps]), lane / kWarps));
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int tr = 8 * n + rank, row = tile * kTileRows + tr;
    if (row >= a.rows) break;  // the same in the whole CTA
    // lane i: the part of warp i of the cluster
    const float2 part = ld_cluster2(mapa_shared(ml0 + ((lane % kWarps) * kTileRows + tr) * 8, lane / kWarps));
    float top = part.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // the factor of row tr, which the lanes of column group rank / 2 have
    const float scale = __shfl_sync(0xffffffffu, (rank & 1) ? factor[n][1] : factor[n][0], rank >> 1);
    const float f = part.x == top ? 1.0f : ex2((part.x - top) * scale);
    float sum = part.y * f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    // this warp's eight parts, each lane four columns
    constexpr int kEach = 32 / kWarps;
    float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
    const bool cols = lane * 4 < D;
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const int p = warp * kEach + i;
      const float fp = __shfl_sync(0xffffffffu, f, p);
      const uint32_t from = __shfl_sync(0xffffffffu, part_at, p);
      if (cols) {
        const float4 u = ld_cluster4(from + (tr * D + lane * 4) * 4);
        t.x += u.x * fp; t.y += u.y * fp; t.z += u.z * fp; t.w += u.w * fp;
      }
    }
    if (cols) join[warp][lane] = t;
    __syncthreads();
    if (warp == 0) {
      const float inv = row_scale(a.c.v_sg, sum, open + row / a.group);
      if (cols) {
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
          const float4 u = join[w][lane];
          t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
        }
        store4<T>(static_cast<T*>(a.out) +
                      ((static_cast<int64_t>(s) * a.q_len + row / a.group) * a.heads + kvh * a.group + row % a.group) * D +
                      lane * 4,
                  t.x * inv, t.y * inv, t.z * inv, t.w * inv);
      }
      if (a.stats != nullptr && lane == 0)
        a.stats[(static_cast<int64_t>(s) * a.c.kv_heads + kvh) * a.rows + row] = row_stats(top, sum);
    }
    __syncthreads();
  }
  cluster_sync_all();  // the others have read this CTA's sums, and every row's stats are written
  if (!weigh) return;
  fence_proxy_async_smem();
  float2 stats[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int row = 8 * n + 2 * c + r;
      stats[n][r] = row < a.rows ? a.stats[(static_cast<int64_t>(s) * a.c.kv_heads + kvh) * a.rows + row]
                                 : make_float2(0.0f, 0.0f);
      if (row >= a.rows) seen[n][r] = 0;
    }
  float* dst = a.weights + (static_cast<int64_t>(s) * a.c.kv_heads + kvh) * a.c.max_pages * kKv4Page;
  for (int k = 0; k < mine; ++k) {
    if (next < mine) {
      issue(next);
      ++next;
    }
    const int first = (w0 + k * 32) * kKv4Page;
    float before[2];
    weights_before<D>(dst, first, len, before);
    if (!pr.wait(abort_v, a.status)) break;
    weigh_page<D, NT>(ring + pr.taken % M::kStages * L::kBytes, first, len, 1, [](int) {}, qf, factor, stats, seen, before, dst);
    ++pr.taken;
    __syncwarp();
  }
  pr.drain();
}

// Joins the partial sums of one row of a unit that was cut: a CTA of two or eight
// warps per row. All the runs' factors first, one run per thread, then their O
// rows strided over the warps, each lane four columns, eight loads under way at
// a time.
template <typename T, int D, int kJoinWarps>
__global__ void __launch_bounds__(kJoinWarps * 32) kv4_combine_kernel(const Args a) {
  griddep_wait();
  griddep_launch_dependents();
  constexpr int kJoinThreads = kJoinWarps * 32;
  __shared__ float sm_o[kJoinWarps][D];
  __shared__ float factor[kJoinThreads], row_factor;
  __shared__ float sm_red[kJoinWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.y, tile = row / a.tile_rows, r = row % a.tile_rows;
  const int s = blockIdx.x / a.c.kv_heads, kvh = blockIdx.x % a.c.kv_heads;
  const int per_seq = a.c.kv_heads * a.row_tiles;
  const int64_t total = static_cast<int64_t>(a.prefix[a.c.n_seqs]) * per_seq;
  const int64_t chunk = max(static_cast<int64_t>(kMinPages), (total + a.runs - 1) / a.runs);
  const int span = a.prefix[s + 1] - a.prefix[s];
  const int64_t lo = static_cast<int64_t>(a.prefix[s]) * per_seq + static_cast<int64_t>(kvh * a.row_tiles + tile) * span;
  const int i0 = static_cast<int>((lo + kUnitPages) / chunk), i1 = static_cast<int>((lo + span - 1) / chunk);
  float2* stats = a.stats == nullptr ? nullptr : a.stats + (static_cast<int64_t>(s) * a.c.kv_heads + kvh) * a.rows + row;
  if (span == 0) {
    if (stats != nullptr && threadIdx.x == 0) *stats = make_float2(0.0f, 0.0f);
    return;
  }
  if (i0 == i1) return;  // one run held the unit: done there
  // the run that the unit starts in may hold another unit before it
  auto at = [&](int i) {
    return (2 * static_cast<int64_t>(i) + (i * chunk >= lo ? 0 : 1)) * a.tile_rows + r;
  };
  float top = -INFINITY, sum = 0.0f;
  float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
  const bool mine = lane * 4 < D;
  for (int base = i0; base <= i1; base += kJoinThreads) {  // as a rule once
    const int n = min(kJoinThreads, i1 - base + 1);
    float4 ml = make_float4(-INFINITY, 0.0f, 0.0f, 0.0f);
    if (static_cast<int>(threadIdx.x) < n) ml = a.part_ml[at(base + threadIdx.x)];
    float m = ml.x;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    __syncthreads();
    if (lane == 0) sm_red[warp] = m;
    if (threadIdx.x == 0) row_factor = ml.z;  // the same in every part
    __syncthreads();
    const float scale = row_factor;
    m = top;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, sm_red[w]);
    const float rescale = top == m ? 1.0f : ex2((top - m) * scale);
    const float f = ml.x == m ? 1.0f : ex2((ml.x - m) * scale);
    factor[threadIdx.x] = f;
    top = m;
    sum = sum * rescale + ml.y * f;
    t.x *= rescale; t.y *= rescale; t.z *= rescale; t.w *= rescale;
    __syncthreads();
    if (mine) {
#pragma unroll 8
      for (int i = warp; i < n; i += kJoinWarps) {
        const float4 u = *reinterpret_cast<const float4*>(a.part_o + at(base + i) * D + lane * 4);
        const float g = factor[i];
        t.x += u.x * g; t.y += u.y * g; t.z += u.z * g; t.w += u.w * g;
      }
    }
  }
  if (mine) *reinterpret_cast<float4*>(&sm_o[warp][lane * 4]) = t;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  __syncthreads();
  if (lane == 0) sm_red[warp] = sum;
  __syncthreads();
  if (warp != 0) return;
  sum = 0.0f;
  t = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    sum += sm_red[w];
    if (mine) {
      const float4 u = *reinterpret_cast<const float4*>(&sm_o[w][lane * 4]);
      t.x += u.x; t.y += u.y; t.z += u.z; t.w += u.w;
    }
  }
  const int seen = sum != 0.0f ? 0 : kv4_len(a.c, s, nullptr) - a.q_len + 1 + row / a.group;
  const float inv = row_scale(a.c.v_sg, sum, seen);
  if (mine)
    store4<T>(static_cast<T*>(a.out) +
                  ((static_cast<int64_t>(s) * a.q_len + row / a.group) * a.heads + kvh * a.group + row % a.group) * D +
                  lane * 4,
              t.x * inv, t.y * inv, t.z * inv, t.w * inv);
  if (stats != nullptr && lane == 0) *stats = row_stats(top, sum);
}

// weights[s, kvh, j] += sum over the rows of 2^(logit - maximum) / sum: the logits once
// more from the keys alone (half the cache's bytes; storing them in the first
// kernel would cost 8 bytes per row and token). One warp owns a slice and sums
// its rows in a fixed order, so no atomics.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) kv4_weights_kernel(const Args a) {
  using M = Map<D>;
  using L = Kv4Layout<D>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ Smem<D> sm;
  int* prefix = reinterpret_cast<int*>(smem + kWarps * M::kRing);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane & 3;
  const uint8_t* ring = smem + warp * M::kRing;
  PageRing<D> pr{smem_u32(ring), smem_u32(sm.bars[warp])};
  init_smem(sm, warp, lane);
  volatile int* abort_v = &sm.abort_flag;
  griddep_wait();
  griddep_launch_dependents();
  const Plan plan = make_plan(a.c, a.c.kv_heads, a.runs, prefix, sm.warp_sum, nullptr);
  const int run = warp * gridDim.x + blockIdx.x;
  const int64_t begin = run * plan.chunk;
  const int64_t end = min(plan.total, begin + plan.chunk);
  int64_t x = begin;
  while (x < end) {
    const Place at = place_of(prefix, a.c.n_seqs, a.c.kv_heads, 1, x, end);
    x += at.length;
    const int p0 = at.p0, p1 = at.p1;
    if (p0 == p1) continue;
    const int len = kv4_len(a.c, at.s, nullptr);
    const int mine = p1 - p0;
    int ids = 0;  // the numbers of the next 32 pages, one per lane
    auto issue = [&](int k) {  // k in order, all lanes together
      if (k % 32 == 0) ids = p0 + k + lane < p1 ? static_cast<int>(kv4_page(a.c, at.s, p0 + k + lane, a.status)) : 0;
      pr.issue(a.c.pages + (static_cast<int64_t>(__shfl_sync(0xffffffffu, ids, k % 32)) * a.c.kv_heads + at.kvh) * L::kBytes,
               lane);
    };
    int next = 0;
    for (; next < min(mine, M::kStages); ++next) issue(next);
    const int open = len - a.q_len + 1;
    const float2* of_row = a.stats + (static_cast<int64_t>(at.s) * a.c.kv_heads + at.kvh) * a.rows;
    float* dst = a.weights + (static_cast<int64_t>(at.s) * a.c.kv_heads + at.kvh) * a.c.max_pages * kKv4Page;
    uint32_t qf[NT][M::kSteps][2];
    float factor[NT][2];
    float2 stats[NT][2];
    int seen[NT][2];
    auto rows_of = [&](int tile) {
      load_q<T, D, NT>(a, at.s, at.kvh, tile * 8 * NT, qf, factor);
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int row = tile * 8 * NT + 8 * n + 2 * c + r;
          stats[n][r] = row < a.rows ? of_row[row] : make_float2(0.0f, 0.0f);
          seen[n][r] = row < a.rows ? open + row / a.group : 0;
        }
    };
    rows_of(0);
    bool ok = true;
    for (int k = 0; k < mine; ++k) {
      const int first = (p0 + k) * kKv4Page;
      float before[2];
      weights_before<D>(dst, first, len, before);
      ok = pr.wait(abort_v, a.status);
      if (!ok) break;
      weigh_page<D, NT>(ring + pr.taken % M::kStages * L::kBytes, first, len, a.row_tiles, rows_of, qf, factor, stats,
                        seen, before, dst);
      ++pr.taken;
      __syncwarp();
      if (next < mine) {
        issue(next);
        ++next;
      }
    }
    if (!ok) {
      pr.drain();
      break;
    }
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
      cudaFuncSetAttribute(kv4_weights_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess ||
      cudaFuncSetAttribute(kv4_cluster_attn_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
    return false;
  if (dev < 64) done[dev] = true;
  return true;
}

}  // namespace

namespace {
// One 8-row tile holds the rows, or tiles of 16 (two of 8 that share the
// operand made from codes); the CTAs; the workspace's parts.
struct Shape {
  int tile_rows, grid, seqs;
  size_t prefix, part_o, part_ml, stats;
  size_t total() const { return prefix + part_o + part_ml + stats; }
};
Shape shape_of(int n_seqs, int heads, int rows, int head_dim, int q_len) {
  Shape z;
  z.tile_rows = rows <= 8 ? 8 : 16;
  z.grid = kCtasPerSm * num_sms();
  z.seqs = std::min(n_seqs, kMaxSeqs);
  const size_t slots = 2 * static_cast<size_t>(z.grid) * kWarps * z.tile_rows;
  z.prefix = up((static_cast<size_t>(z.seqs) + 1) * 4);
  z.part_o = up(slots * head_dim * 4);
  z.part_ml = up(slots * 16);
  z.stats = up(static_cast<size_t>(z.seqs) * heads * q_len * 8);
  return z;
}
}  // namespace

size_t kv4_attention_workspace(int n_seqs, int heads, int kv_heads, int head_dim, int q_len) {
  return shape_of(n_seqs, heads, heads / kv_heads * q_len, head_dim, q_len).total();
}

int launch_kv4_attention(const Kv4& c0, int head_dim, int heads, int q_len, int dtype, const void* q, int64_t q_stride,
                         float scale, void* out, float* weights, void* ws, int32_t* status, cudaStream_t s) {
  Args a;
  a.q_stride = q_stride;
  a.heads = heads;
  a.group = heads / c0.kv_heads;
  a.q_len = q_len;
  a.rows = a.group * q_len;
  const Shape z = shape_of(c0.n_seqs, heads, a.rows, head_dim, q_len);
  const bool one = z.tile_rows == 8;
  a.tile_rows = z.tile_rows;
  a.row_tiles = (a.rows + a.tile_rows - 1) / a.tile_rows;
  a.scale = scale;
  const int grid = z.grid;
  a.runs = grid * kWarps;
  a.status = status;
  uint8_t* w = static_cast<uint8_t*>(ws);
  a.prefix = reinterpret_cast<int32_t*>(w);
  a.part_o = reinterpret_cast<float*>(w + z.prefix);
  a.part_ml = reinterpret_cast<float4*>(w + z.prefix + z.part_o);
  a.stats = weights == nullptr ? nullptr : reinterpret_cast<float2*>(w + z.prefix + z.part_o + z.part_ml);
  const size_t smem = kWarps * (head_dim == 128 ? Map<128>::kRing : Map<64>::kRing) +
                      (static_cast<size_t>(z.seqs) + 1) * 4;
  // A small batch goes by clusters, no warp with more than a few pages: where all units'
  // clusters run at once, or in two waves if the weights are wanted too, which the cluster
  // takes from the pages that it has at hand (one row tile), and the table has a page for
  // every warp. The table's width stands in for the lengths, which only the device knows: a
  // wider table goes by runs however short its sequences are. By runs against by clusters, heads of 128, group 4: one sequence of 3,242
  // places, 8 key heads, 12.6 and 8.5 us; 12 of up to 4,000, 4 key heads (48 units), 18.5
  // and 12.4; 8 of up to 8,000, 8 key heads (64 units), 22.7 and 24.8. With weights, 4
  // tokens: 24 of up to 4,000, 4 key heads (96 units), 50.8 and 45.2; of 500 places, 26.7
  // and 33.3; heads of 64, 24 of up to 6,000, 43 and 33.
  const int64_t units = static_cast<int64_t>(c0.n_seqs) * c0.kv_heads * a.row_tiles;
  const bool fused = weights != nullptr && a.row_tiles == 1 && c0.max_pages >= kCluster * kWarps;
  const int64_t most = static_cast<int64_t>(kCtasPerSm) * num_sms() * (fused ? 2 : 1);
  const bool small = units * kCluster <= most && c0.max_pages <= kClusterPages;
  const bool weigh_after = weights != nullptr && !(small && a.row_tiles == 1);
  const int launches = 1 + (small ? 0 : 1) + (weigh_after ? 1 : 0);
  auto run = [&](auto attn, auto cluster, auto combine, int join_threads, auto weigh, int elem, bool ready) -> int {
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
      cudaError_t e = small ? launch_pdl(cluster, dim3(kCluster * units), dim3(kThreads), smem, s, a)
                            : launch_pdl(attn, dim3(grid), dim3(kThreads), smem, s, a);
      if (e == cudaSuccess && !small)
        e = launch_pdl(combine, dim3(a.c.n_seqs * a.c.kv_heads, a.rows), dim3(join_threads), 0, s, a);
      if (e == cudaSuccess && weigh_after) e = launch_pdl(weigh, dim3(grid), dim3(kThreads), smem, s, a);
      if (e != cudaSuccess) return VLM_ERR_CUDA;
    }
    return VLM_OK;
  };
  launch_begin(KC_KV4_ATTN, s);
  auto pick = [&](auto type, auto dim, auto nt) {
    using T = decltype(type);
    constexpr int D = decltype(dim)::value, NT = decltype(nt)::value;
    // two warps per joined row where a unit has a dozen parts at most, or where the rows fill
    // the SMs anyway: with eight 24 sequences of 3,000 places, 16 rows of 64, 23.9 and not
    // 20.6 us, 16 of 9,000, 16 rows of 128, 61.5 and not 55.5; with two always 24 of 3,000,
    // 4 rows of 64, 20.6 and not 18.6
    const int64_t rows_in_all = static_cast<int64_t>(z.seqs) * c0.kv_heads * a.rows;
    const bool few = a.runs <= 12LL * z.seqs * c0.kv_heads * a.row_tiles || rows_in_all > 8LL * num_sms();
    return run(kv4_attn_kernel<T, D, NT>, kv4_cluster_attn_kernel<T, D, NT>, few ? kv4_combine_kernel<T, D, 2> : kv4_combine_kernel<T, D, 8>, few ? 64 : 256,
               kv4_weights_kernel<T, D, NT>, 2, smem_ready<T, D, NT>());
  };
  auto by_rows = [&](auto type, auto dim) {
    return one ? pick(type, dim, std::integral_constant<int, 1>()) : pick(type, dim, std::integral_constant<int, 2>());
  };
  auto by_dim = [&](auto type) {
    return head_dim == 128 ? by_rows(type, std::integral_constant<int, 128>()) : by_rows(type, std::integral_constant<int, 64>());
  };
  const int rc = dtype == VLM_DTYPE_F16 ? by_dim(__half()) : by_dim(__nv_bfloat16());
  launch_end(KC_KV4_ATTN, s);
  note_extra_launches(((c0.n_seqs + kMaxSeqs - 1) / kMaxSeqs) * launches - 1);
  return rc;
}

}  // namespace vlm
