// Causal attention of packed prompts with grouped heads on the sm_100a tensor
// cores, head dimension 64 or 128, bf16 or fp16. Sequence s has q_len queries
// and kv_len keys; its last query sees every key:
//   o_i = sum_{j <= i + kv_len - q_len} softmax_j(scale q_i . k_j) v_j,
// query head h reads key head h / (heads / kv_heads).
//
// One work item = 2 row tiles of one sequence and one key head. A row tile
// holds TPT = 128 / G consecutive tokens times the G query heads of the group
// (row = token * G + head), so both tiles, 2 TPT tokens, share every key and
// value tile that is loaded, and a short prompt still fills its rows. CTAs
// (one per SM, 512 TMEM columns) take items in turn, forwards and backwards
// through the list, which is sorted by key tiles, or where there are few items
// those that the host chose for them. 20 warps:
//   warp 0       TMA: both Q tiles, then K and V tiles of 128 keys into two
//                2-stage rings (128-byte swizzle, 64-column boxes).
//   warps 1, 2   issue row tile t's products, one warp each, for key tile j
//                  S_t  = Q_t K_j^T           (tcgen05.mma kind::f16, M = N = 128)
//                  O_t += P_t V_{j-1}         (A = P in TMEM, V in smem, MN-major)
//                An instruction takes the tensor core 64 cycles. Issued by one
//                lane of a divergent branch it cost that lane 100, so that one
//                warp for both tiles was the bound (4,190 cycles per key tile);
//                as a predicated instruction of a converged warp it costs 65.
//   warps 4..19  softmax, two threads per row (keys [0, 64) and [64, 128) of
//                the tile), 256 threads per row tile: running maximum (moved
//                only when it grows by more than 8 in log2 units), P as 16-bit
//                pairs in TMEM, fp32 sums, O rescaled in TMEM when the maximum
//                moved, and O / l at the end.
// Both row tiles take every key tile of the item, so they alternate strictly;
// the products of key tiles that a row tile does not see at all (one in
// several) have weight 0.
// Bound, D = 128: the chain of hand-overs through the shared S buffer. S_0 is
// copied (250 cycles), handed over (350), S_1's product runs (512) and is
// reported (430): about 3,000 cycles per key tile against the tensor core's
// 2,048 and the exponential unit's 1,800. Handing S over in halves of 64 keys
// (N = 64 products) was slower; P over its own S, which would leave each row tile a
// buffer of its own, is not built. D = 64: the softmax itself, 2,500 cycles per key
// tile. An item costs 5,000 to 9,000 cycles besides: its last product, O to memory,
// and the look at V below. Measured, one call replayed on the same inputs, 32/8 heads of
// 128, bf16: 4,096 tokens 112 to 118 us, 1,170 to 1,230 TFLOP/s (0.71 to 0.75 of the
// measured peak, by the box); 8,192 tokens 411 to 425 us, 1,290 to 1,340; 3,241 tokens
// 74 to 83 us; four of 4,096 465 us, 1,180; heads of 64: 8,192 tokens 367 to 383 us,
// 720 to 740. Passes over several sets of inputs in turn run into the power cap: 3,241
// tokens 90 us, 955 TFLOP/s; four of 4,096 541 us, 1,020. The softmax's instructions
// count as well, 57% of the issue slots: exponentials from polynomials beside
// the unit (2% slower), maxima exchanged on every tile instead of where one
// moves and a vote on the logits' size per tile (5% together) went for that.
// TMEM, D = 128: one S buffer that the row tiles take in turn [0, 128), P
// [128, 192) and [192, 256), O [256, 384) and [384, 512); a tile's logits leave
// S for registers at once, so the buffer is free again while its softmax runs.
// D = 64: S [0, 128) and [128, 256), P [256, 384), O [384, 512).
//
// Roundings: P to the inputs' type (half a step; fp16 weights, which are made 2^7
// times as large, below 2^-21 of the row's largest to within 2^-32 of it; its fp32
// sum is taken before rounding), the output once; everything else is fp32.
// Places that a row does not see get weight 0. A weight of 0 does not stop an
// infinity or NaN in V, so on key tiles that some row of the item does not see in
// full the softmax threads of both row tiles look V over in shared memory before
// their product: rows behind the sequence's keys become 0, and a value that is not
// finite is replaced by 0 and its key noted; at the end rows that do see a noted
// key add its values. (On other key tiles the product takes it, with NaN where the
// row's weight rounds to 0.)
// A query that sees no key (kv_len < q_len) gives 0.
#include <algorithm>
#include <cfloat>
#include <functional>
#include <numeric>
#include <vector>

#include "softmax.cuh"
#include "text_attention.cuh"

namespace vlm {

namespace {

constexpr int BK = 128;        // keys per tile
constexpr int kRows = 128;     // rows per row tile
constexpr int HK = BK / 2;     // keys per softmax thread
constexpr int kSoftWarps = 16;
constexpr int kThreads = 32 * (4 + kSoftWarps);
constexpr int kStages = 2;
constexpr int kMaxSeqs = 256;    // sequences per launch (their table is a kernel argument)
constexpr int kMaxOrder = 1024;  // tiles per key head whose order is passed along
constexpr int kItemSlots = 512;  // items per CTA and launch
constexpr int kMaxPacked = 512;  // items whose CTAs are chosen one by one
constexpr int kMaxCtas = 256;     // and the CTAs then
constexpr int kIssueRegs = 32, kSoftRegs = 112;
static_assert(128 * kIssueRegs + 32 * kSoftWarps * kSoftRegs <= kThreads * 96, "the launch's registers");
constexpr int kSets = 8;       // items whose noted keys are kept apart
constexpr float kRescaleThreshold = 8.0f;  // log2 units

struct SeqTable {
  int n;
  int off[kMaxSeqs + 1];  // work items before each sequence
  int q0[kMaxSeqs], k0[kMaxSeqs], q_len[kMaxSeqs], kv_len[kMaxSeqs], tiles[kMaxSeqs];  // tiles: items per key head
  int ordered;               // pairs in `order`, or 0: sequence by sequence, last tile first
  uint32_t order[kMaxOrder];  // sequence << 16 | tile, the most key tiles first
  // CTA b's items are item[first[b]] to item[first[b + 1] - 1], numbers in the launch's list;
  // first[gridDim.x] is 0 where the list is dealt out in turn
  uint16_t first[kMaxCtas + 1], item[kMaxPacked];
};

struct Args {
  SeqTable t;
  int kv_heads, group, tpt;
  float sl2;  // scale * log2(e)
  const void* v;
  int64_t v_stride;
  void* out;
  int64_t out_stride;
  int32_t* status;
};

template <int D>
struct Cfg {
  static constexpr int kSub = 128 * 128;           // bytes of 128 rows x 64 columns
  static constexpr int kTile = kSub * (D / 64);    // one Q, K or V tile
  static constexpr int kQ = 0, kK = 2 * kTile, kV = kK + kStages * kTile;
  static constexpr int kBars = kV + kStages * kTile;
  // row maxima [tile][parity of the key tile][half][row], sums [tile][parity of the item][half][row]
  static constexpr int kXch = kBars + 256;
  static constexpr int kFlags = kXch + (8 + 8) * kRows * 4;  // noted keys, kSets sets of 512 bits
  static constexpr int kItems = kFlags + kSets * 64;         // this CTA's first items, decoded
  static constexpr int kSmem = kItems + kItemSlots * 32 + 1024;
  static constexpr uint32_t s_col(int t) { return D == 128 ? 0 : 128 * t; }
  static constexpr uint32_t p_col(int t) { return D == 128 ? 128 + 64 * t : 256 + 64 * t; }
  static constexpr uint32_t o_col(int t) { return D == 128 ? 256 + 128 * t : 384 + 64 * t; }
};

template <typename T>
constexpr bool is_half = std::is_same_v<T, __half>;

template <typename T>
__host__ __device__ constexpr uint32_t idesc16(int m, int n, bool b_mn_major = false) {
  return idesc_bf16(m, n, b_mn_major) & (is_half<T> ? ~((1u << 7) | (1u << 10)) : ~0u);  // format 0: fp16
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// True in one lane of the (converged) warp, the same one each time.
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p;
}
// tcgen05 instructions issued by the lane with `go` set, as predicated
// instructions of the whole warp: in a divergent branch their operands would
// have to be moved into uniform registers one by one.
__device__ __forceinline__ void mma_ss(uint32_t go, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(go)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t go, uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(go)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint32_t go, uint32_t bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar),
      "r"(go)
      : "memory");
}
// One arrival for a warp, after all its lanes got here: arrivals of single
// threads on one barrier are taken one after the other.
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}
// a + 0 b on 16-bit pairs: 0 as long as every b is finite, NaN from then on.
template <typename T>
__device__ __forceinline__ uint32_t add_zero_times(uint32_t a, uint32_t b) {
  uint32_t d;
  if constexpr (is_half<T>)
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(b), "r"(0u), "r"(a));
  else
    asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(b), "r"(0u), "r"(a));
  return d;
}
// mbar_wait_warp that polls instead of suspending the warp: for the two issuing
// warps, whose wake-up the whole key tile waits for.
__device__ __forceinline__ bool mbar_poll_warp(uint32_t bar, uint32_t parity, volatile int* abort, int32_t* status) {
  auto test = [&]() {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
  };
  if (__all_sync(0xffffffffu, test())) return true;
  const long long t0 = clock64();
  for (uint32_t i = 1;; ++i) {
    if (__all_sync(0xffffffffu, test())) return true;
    if ((i & 255u) == 0) {
      bool stop = *abort != 0;
      if (!stop && clock64() - t0 > kWaitBudgetCycles) {
        *abort = 1;
        set_status(status, VLM_ERR_TIMEOUT);
        stop = true;
      }
      if (__any_sync(0xffffffffu, stop)) return false;
    }
  }
}
// The 64 threads of a named barrier meet; true for all if `mine` is for one.
__device__ __forceinline__ bool bar_any(int id, bool mine) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, %2, 64, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(static_cast<uint32_t>(mine)), "r"(id)
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void bar_sync(int id, int threads) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// How many of the launch's items are this CTA's, and the number of its k-th. Dealt out in
// turn, forwards and backwards, so that with items sorted by size every CTA's share is
// alike, or as the host chose.
__device__ __forceinline__ bool chosen(const SeqTable& t) { return t.first[gridDim.x] != 0; }
__device__ __forceinline__ int dealt(int k) {
  return k * gridDim.x + ((k & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
}
__device__ __forceinline__ int count_items(const SeqTable& t, int n_items) {
  if (chosen(t)) return t.first[blockIdx.x + 1] - t.first[blockIdx.x];
  const int rounds = n_items / static_cast<int>(gridDim.x);
  return rounds + (dealt(rounds) < n_items ? 1 : 0);
}
__device__ __forceinline__ int nth_item(const SeqTable& t, int k) {
  return chosen(t) ? t.item[t.first[blockIdx.x] + k] : dealt(k);
}

// A work item: sequence, key head, the first token of its row tiles, its key tiles.
struct alignas(16) Item {
  int q0, k0, q_len, kv_len, head, tok0;
  int n;       // key tiles
  int shift;   // kv_len - q_len
  __device__ __forceinline__ int tok(int t, int tpt) const { return tok0 + t * tpt; }
};
__device__ __forceinline__ Item item_of(const Args& a, int idx) {
  Item it;
  int lo = 0, tile;
  if (a.t.ordered > 0) {
    const int pair = idx / a.kv_heads;
    it.head = idx - pair * a.kv_heads;
    lo = a.t.order[pair] >> 16;
    tile = a.t.order[pair] & 0xFFFF;
  } else {
    int hi = a.t.n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.t.off[mid] <= idx) lo = mid; else hi = mid - 1;
    }
    const int r = idx - a.t.off[lo], row = r / a.kv_heads;
    it.head = r - row * a.kv_heads;
    tile = a.t.tiles[lo] - 1 - row;
  }
  it.q0 = a.t.q0[lo];
  it.k0 = a.t.k0[lo];
  it.q_len = a.t.q_len[lo];
  it.kv_len = a.t.kv_len[lo];
  it.tok0 = tile * 2 * a.tpt;
  it.shift = it.kv_len - it.q_len;
  const int end = it.shift + min(it.q_len, it.tok0 + 2 * a.tpt);  // keys that the last row sees
  it.n = max(0, (end + BK - 1) / BK);
  return it;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ Args args, int first_item,
                       int n_items) {
  using C = Cfg<D>;
  constexpr bool kHalf = is_half<T>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBars);
  uint64_t* q_full = bars;
  uint64_t* q_empty = bars + 1;
  uint64_t* k_full = bars + 2;
  uint64_t* k_empty = k_full + kStages;
  uint64_t* v_full = k_empty + kStages;
  uint64_t* v_empty = v_full + kStages;
  uint64_t* s_full = v_empty + kStages;  // [2] row tiles
  uint64_t* s_free = s_full + 2;         // [2] S buffers
  uint64_t* p_full = s_free + 2;         // [2]
  uint64_t* o_done = p_full + 2;         // [2]
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(o_done + 2);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  uint32_t* flags = reinterpret_cast<uint32_t*>(smem + C::kFlags);  // [kSets][16]

  // the warp index as a warp-uniform value, so that its branches and what they compute stay uniform
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(q_full), 1);
    mbar_init(smem_u32(q_empty), 2);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(smem_u32(k_full + s), 1);
      mbar_init(smem_u32(k_empty + s), 2);
      mbar_init(smem_u32(v_full + s), 1);
      mbar_init(smem_u32(v_empty + s), 2);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(smem_u32(s_full + t), 1);
      mbar_init(smem_u32(s_free + t), kSoftWarps / 2);
      mbar_init(smem_u32(p_full + t), kSoftWarps / 2);
      mbar_init(smem_u32(o_done + t), 1);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (threadIdx.x < kSets * 16) flags[threadIdx.x] = 0;
  // Decoding an item (divisions, indexed argument loads) takes some 2,000 cycles in
  // the middle of the pipeline, so it is done for the whole list at the start.
  Item* items_s = reinterpret_cast<Item*>(smem + C::kItems);
  const int my_items = count_items(args.t, n_items);
  for (int k = threadIdx.x; k < my_items; k += kThreads) items_s[k] = item_of(args, first_item + nth_item(args.t, k));
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  volatile int* abort_v = abort_flag;
  griddep_wait();
  griddep_launch_dependents();
  // 640 threads x 96 registers at launch: the issuing warps give some up to the softmax
  if (warp < 4)
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kIssueRegs));
  else
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftRegs));

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t q_bytes = 128u * args.group * args.tpt * (D / 64);
      uint32_t kc = 0, vc = 0, qc = 0;
      bool ok = true;
      for (int w = 0; ok && w < my_items; ++w) {
        const Item it = items_s[w];
        const int n = it.n, tiles = it.tok(1, args.tpt) < it.q_len ? 2 : 1;
        if (n == 0) continue;
        if (!mbar_wait(smem_u32(q_empty), (qc & 1) ^ 1, abort_v, args.status)) break;
        const uint32_t qb = smem_u32(q_full);
        mbar_arrive_expect_tx(qb, q_bytes * tiles);
        for (int t = 0; t < tiles; ++t)
          for (int x = 0; x < D / 64; ++x)
            tma_load_3d(smem_u32(smem + C::kQ + t * C::kTile + x * C::kSub), &tm_q, qb, 64 * x, it.head * args.group,
                        it.q0 + it.tok(t, args.tpt));
        ++qc;
        for (int j = 0; j <= n; ++j) {
          if (j < n) {
            const uint32_t st = kc % kStages;
            if (!(ok = mbar_wait(smem_u32(k_empty + st), ((kc / kStages) & 1) ^ 1, abort_v, args.status))) break;
            const uint32_t fb = smem_u32(k_full + st);
            mbar_arrive_expect_tx(fb, C::kTile);
            for (int x = 0; x < D / 64; ++x)
              tma_load_3d(smem_u32(smem + C::kK + st * C::kTile + x * C::kSub), &tm_k, fb, 64 * x, it.head,
                          it.k0 + j * BK);
            ++kc;
          }
          if (j > 0) {
            const uint32_t st = vc % kStages;
            if (!(ok = mbar_wait(smem_u32(v_empty + st), ((vc / kStages) & 1) ^ 1, abort_v, args.status))) break;
            const uint32_t fb = smem_u32(v_full + st);
            mbar_arrive_expect_tx(fb, C::kTile);
            for (int x = 0; x < D / 64; ++x)
              tma_load_3d(smem_u32(smem + C::kV + st * C::kTile + x * C::kSub), &tm_v, fb, 64 * x, it.head,
                          it.k0 + (j - 1) * BK);
            ++vc;
          }
        }
      }
      // Every copy has landed, or is given up, before the CTA ends: as a rule the products
      // wait for it anyway, after an abort nobody else does.
      if (qc > 0) mbar_wait_landed(smem_u32(q_full), (qc - 1) & 1);
      for (uint32_t st = 0; st < kStages; ++st) {
        // fills of stage st so far: its last one is in phase (fills - 1)
        const uint32_t kf = (kc + kStages - 1 - st) / kStages, vf = (vc + kStages - 1 - st) / kStages;
        if (kf > 0) mbar_wait_landed(smem_u32(k_full + st), (kf - 1) & 1);
        if (vf > 0) mbar_wait_landed(smem_u32(v_full + st), (vf - 1) & 1);
      }
    }
  } else if (warp < 3) {
    // The whole warp walks the loop and one elected lane issues: descriptors
    // and addresses then live in uniform registers.
    const int t = warp - 1;
    const uint32_t go = elect_one();
    constexpr uint32_t idesc_s = idesc16<T>(kRows, BK);
    constexpr uint32_t idesc_o = idesc16<T>(kRows, D, /*b_mn_major=*/true);
    const uint64_t qdesc = smem_desc_sw128(smem_u32(smem + C::kQ + t * C::kTile));
    const uint64_t kdesc = smem_desc_sw128(smem_u32(smem + C::kK));
    const uint64_t vdesc = smem_desc_sw128(smem_u32(smem + C::kV), 1024, C::kSub);
    const uint32_t s_at = tmem + C::s_col(t), p_at = tmem + C::p_col(t), o_at = tmem + C::o_col(t);
    const uint32_t bar0 = smem_u32(bars);
    auto bar = [&](const uint64_t* x) { return bar0 + static_cast<uint32_t>(x - bars) * 8; };
    auto wait = [&](const uint64_t* x, uint32_t parity) {
      return mbar_poll_warp(bar(x), parity, abort_v, args.status);
    };
    // The row tiles' logits are made in turn, S_0 S_1 S_0 ..., each once the softmax has
    // copied the one before: at D = 128 they share the buffer, at D = 64 it keeps the two
    // softmaxes out of step, so that one's exponentials run beside the other's loads and
    // hand-overs (8,192 tokens, 32/8 heads of 64: 457 us left to themselves, in step; 400 us).
    const uint64_t* s_prev = s_free + (1 - t);
    const uint32_t s_lag = t == 1 ? 0 : 1;
    uint32_t kc = 0, vc = 0, qc = 0;  // K, V and Q tiles so far (S and P run with K and V)
    bool ok = true;
    for (int w = 0; ok && w < my_items; ++w) {
      const Item it = items_s[w];
      const int n = it.n;
      if (n == 0) continue;
      if (!(ok = wait(q_full, qc & 1))) break;
      for (int j = 0; j <= n; ++j) {
        if (j < n) {
          const uint32_t ks = kc % kStages;
          if (!(ok = wait(k_full + ks, (kc / kStages) & 1))) break;
          if (kc >= s_lag && !(ok = wait(s_prev, (kc - s_lag) & 1))) break;
          tc_fence_after();
          const uint64_t kd = kdesc + ks * (C::kTile / 16);
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k / 4) * (C::kSub / 16) + 2 * (k % 4);
            mma_ss(go, s_at, qdesc + off, kd + off, idesc_s, k > 0 ? 1u : 0u);
          }
          mma_commit(go, bar(s_full + t));
          mma_commit(go, bar(k_empty + ks));
          if (j == n - 1) mma_commit(go, bar(q_empty));
          ++kc;
        }
        if (j > 0) {
          const uint32_t vs = vc % kStages;
          if (!(ok = wait(v_full + vs, (vc / kStages) & 1))) break;
          // P is written by the threads that read O at the end of an item, after they did
          if (!(ok = wait(p_full + t, vc & 1))) break;
          tc_fence_after();
          const uint64_t vd = vdesc + vs * (C::kTile / 16);
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)  // 16 keys: 8 TMEM columns of pairs, 2048 bytes of V
            mma_ts(go, o_at, p_at + 8 * kk, vd + 128 * kk, idesc_o, (j > 1 || kk > 0) ? 1u : 0u);
          mma_commit(go, bar(o_done + t));
          mma_commit(go, bar(v_empty + vs));
          ++vc;
        }
      }
      ++qc;
    }
  } else if (warp >= 4) {
    const int t = (warp - 4) >> 3, hf = ((warp - 4) >> 2) & 1, quad = warp & 3;
    const int r = quad * 32 + lane;            // row of the tile = TMEM lane
    const int pair_id = 1 + t * 4 + quad;      // named barrier of the two warps of these rows
    const int tid = (warp - 4 - 8 * t) * 32 + lane;  // 0..255 in the row tile's threads
    const uint32_t trow = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    float* xmax = reinterpret_cast<float*>(smem + C::kXch) + t * 4 * kRows;
    float* xsum0 = reinterpret_cast<float*>(smem + C::kXch) + (8 + t * 4) * kRows;
    const uint64_t sl2x2 = pair_f32(args.sl2);
    const float grow_by = fminf(kRescaleThreshold / args.sl2, 1e38f);  // in the logits' own units, as the maximum is
    const int row_tok = r / args.group, row_head = r - row_tok * args.group;
    const bool wide = ((reinterpret_cast<uintptr_t>(args.out) | (args.out_stride * 2)) & 31) == 0;
    uint32_t sc = 0, oc = 0, vc_item = 0, live_items = 0;
    int items = 0;
    bool ok = true;
    // A warp whose wait failed keeps meeting its partner at the named barrier,
    // doing nothing else, so that the partner never waits for it.
    for (; items < my_items; ++items) {
      const Item it = items_s[items];
      const int tok = it.tok(t, args.tpt) + row_tok;
      const bool live = tok < it.q_len && row_tok < args.tpt;
      const int lim = it.shift + tok + 1;                     // the row sees keys [0, lim)
      const int lim_min = it.shift + it.tok(t, args.tpt) + 1;  // what every row of the tile sees
      const int lim_item = it.shift + it.tok0 + 1;             // and every row of the item
      const int flag_base = max(0, lim_item) / BK * BK;
      // The row tiles' threads are at most three key tiles apart (two K stages and the
      // alternation of S), so the notes of four items back are no longer in use: cleared
      // here for the item four ahead. Items without keys have no notes and do not count.
      uint32_t* flag = flags + 16 * (live_items % kSets);
      if (it.n > 0) {
        if (t == 0 && tid < 16) flags[16 * ((live_items + kSets / 2) % kSets) + tid] = 0;
        ++live_items;
      }
      const int n = it.n;
      const bool idle = it.tok(t, args.tpt) >= it.q_len;  // a row tile without tokens
      float m = -INFINITY, l = 0.f, ref = 0.0f;  // ref: m, or 0 before the row sees a key
      bool large = false;
      for (int j = 0; j < n; ++j) {
        if (ok) ok = mbar_poll_warp(smem_u32(s_full + t), sc & 1, abort_v, args.status);
        ++sc;
        if (!ok) {
          if (!idle && bar_any(pair_id, false)) bar_sync(pair_id, 64);
          continue;
        }
        tc_fence_after();
        if (idle) {
          warp_arrive(smem_u32(s_free + t), lane);
          if (j > 0) ok = mbar_wait_warp(smem_u32(o_done + t), (oc - 1) & 1, abort_v, args.status);
          if (ok) warp_arrive(smem_u32(p_full + t), lane);
          ++oc;
          continue;
        }
        uint32_t u[HK];
        tmem_ld64(trow + C::s_col(t) + HK * hf, u);
        tc_fence_before();
        warp_arrive(smem_u32(s_free + t), lane);
        const bool masked = (j + 1) * BK > lim_min;
        if (masked) {
          const int nvalid = lim - j * BK - HK * hf;
#pragma unroll
          for (int c = 0; c < HK; ++c)
            if (c >= nvalid) u[c] = __float_as_uint(-INFINITY);
        }
        // The two threads of a row meet here; only where one of the 32 rows' maxima
        // moves do they tell each other theirs.
        const float m_own = row_max(u);
        const bool grows = bar_any(pair_id, m_own > m + grow_by);
        float corr = 1.0f;
        if (grows) {
          xmax[((j & 1) * 2 + hf) * kRows + r] = m_own;
          bar_sync(pair_id, 64);
          const float m_cand = fmaxf(m_own, xmax[((j & 1) * 2 + (hf ^ 1)) * kRows + r]);
          if (m_cand > m + grow_by) {
            corr = ex2((m - m_cand) * args.sl2);
            m = m_cand;
          }
          l *= corr;
          ref = m == -INFINITY ? 0.0f : m;
          // Logits of ordinary size: 2^(s sl2 - m sl2) in one operation; the rounding of
          // m sl2 (less fp16's lift) scales the row's weights by up to 2^(2^-13) alike.
          // Masked tiles and large logits are subtracted before they are scaled. (Rows
          // without a token do not vote: they hold other sequences' queries or nothing.)
          large = __any_sync(0xffffffffu, live && fabsf(ref * args.sl2) > 4096.0f - kHalfLift);
        }
        uint32_t pk[HK / 2];
        l += !masked && !large ? row_exp<false, kHalf>(u, sl2x2, fmaf(ref, args.sl2, kHalf ? -kHalfLift : 0.0f), pk)
                               : row_exp<false, kHalf, true>(u, sl2x2, ref, pk);
        if (j > 0) {
          // the product with the tile before must be done before O is rescaled and P overwritten
          ok = mbar_wait_warp(smem_u32(o_done + t), (oc - 1) & 1, abort_v, args.status);
          if (!ok) continue;
          tc_fence_after();
        }
        tmem_st32(trow + C::p_col(t) + 32 * hf, pk);
        if (j > 0 && grows) {
#pragma unroll
          for (int x = 0; x < D / 64; ++x) {
            const uint32_t col = trow + C::o_col(t) + (D / 2) * hf + 32 * x;
            uint32_t o[32];
            tmem_ld32(col, o);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * corr);
            tmem_st32(col, o);
          }
        }
        if ((j + 1) * BK > lim_item) {
          // Look this V tile over before its product. Both row tiles' threads do so, the second's
          // also where its own rows see the whole tile: its product would otherwise read values
          // that the first one's threads are replacing. What one writes the other would write as well.
          const uint32_t vc = vc_item + j, vs = vc % kStages;
          ok = mbar_wait_warp(smem_u32(v_full + vs), (vc / kStages) & 1, abort_v, args.status);
          if (ok) {
            const int valid = it.kv_len - j * BK;
            constexpr int kChunks = BK * D / 8 / 256;  // 16-byte chunks per thread
            constexpr uint32_t e = kHalf ? 0x7C007C00u : 0x7F807F80u;
            uint8_t* tile = smem + C::kV + vs * C::kTile;
            // chunk x of the thread: row tid / 8 + 32 (x % 4), column group tid % 8 of 64-column box x / 4
            uint8_t* mine = tile + (tid >> 3) * 128 + (((tid & 7) ^ ((tid >> 3) & 7)) << 4);
            uint32_t odd = 0;
#pragma unroll
            for (int x = 0; x < kChunks; ++x) {
              const uint4 w = *reinterpret_cast<const uint4*>(mine + (x / 4) * C::kSub + (x % 4) * 4096);
              odd = add_zero_times<T>(add_zero_times<T>(odd, w.x), w.y);
              odd = add_zero_times<T>(add_zero_times<T>(odd, w.z), w.w);
            }
            if ((odd & 0x7FFF7FFFu) != 0 || valid < BK) {
#pragma unroll 1
              for (int x = 0; x < kChunks; ++x) {
                const int row = (tid >> 3) + 32 * (x % 4);
                uint4* at = reinterpret_cast<uint4*>(mine + (x / 4) * C::kSub + (x % 4) * 4096);
                if (row >= valid) {
                  *at = make_uint4(0, 0, 0, 0);
                } else {
                  uint4 w = *at;
                  if ((__vcmpeq2(w.x & e, e) | __vcmpeq2(w.y & e, e) | __vcmpeq2(w.z & e, e) | __vcmpeq2(w.w & e, e)) == 0)
                    continue;
                  w.x &= ~__vcmpeq2(w.x & e, e);
                  w.y &= ~__vcmpeq2(w.y & e, e);
                  w.z &= ~__vcmpeq2(w.z & e, e);
                  w.w &= ~__vcmpeq2(w.w & e, e);
                  const int key = j * BK + row - flag_base;
                  if (key >= 0 && key < 512) atomicOr(flag + (key >> 5), 1u << (key & 31));
                  __threadfence_block();  // whoever finds the value replaced finds the note
                  *at = w;
                }
              }
            }
            // also for what the other row tile's threads wrote and this one found done
            fence_proxy_async_smem();
          }
        }
        tmem_st_wait();
        tc_fence_before();
        warp_arrive(smem_u32(p_full + t), lane);
        ++oc;
      }
      // By the item's parity: a warp that is done with an item without key tiles, or with one key tile and
      // an idle row tile (neither meets its partner before this), must not write over the sum that the
      // partner still has to read from the item before. Two items on, the barrier of the one between is passed.
      float* xsum = xsum0 + (items & 1) * 2 * kRows;
      xsum[hf * kRows + r] = l;
      bar_sync(pair_id, 64);
      l += xsum[(hf ^ 1) * kRows + r];
      if (ok && n > 0) ok = mbar_wait_warp(smem_u32(o_done + t), (oc - 1) & 1, abort_v, args.status);
      if (ok) {
        tc_fence_after();
        // a sum of 0: no key seen, or logits that are all -inf, whose softmax is 0 / 0
        const float inv = l != 0.0f ? 1.0f / l : lim > 0 ? NAN : 0.0f;
        uint32_t noted = 0;
        if (n > 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint4 w = reinterpret_cast<const uint4*>(flag)[i];
            noted |= w.x | w.y | w.z | w.w;
          }
        }
        T* dst = static_cast<T*>(args.out) + static_cast<int64_t>(it.q0 + tok) * args.out_stride +
                 (it.head * args.group + row_head) * D + (D / 2) * hf;
#pragma unroll
        for (int x = 0; x < D / 64; ++x) {
          uint32_t o[32];
          if (n > 0) {
            tmem_ld32(trow + C::o_col(t) + (D / 2) * hf + 32 * x, o);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0;
          }
          if (live) {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv);
            if (noted != 0) {
              // keys whose values are not finite: rows that see them take those values
              for (int key = 0; key < 512 && flag_base + key < lim; ++key) {
                if (!((flag[key >> 5] >> (key & 31)) & 1)) continue;
                const T* vr = static_cast<const T*>(args.v) + static_cast<int64_t>(it.k0 + flag_base + key) * args.v_stride +
                              it.head * D + (D / 2) * hf + 32 * x;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  const float val = static_cast<float>(vr[i]);
                  if (!(fabsf(val) < INFINITY)) o[i] = __float_as_uint(__uint_as_float(o[i]) + val);
                }
              }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t w[8];
#pragma unroll
              for (int k = 0; k < 8; ++k)
                w[k] = pack16<T>(__uint_as_float(o[16 * i + 2 * k]), __uint_as_float(o[16 * i + 2 * k + 1]));
              store32(dst + 32 * x + 16 * i, w, wide);
            }
          }
        }
      }
      tc_fence_before();
      vc_item += n;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Opts the kernel in to its shared memory, once per device.
template <typename T, int D>
bool smem_ready() {
  static bool done[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  if (dev < 64 && done[dev]) return true;
  if (cudaFuncSetAttribute(prompt_attn_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmem) !=
      cudaSuccess)
    return false;
  if (dev < 64) done[dev] = true;
  return true;
}

// Key tiles of tile `tile` of sequence i.
int key_tiles(const SeqTable& t, int i, int tile, int tokens) {
  const int end = t.kv_len[i] - t.q_len[i] + std::min(t.q_len[i], (tile + 1) * tokens);
  return end <= 0 ? 0 : (end + BK - 1) / BK;
}

// Sorts all (sequence, tile) pairs by their key tiles, descending, where few
// enough of them are passed along: dealt out forwards and backwards they then
// load the CTAs alike. With more of them every CTA has so many items that the
// order inside the sequences does. A counting sort: levels are key tiles.
int order_tiles(SeqTable& t, int tokens, int64_t pairs) {
  constexpr int kLevels = 4096;
  if (pairs > kMaxOrder || t.n > 65536) return 0;
  int most = 0;
  for (int i = 0; i < t.n; ++i) most = std::max(most, (t.kv_len[i] + BK - 1) / BK);
  if (most >= kLevels) return 0;
  auto level = [&](int i, int tile) { return key_tiles(t, i, tile, tokens); };
  int start[kLevels + 1];
  std::fill(start, start + most + 2, 0);
  for (int i = 0; i < t.n; ++i)
    for (int x = 0; x < t.tiles[i]; ++x) ++start[most - level(i, x) + 1];
  for (int l = 0; l < most; ++l) start[l + 1] += start[l];
  for (int i = 0; i < t.n; ++i)
    for (int x = t.tiles[i] - 1; x >= 0; --x)
      t.order[start[most - level(i, x)]++] = static_cast<uint32_t>(i) << 16 | static_cast<uint32_t>(x);
  return static_cast<int>(pairs);
}

// Chooses the CTA of every item of a sorted list where each CTA gets only a few: dealt out
// in turn, the third of three rounds lands on shares that are already equal (3,241 tokens,
// 8 key heads: the largest share 12% above the mean). An item's cost is its key tiles and,
// in quarters of one, item_cost. First every item goes, in order, to the CTA with the least
// so far; where that leaves the largest share more than 4% above the least possible (at
// 4,096 tokens, 2.7%, it measured 1% better than the other), every item goes to the
// fullest CTA that has room for it under a limit, which is raised from the least possible
// share until all fit. Dealt out and chosen: one image's prompt 86 and 80 us, nine ragged
// prompts of heads of 64 54 and 45, 1,024 items of 8,192 tokens 423 and 426 (so not for
// more than kMaxPacked). With 7 for heads of 128 86 and 436 us, with 10 for heads of 64 47.
// It takes the host 3 to 17 us, less than such a launch runs.
void choose_ctas(SeqTable& t, int tokens, int head_dim, int kv_heads, int ctas) {
  const int item_cost = head_dim == 128 ? 10 : 7;
  constexpr int kLevels = 2048;
  const int items = t.ordered * kv_heads;
  t.first[ctas] = 0;
  if (t.ordered == 0 || items > kMaxPacked || items <= ctas || ctas > kMaxCtas) return;
  int cost[kMaxPacked], sum = 0;
  for (int p = 0; p < t.ordered; ++p)
    for (int h = 0; h < kv_heads; ++h) {
      cost[p * kv_heads + h] = 4 * key_tiles(t, t.order[p] >> 16, t.order[p] & 0xFFFF, tokens) + item_cost;
      sum += cost[p * kv_heads + h];
    }
  const int least = std::max(cost[0], (sum + ctas - 1) / ctas);  // the largest share is at least this
  uint8_t cta[kMaxPacked];
  // the least loaded first: a heap of load << 8 | CTA
  int heap[kMaxCtas];
  for (int b = 0; b < ctas; ++b) heap[b] = b;
  const auto more = std::greater<int>();
  int most = 0;
  for (int i = 0; i < items; ++i) {
    std::pop_heap(heap, heap + ctas, more);
    int& top = heap[ctas - 1];
    cta[i] = static_cast<uint8_t>(top & 0xFF);
    top += cost[i] << 8;
    most = std::max(most, top >> 8);
    std::push_heap(heap, heap + ctas, more);
  }
  if (most * 100LL > least * 104LL && most < kLevels) {
    uint8_t fit[kMaxPacked];
    int16_t bin[kLevels], next[kMaxCtas];  // CTAs by their room, in lists
    for (int limit = least; limit < most; limit += 1 + limit / 128) {
      uint64_t some[kLevels / 64] = {};  // which lists have one
      std::fill(bin, bin + limit + 1, static_cast<int16_t>(-1));
      auto put = [&](int b, int room) {
        next[b] = bin[room];
        bin[room] = static_cast<int16_t>(b);
        some[room / 64] |= 1ull << (room % 64);
      };
      for (int b = ctas - 1; b >= 0; --b) put(b, limit);
      int i = 0;
      for (; i < items; ++i) {
        int w = cost[i] / 64;
        uint64_t bits = some[w] & (~0ull << (cost[i] % 64));
        while (bits == 0 && ++w <= limit / 64) bits = some[w];
        if (bits == 0) break;
        const int room = 64 * w + __builtin_ctzll(bits), b = bin[room];
        bin[room] = next[b];
        if (bin[room] < 0) some[w] &= ~(1ull << (room % 64));
        fit[i] = static_cast<uint8_t>(b);
        put(b, room - cost[i]);
      }
      if (i < items) continue;
      std::copy(fit, fit + items, cta);
      break;
    }
  }
  // by CTA, the largest first
  int at[kMaxCtas + 1] = {};
  for (int i = 0; i < items; ++i) ++at[cta[i] + 1];
  if (*std::max_element(at, at + ctas + 1) > kItemSlots) return;
  for (int b = 0; b < ctas; ++b) at[b + 1] += at[b];
  for (int b = 0; b <= ctas; ++b) t.first[b] = static_cast<uint16_t>(at[b]);
  for (int i = 0; i < items; ++i) t.item[at[cta[i]]++] = static_cast<uint16_t>(i);
}

// Tensor map of 16-bit [tokens, heads, D] with `stride` elements between
// tokens: 128-byte swizzle, box 64 columns x box_heads x box_tokens.
bool tmap_3d(CUtensorMap* map, bool half, const void* ptr, int64_t tokens, int heads, int d, int64_t stride,
             int box_heads, int box_tokens) {
  const uint64_t dims[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(heads), static_cast<uint64_t>(tokens)};
  const uint64_t strides[2] = {static_cast<uint64_t>(d) * 2, static_cast<uint64_t>(stride) * 2};
  const uint32_t box[3] = {64, static_cast<uint32_t>(box_heads), static_cast<uint32_t>(box_tokens)};
  return make_tmap_3d_16(map, half, ptr, dims, strides, box);
}

}  // namespace

int launch_prompt_attention(const PromptAttn& p, cudaStream_t s) {
  const int group = p.heads / p.kv_heads;
  const bool half = p.dtype == VLM_DTYPE_F16;
  int64_t total_q = 0, total_k = 0;
  for (int i = 0; i < p.n_seqs; ++i) {
    total_q += p.q_lens[i];
    total_k += p.kv_lens[i];
  }
  if (total_q == 0) return VLM_OK;
  CUtensorMap tq, tk, tv;
  const int tpt = kRows / group;
  // no key at all: the key and value maps are never used
  if (!tmap_3d(&tq, half, p.q, total_q, p.heads, p.head_dim, p.q_stride, group, tpt)) return VLM_ERR_CUDA;
  if (total_k > 0) {
    if (!tmap_3d(&tk, half, p.k, total_k, p.kv_heads, p.head_dim, p.k_stride, 1, BK) ||
        !tmap_3d(&tv, half, p.v, total_k, p.kv_heads, p.head_dim, p.v_stride, 1, BK))
      return VLM_ERR_CUDA;
  } else {
    tk = tv = tq;
  }
  auto run = [&](auto kern, int smem, bool ready) -> int {
    if (!ready) return VLM_ERR_CUDA;
    // the longest sequences first: their items are the largest
    std::vector<int> order(p.n_seqs);
    std::iota(order.begin(), order.end(), 0);
    std::vector<int> q0(p.n_seqs), k0(p.n_seqs);
    for (int i = 0, q = 0, k = 0; i < p.n_seqs; ++i) {
      q0[i] = q;
      k0[i] = k;
      q += p.q_lens[i];
      k += p.kv_lens[i];
    }
    std::stable_sort(order.begin(), order.end(), [&](int x, int y) { return p.kv_lens[x] > p.kv_lens[y]; });
    int launches = 0;
    for (int first = 0; first < p.n_seqs; first += kMaxSeqs) {
      Args a;
      a.t.n = 0;
      int64_t items = 0;
      for (int i = first; i < std::min(p.n_seqs, first + kMaxSeqs); ++i) {
        const int x = order[i];
        if (p.q_lens[x] == 0) continue;
        const int k = a.t.n++;
        a.t.off[k] = static_cast<int>(items);
        a.t.q0[k] = q0[x];
        a.t.k0[k] = k0[x];
        a.t.q_len[k] = p.q_lens[x];
        a.t.kv_len[k] = p.kv_lens[x];
        a.t.tiles[k] = static_cast<int>((static_cast<int64_t>(p.q_lens[x]) + 2 * tpt - 1) / (2 * tpt));
        items += static_cast<int64_t>(a.t.tiles[k]) * p.kv_heads;
        if (items > 0x7FFFFFFF - 65536) return VLM_ERR_BAD_SHAPE;
      }
      if (a.t.n == 0) continue;
      a.t.off[a.t.n] = static_cast<int>(items);
      a.t.ordered = order_tiles(a.t, 2 * tpt, items / p.kv_heads);
      a.kv_heads = p.kv_heads;
      a.group = group;
      a.tpt = tpt;
      a.sl2 = std::min(p.scale * 1.4426950408889634f, FLT_MAX);  // not infinite: it multiplies differences of 0
      a.v = p.v;
      a.v_stride = p.v_stride;
      a.out = p.out;
      a.out_stride = p.out_stride;
      a.status = p.status;
      for (int64_t at = 0; at < items;) {
        const int slots = std::min(num_sms(), kMaxCtas);
        const int n = static_cast<int>(std::min<int64_t>(items - at, static_cast<int64_t>(slots) * kItemSlots));
        choose_ctas(a.t, 2 * tpt, p.head_dim, p.kv_heads, std::min(n, slots));
        const cudaError_t e = launch_pdl(kern, dim3(std::min(n, slots)), dim3(kThreads), smem, s, tq, tk, tv, a,
                                         static_cast<int>(at), n);
        if (e != cudaSuccess) return VLM_ERR_CUDA;
        at += n;
        ++launches;
      }
    }
    note_extra_launches(launches - 1);
    return VLM_OK;
  };
  launch_begin(KC_PROMPT_ATTN, s);
  int rc;
  if (half)
    rc = p.head_dim == 128 ? run(prompt_attn_kernel<__half, 128>, Cfg<128>::kSmem, smem_ready<__half, 128>())
                           : run(prompt_attn_kernel<__half, 64>, Cfg<64>::kSmem, smem_ready<__half, 64>());
  else
    rc = p.head_dim == 128 ? run(prompt_attn_kernel<__nv_bfloat16, 128>, Cfg<128>::kSmem, smem_ready<__nv_bfloat16, 128>())
                           : run(prompt_attn_kernel<__nv_bfloat16, 64>, Cfg<64>::kSmem, smem_ready<__nv_bfloat16, 64>());
  launch_end(KC_PROMPT_ATTN, s);
  return rc;
}

}  // namespace vlm
