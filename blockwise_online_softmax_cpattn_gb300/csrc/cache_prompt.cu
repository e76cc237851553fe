// Attention of many new tokens over the 4-bit cache (chunks of a prompt, drafts of many
// heads) on the 5th-generation tensor cores.
//
// An item is 256 query rows of one request and K/V head; its units are 128 cached tokens.
// One CTA an SM takes an equal run of the line of items; items that cross CTAs are joined
// by a second, small launch.  Two softmax warpgroups, sides a and b, each own 128 rows'
// scores and output in TMEM: with more than 128 rows the sides are the item's two halves and
// work on the same tokens, so every tile of codes is turned into numbers once for 256 rows;
// an item of at most 128 rows goes to both sides, a taking its even and b its odd tiles, and
// their sums are joined at the end.  While one side forms its P, the tensor cores work for
// the other.
//
// Roles (512 threads):
//   warps 0, 1   issue side a's and b's MMAs: O += P V (P in TMEM, over the scores it came
//                from) and the next S = Q K^T (both operands in shared memory).
//   warp 2       loads codes, K and V of a tile apart, into a ring of three.
//   warp 3       keeps count of the tiles that are ready: sides that take turns pass over
//                tiles, and a barrier's phases can only be waited for one by one.
//   warps 4-7    side a's softmax, a thread a row; warps 8-11 side b's.
//   warps 12-15  turn codes into bf16 K and V tiles of 128 tokens with the 128-byte
//                swizzle that the MMA reads, two of each.
// A softmax thread holds its 128 scores in registers, which the other warpgroups give up
// (reading them from TMEM a second time to form P cost a third of the time).  O is rescaled
// only when the running maximum grew by more than 2^8 (exact after the division).
//
// Roundings: P becomes bf16, half a step 2^-9 of each term, because the MMA takes no wider operand;
// l sums it before that; all else is float32 up to the result.
//
// TMEM (512 columns): S_a [0,128), S_b [128,256), O_a, O_b D columns each from 256; P of a
// side takes the first 64 columns of its S.
// Every wait is bounded; on a time-out the CTA's roles give up, its copies and MMAs are
// drained and TMEM is freed.
//
// Measured (2048 new tokens behind 30000, 32 query heads, 8 K/V heads, D 128, group 64): 844 us,
// 1233 TFLOP/s (without the spans below 830), the tensor pipe 54 % busy.
// No unit is full: of the 3800 clocks that a tile takes, the tensor pipe works 54 %, and shared
// memory some 57 % by count (the MMAs' operands 1540 at its 128 bytes a clock, of which QK, that
// reads both from there, 1024; unpacking 640 to write and read codes).  What is left is latency: a
// side's chain from one tile's scores to the next's (128 scores a thread, a maximum, 128
// exponentials, P out, PV and the next QK), which the other side fills only in part.
// D 64: the same chunk with 32 and 8 heads 682 us, 763 TFLOP/s (half the products a score).
// Tried and slower: one warp that issues for both sides, or QK and PV apart; scores in halves
// of 64 tokens, the next half's formed under a half's softmax (939 us: queries are read twice
// as often); masks through TMEM; eight warps that unpack where 64 rows leave softmax warps over
// (132 us for 8 rows where this takes 97).  No change: codes, or the table's entries, loaded a
// step ahead.
#include <atomic>

#include "cache_work.cuh"

namespace cpattn {
namespace cprompt {

using namespace cattn;

constexpr int kTile = 128;      // cached tokens of a unit, rows of a side
constexpr int kRows = 256;      // query rows of an item
constexpr int kThreads = 512;
constexpr int kRing = 3;        // tiles' K or V codes in shared memory
// registers a thread: issuers and loader, dequantising, softmax (two warpgroups)
constexpr int kRegsLaunch = 128, kRegsIssue = 64, kRegsCodes = 80, kRegsSoftmax = 184;
static_assert(kRegsIssue + kRegsCodes + 2 * kRegsSoftmax <= 4 * kRegsLaunch, "an increase would wait forever");
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
constexpr int kItemCost = 3;    // queries in, results out, in units
// Tiles of a side after which its sums are folded.  An MMA cuts its sum off where a float32
// addition rounds: up to 2^-23 of the sum so far is lost at each of a tile's 8 steps, always
// downwards (a million tokens: o 6e-3 too small).  So O, m and l are kept a span at a time and
// folded into float32 sums in the workspace: at most 2^-13 of a span's sum is lost, little
// beside P's 2^-9 a term.
constexpr int kSpan = 128;   // (a power of 2)
using It = Item<kRows, kTile, kItemCost>;

template <int D, int G>
struct Smem {
  static constexpr int kOperand = kTile * D * 2;          // bf16 tile, also one side's Q
  static constexpr int kHalf = kCacheTile * (D / 2 + 4 * (D / G));  // of a tile in the cache
  static constexpr int kQ = 0;
  static constexpr int kK = 2 * kOperand;
  static constexpr int kV = kK + 2 * kOperand;
  static constexpr int kCode = kV + 2 * kOperand;
  static constexpr int kCodes = kTile / kCacheTile * kHalf;  // codes of a tile's K or V
  static constexpr int kBar = kCode + kRing * kCodes;
  // barriers: k_full[2], k_empty[2], v_full[2], v_empty[2], q_full[2], s_full[2], p_full[2],
  // o_full[2], o_free[2], share (stored, read), turn[2], done[2], codes full,
  // empty
  static constexpr int kNumBars = 24 + 2 * kRing;
  static constexpr int kMisc = kBar + kNumBars * 8;
  static constexpr int kBytes = kMisc + 16;
};

struct Static {
  int64_t sums[kSums];
  int64_t warp_part[kThreads / 32];
  It start;
  Place end;
  CtaMeta meta;
  uint32_t valid[8];   // per tile (the last 8): which of its 16-token tiles are there
  int abort;
  uint32_t tmem;
  volatile int seen_k, seen_v;   // tiles whose K, V is ready
};

// tmem_wait_ld with the loaded registers as operands, so that nothing that reads them can be
// moved above the wait.
#define CPATTN_RW8(i) "+r"(r[i + 0]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), \
                      "+r"(r[i + 4]), "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
__device__ __forceinline__ void tmem_wait_ld_of(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : CPATTN_RW8(0), CPATTN_RW8(8), CPATTN_RW8(16), CPATTN_RW8(24)
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait_ld_of(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" : CPATTN_RW8(0), CPATTN_RW8(8) : : "memory");
}

// Waits until *c reaches `want`, bounded as the waits for barriers are.
__device__ __forceinline__ bool count_wait(const volatile int* c, int want, volatile int* abort, const Params& p) {
  bool ok = *c >= want;
  if (!ok) {
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1; !(ok = *c >= want); ++i)
      if ((i & 63u) == 0 && (*abort || globaltimer_ns() - t0 > p.timeout_ns)) break;
    if (!ok && !*abort) {
      *abort = 1;
      latch_status(p.a.status, kStatusTimeout);
    }
  }
  ok = __all_sync(0xffffffffu, ok);
  __threadfence_block();
  return ok;
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t par, volatile int* abort, const Params& p) {
  return __all_sync(0xffffffffu, mbar_wait(bar, par, abort, p.a.status, p.timeout_ns));
}
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t par, const Params& p) {
  int never = 0;
  mbar_wait(bar, par, &never, nullptr, p.drain_ns());
}
// Workspace: a head and a tail slot per CTA, the CTAs' states, the spans' sums per CTA: O as
// [D / 4][rows] float4, (m, l) of the rows.
template <int D>
struct Work {
  static constexpr size_t kSums = (size_t)kRows * (D + 2);
  static __host__ __device__ size_t meta(int ctas) { return 2 * (size_t)ctas * Slot<D, kRows>::kFloats; }
  static __host__ __device__ size_t sums(int ctas) {
    return meta(ctas) + (ctas * sizeof(CtaMeta) + 15) / 16 * 4;
  }
  static __host__ __device__ size_t floats(int ctas) { return sums(ctas) + ctas * kSums; }
};
// A span's O (in TMEM), m and l of a thread's row join those of the spans before it (none: first):
// in the workspace, or, of an item's last span, in TMEM; m and l are returned.  Out of line and out of
// the loop over tiles: inlined into the softmax it cost 10 %, called from the loop 4.
template <int D>
__device__ __noinline__ float2 fold_span(const Params& p, uint32_t t_o, float m, float l, bool first, bool last) {
  float* const sums = static_cast<float*>(p.a.ws) + Work<D>::sums(gridDim.x) + (size_t)blockIdx.x * Work<D>::kSums;
  const int row = threadIdx.x - 128;   // of the two softmax warpgroups
  float4* const sum_o = reinterpret_cast<float4*>(sums) + row;
  float2* const sum_ml = reinterpret_cast<float2*>(sums + (size_t)kRows * D) + row;
  const float2 ml = first ? make_float2(-INFINITY, 0.f) : *sum_ml;
  const float mm = max_nan(m, ml.x), mb = mm == -INFINITY ? 0.f : mm;
  const float f = ex2(ml.x - mb), w = ex2(m - mb);
  const float2 joined = make_float2(mm, fmaf(ml.y, f, l * w));
#pragma unroll 1
  for (int c = 0; c < D / 16; ++c) {
    uint32_t o[16];
    tmem_ld16(t_o + c * 16, o);
    tmem_wait_ld_of(o);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float4* const at = sum_o + (c * 4 + j) * kRows;
      const float4 y = first ? make_float4(0.f, 0.f, 0.f, 0.f) : *at;
      const float4 v = make_float4(
          fmaf(y.x, f, w * __uint_as_float(o[4 * j])), fmaf(y.y, f, w * __uint_as_float(o[4 * j + 1])),
          fmaf(y.z, f, w * __uint_as_float(o[4 * j + 2])), fmaf(y.w, f, w * __uint_as_float(o[4 * j + 3])));
      if (!last) *at = v;
      o[4 * j] = __float_as_uint(v.x), o[4 * j + 1] = __float_as_uint(v.y);
      o[4 * j + 2] = __float_as_uint(v.z), o[4 * j + 3] = __float_as_uint(v.w);
    }
    if (last) tmem_st16(t_o + c * 16, o);
  }
  if (last) tmem_wait_st();
  else *sum_ml = joined;
  return joined;
}
// What both sides' walks have in common: the tiles [u, u + n) of an item, and which of them
// side x takes.
struct Part {
  int n, rows;
  bool split;   // the sides share the rows and alternate between tiles
  __device__ __forceinline__ int count(int x) const { return split ? (n + 1 - x) >> 1 : (x == 0 || rows > kTile ? n : 0); }
  __device__ __forceinline__ int tile(int x, int i) const { return split ? 2 * i + x : i; }
};
__device__ __forceinline__ Part part(const Params& p, const It& it, const Place& end) {
  Part t;
  t.n = it.left(end);
  t.rows = block_rows(p, it.q.nq, it.rb, kRows);
  t.split = t.rows <= kTile;
  return t;
}
// The next item of the run; false at its end.
__device__ __forceinline__ bool advance(const Params& p, It& it, const Place& end) {
  if (it.same(end)) return false;
  it.next(p);
  return it.r < p.a.n_req && it.left(end) > 0;
}

template <int D, int G>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ Params p) {
  using L = Smem<D, G>;
  using S = Slot<D, kRows>;
  constexpr int kTiles = kTile / kCacheTile;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ Static sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + L::kBar;
  auto bar = [&](int group, int i) { return bars + 8 * (2 * group + i); };
  enum { K_FULL, K_EMPTY, V_FULL, V_EMPTY, Q_FULL, S_FULL, P_FULL, O_FULL, O_FREE, SHARE, TURN, DONE, CODES };
  auto codes_full = [&](int i) { return bars + 8 * (2 * CODES + i); };
  auto codes_empty = [&](int i) { return bars + 8 * (2 * CODES + kRing + i); };
  volatile int* abort = &sh.abort;
  float* const ws = static_cast<float*>(p.a.ws);
  CtaMeta* const out_meta = reinterpret_cast<CtaMeta*>(ws + Work<D>::meta(gridDim.x));

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kNumBars; ++i) {
      const int group = i >> 1;
      int n = 1;
      if (group == K_FULL || group == V_FULL || group == TURN || i >= 2 * CODES + kRing) n = 4;  // a warpgroup's warps
      if (group == K_EMPTY || group == V_EMPTY) n = 3;  // both sides, the count's keeper
      if (group == Q_FULL || group == P_FULL || group == O_FREE || group == SHARE) n = 128;  // a side's threads
      // fault hook: one arrival more than there will be
      if (p.c.debug_fault == 2 && i == 2 * CODES) n = 2;
      mbar_init(bars + 8 * i, n);
    }
    sh.abort = (sbase & 1023u) ? 1 : 0;  // the layout has no alignment slack
    if (sh.abort) latch_status(p.a.status, kStatusLaunch);
    sh.seen_k = sh.seen_v = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(&sh.tmem), 512);
    tmem_relinquish();
  }
  const int64_t total = sum_costs<It, kThreads>(p, sh.sums, sh.warp_part);
  if (warp == 0) {
    int64_t c0, c1;
    cta_run(total, c0, c1);
    const It x = item_at<It>(p, sh.sums, lane < 16 ? c0 : c1);
    if (lane == 0) sh.start = x;
    if (lane == 16) sh.end = x;
    if (lane == 0) sh.meta.head = sh.meta.tail = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const Place end = sh.end;
  const bool any = sh.start.r < p.a.n_req && sh.start.left(end) > 0 && !*abort;
  bool ok = true;

  if (warp < 4) {
    regs_down<kRegsIssue>();
    if (!any) {
      // nothing to do
    } else if (warp == 2) {
      // ------------------------------------------------------------ codes
      // A ring of three: K and V halves of the tiles in turn.
      It it = sh.start;
      uint32_t n = 0;   // halves so far
      int slot = 0;
      uint32_t par = 0;
      do {
        const int tiles = it.left(end);
        for (int i = 0; ok && i < tiles; ++i) {
          // lane j < 8 loads 16-token tile j
          const int tok = (it.u + i) * kTile + lane * kCacheTile;
          int pg = -1;
          const int64_t at = (int64_t)it.r * p.a.max_pages + tok / p.c.page;
          if (lane < kTiles && tok < it.seen && page_at_ok(p, at)) pg = p.a.table[at];
          const bool there = (unsigned)pg < (unsigned)p.c.n_pages;
          const uint32_t have = __ballot_sync(0xffffffffu, there);
          const uint8_t* src = p.a.cache + it.h * p.c.block_bytes() + (there ? pg * p.page_bytes : 0) +
                               (int64_t)(tok % p.c.page / kCacheTile) * (2 * L::kHalf);
          for (int kv = 0; kv < 2; ++kv, ++n) {
            if (!(ok = warp_wait(codes_empty(slot), par ^ 1, abort, p))) break;
            if (lane == 0) {
              if (kv == 0) sh.valid[(n >> 1) & 7] = have;
              mbar_expect_tx(codes_full(slot), __popc(have) * L::kHalf);
            }
            __syncwarp();
            if (there)
              bulk_load(sbase + L::kCode + slot * L::kCodes + lane * L::kHalf, src + kv * L::kHalf, L::kHalf,
                        codes_full(slot));
            if (++slot == kRing) slot = 0, par ^= 1;
          }
        }
      } while (ok && advance(p, it, end));
      if (!ok && lane == 0) {
        // never leave with a copy still writing into this CTA's shared memory
        for (int i = 0; i < kRing; ++i)
          if (n >= (uint32_t)kRing - i) {
            drain_wait(codes_full(slot), par ^ 1, p);
            if (++slot == kRing) slot = 0, par ^= 1;
          }
      }
    } else if (warp == 3) {
      // ------------------------------------------------------------ which tiles are ready
      // A barrier's phases can only be waited for one by one, and a side that shares an item
      // passes over every other tile: this warp meets all of them and keeps count.  It takes
      // part in a tile's release, so no phase goes by it.
      It it = sh.start;
      uint32_t n = 0;
      do {
        const int tiles = it.left(end);
        for (int i = 0; ok && i < tiles; ++i, ++n) {
          if (!(ok = warp_wait(bar(K_FULL, n & 1), (n >> 1) & 1, abort, p))) break;
          if (lane == 0) {
            __threadfence_block();
            sh.seen_k = n + 1;
            mbar_arrive(bar(K_EMPTY, n & 1));
          }
          if (!(ok = warp_wait(bar(V_FULL, n & 1), (n >> 1) & 1, abort, p))) break;
          if (lane == 0) {
            __threadfence_block();
            sh.seen_v = n + 1;
            mbar_arrive(bar(V_EMPTY, n & 1));
          }
        }
      } while (ok && advance(p, it, end));
    } else {
      // ------------------------------------------------------------ MMAs of side `warp`
      // PV of a tile and the scores of the side's next one are issued back to back (the MMAs
      // of a thread execute in order, so the scores may overwrite the P that PV reads), with
      // every wait before them: a thread that committed MMAs waits for their end at its next
      // access to memory.
      const bool leader = elect_one();
      constexpr uint32_t kIdescS = idesc_bf16(128, 128, false, false);
      constexpr uint32_t kIdescPV = idesc_bf16(128, D, false, true);
      constexpr uint32_t kOp = L::kOperand >> 4;
      const int x = warp;
      const uint64_t qd = sdesc_sw128(sbase + L::kQ + x * L::kOperand, 16, 1024);
      const uint64_t kd = sdesc_sw128(sbase + L::kK, 16, 1024);
      const uint64_t vd = sdesc_sw128(sbase + L::kV, kTile * 128, 1024);
      const uint32_t t_s = tmem + x * 128, t_o = tmem + 256 + x * D;
      It it = sh.start;
      uint32_t base = 0, items = 0, n = 0;   // tiles of the items before; the side's items, scores
      do {
        const Part t = part(p, it, end);
        const int cnt = t.count(x);
        for (int i = 0; i <= cnt && cnt > 0; ++i) {
          const uint32_t gk = base + t.tile(x, i), gv = base + t.tile(x, i - 1);
          if (i > 0 && !(ok = count_wait(&sh.seen_v, gv + 1, abort, p))) break;
          // (sides that share an item wait for its K tiles one after the other: there PV goes first)
          if (i < cnt && (i == 0 || !t.split) && !(ok = count_wait(&sh.seen_k, gk + 1, abort, p))) break;
          if (i == 0 && !(ok = warp_wait(bar(Q_FULL, x), items & 1, abort, p))) break;
          if (i > 0) {
            if (i == 1 && items > 0 && !(ok = warp_wait(bar(O_FREE, x), (items - 1) & 1, abort, p))) break;
            if (!(ok = warp_wait(bar(P_FULL, x), (n - 1) & 1, abort, p))) break;
          }
          tc_fence_after();
          if (i > 0) {
            const uint64_t v = vd + (uint64_t)((gv & 1) * kOp);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              if (leader)
                mma_ts(t_o, t_s + kk * 8, v + (uint64_t)(kk * 128), kIdescPV,
                       (((i - 1) & (kSpan - 1)) != 0 || kk > 0) ? 1u : 0u);
            if (leader) {
              if (t.split) mbar_arrive(bar(V_EMPTY, gv & 1));  // for the side that passes it over
              mma_commit(bar(V_EMPTY, gv & 1));
              if (i == cnt) mma_commit(bar(O_FULL, x));
            }
          }
          if (i < cnt) {
            if (i > 0 && t.split) {
              __syncwarp();
              if (!(ok = count_wait(&sh.seen_k, gk + 1, abort, p))) break;
              tc_fence_after();
            }
            const uint64_t k = kd + (uint64_t)((gk & 1) * kOp);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * 1024 + (kk & 3) * 2;  // 16 KiB blocks, 32 B steps
              if (leader) mma_ss(t_s, qd + off, k + off, kIdescS, kk > 0);
            }
            if (leader) {
              mma_commit(bar(S_FULL, x));
              if (t.split) mbar_arrive(bar(K_EMPTY, gk & 1));
              mma_commit(bar(K_EMPTY, gk & 1));
            }
            ++n;
          }
          __syncwarp();
        }
        base += t.n;
        if (cnt > 0) ++items;
      } while (ok && advance(p, it, end));
      // every MMA has finished before TMEM can be freed
      if (leader) mma_commit(bar(DONE, x));
      __syncwarp();
      drain_wait(bar(DONE, x), 0, p);
    }
  } else if (warp >= 12) {
    regs_down<kRegsCodes>();
    if (any) {
      // ------------------------------------------------------------ codes -> bf16 operands
      // A thread takes 4 words (32 channels) of a row: Q neighbours a row.  The word order of
      // every second pair of lanes is turned, so that the eight 16-byte stores of a quarter of
      // the warp hit eight different bank groups under the swizzle (its rows differ by 1,
      // stored V rows by 2).
      constexpr int Q = D / 32;                 // threads of a row
      constexpr int kRowsAtOnce = 128 / Q, kSteps = kTile / kRowsAtOnce;
      static_assert(kSteps % 2 == 0, "two rows at a time");
      const int q = lane % Q, r0 = (threadIdx.x - 384) / Q;
      It it = sh.start;
      uint32_t n = 0;
      int slot = 0;
      uint32_t code_par = 0;
      do {
        const int tiles = it.left(end);
        for (int i = 0; ok && i < tiles; ++i, ++n) {
          const int left = it.q.len - (it.u + i) * kTile;  // tokens from the tile's first on
          const uint32_t st = n & 1, par = (n >> 1) & 1;
#pragma unroll 1
          for (int kv = 0; kv < 2; ++kv) {
            if (!(ok = warp_wait(codes_full(slot), code_par, abort, p))) break;
            if (!(ok = warp_wait(bar(kv ? V_EMPTY : K_EMPTY, st), par ^ 1, abort, p))) break;
            const uint32_t have = sh.valid[n & 7];
            const uint8_t* codes = smem + L::kCode + slot * L::kCodes;
            uint8_t* dst = smem + (kv ? L::kV : L::kK) + st * L::kOperand;
            // Two rows at a time, keys and values by the same instructions (one rotation more for
            // values): the only such warp of its scheduler has nothing else to wait with, and
            // what is fetched once serves both (851 -> 831 us).
#pragma unroll 1
            for (int s = 0; s < kSteps; s += 2) {
              uint4 w[2];
              uint32_t a2[2], z2[2];
              uint8_t* line[2];
              int swz[2];
              const int turn = q & 2 ? (kv ? 1 : 2) : 0;
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int stored = (s + e) * kRowsAtOnce + r0, tile = stored / kCacheTile, rr = stored % kCacheTile;
                // stored row t + 4e of eight is token 2t + e
                const int row = kv ? (stored & ~7) | ((stored & 3) << 1) | ((stored >> 2) & 1) : stored;
                const uint8_t* half = codes + tile * L::kHalf;
                w[e] = *reinterpret_cast<const uint4*>(half + rr * (D / 2) + q * 16);
                uint32_t az = *reinterpret_cast<const uint32_t*>(half + kCacheTile * (D / 2) + (rr * (D / G) + q * 32 / G) * 4);
                // rows nothing was appended to, or that were not loaded, hold anything: as zeros
                if (row >= left || !((have >> tile) & 1u)) az = 0u;
                a2[e] = az_a2(az);
                z2[e] = az_z2(az);
                line[e] = dst + (q >> 1) * (kTile * 128) + row * 128;
                swz[e] = row & 7;
              }
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                if (turn == 2) w[e] = make_uint4(w[e].z, w[e].w, w[e].x, w[e].y);
                if (turn == 1) w[e] = make_uint4(w[e].y, w[e].x, w[e].w, w[e].z);
              }
#pragma unroll
              for (int x = 0; x < 4; ++x)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const uint32_t ww = x == 0 ? w[e].x : x == 1 ? w[e].y : x == 2 ? w[e].z : w[e].w;
                  uint32_t u[4];
                  codes_to_bf16<true>(__funnelshift_l(ww, ww, kv ? 3 : 0), p.ones, u);
#pragma unroll
                  for (int y = 0; y < 4; ++y) u[y] = bf16x2_fma(u[y], a2[e], z2[e]);
                  const int chunk = (q & 1) * 4 + (x ^ turn);
                  *reinterpret_cast<uint4*>(line[e] + ((chunk ^ swz[e]) << 4)) = make_uint4(u[0], u[1], u[2], u[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(codes_empty(slot));
              mbar_arrive(bar(kv ? V_FULL : K_FULL, st));
            }
            if (++slot == kRing) slot = 0, code_par ^= 1;
          }
        }
      } while (ok && advance(p, it, end));
    }
  } else {
    regs_up<kRegsSoftmax>();
    if (any) {
      // ------------------------------------------------------------ softmax
      const int x = (warp - 4) >> 2;            // side
      const int row = (warp & 3) * 32 + lane;   // of the side; TMEM lane quadrant warp % 4
      const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
      const uint32_t t_s = tmem + lanes + x * 128, t_o = tmem + lanes + 256 + x * D;
      const float2 sl2 = make_float2(p.sl2, p.sl2);
      const float slack = 8.f / p.sl2;
      It it = sh.start;
      uint32_t n = 0, base = 0, items = 0;      // the side's tiles, all tiles, the side's items
      uint32_t shared = 0, turns = 0;           // items whose rows both sides had; tiles in turn
      bool more = true;
      // this thread's query row into shared memory (zeros behind the item's rows)
      auto load_q = [&](const It& a, const Part& t) {
        const int rho = t.split ? row : x * kTile + row;
        uint8_t* dst = smem + L::kQ + x * L::kOperand;
        const unsigned y = (unsigned)a.rb * kRows + rho, tok = y / (unsigned)p.n_rep;
        const bool in = rho < t.rows && token_ok(p, a.q.begin + (int)tok);
        const uint4* src = nullptr;
        if (in) {
          src = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.a.q) +
                                               (a.q.begin + (int)tok) * p.a.qs.token +
                                               (a.h * p.n_rep + (int)(y - tok * p.n_rep)) * p.a.qs.head);
        }
#pragma unroll 8
        for (int c = 0; c < D / 8; ++c) {
          const uint4 v = in ? src[c] : make_uint4(0u, 0u, 0u, 0u);
          *reinterpret_cast<uint4*>(dst + (c >> 3) * (kTile * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = v;
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(Q_FULL, x));
      };
      Part t = part(p, it, end);
      if (t.count(x) > 0) load_q(it, t);
      while (more && ok) {
        const int cnt = t.count(x);
        const int rho = t.split ? row : x * kTile + row;
        const int lim = seen_by(p, it.q, it.rb * kRows + rho);
        const int least = seen_by(p, it.q, it.rb * kRows + (t.split ? 0 : x * kTile));
        float m = -INFINITY, top = -INFINITY, l = 0.f;
#pragma unroll 1
        for (int from = 0, to; ok && from < cnt; from = to) {
          to = min(cnt, from + kSpan);
          if (from > 0) {
            // the span's sums join those before it; its last PV was done before the next scores
            if (!(ok = warp_wait(bar(S_FULL, x), n & 1, abort, p))) break;
            tc_fence_after();
            fold_span<D>(p, t_o, m, l, from == kSpan, false);
            m = top = -INFINITY;
            l = 0.f;
          }
          for (int i = from; i < to; ++i, ++n) {
            const int tile = t.tile(x, i);
            if (!(ok = warp_wait(bar(S_FULL, x), n & 1, abort, p))) break;
            // Sides with the same tiles take turns: side a's tile, then side b's once a is halfway.
            // Left alone they may fall in step, both working and then both waiting for the tensor
            // cores (up to 0.97 ms where this takes 0.83; with turns of a whole tile: 0.90).
            if (!t.split) {
              if ((x == 1 || turns > 0) && !(ok = warp_wait(bar(TURN, x), (turns - (x == 0)) & 1, abort, p))) break;
              ++turns;
            }
            tc_fence_after();
            const int tok0 = (it.u + tile) * kTile;
            const uint32_t have = sh.valid[(base + tile) & 7];
            const bool whole = have == (1u << kTiles) - 1 && tok0 + kTile <= least;
            // all 128 scores in registers: P goes over them in TMEM
            uint32_t r[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, r[c]);
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_wait_ld_of(r[c]);
            if (!whole) {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const int rel = lim - tok0 - 32 * c;   // columns below it are seen
                const int rel0 = (have >> (2 * c)) & 1u ? rel : 0, rel1 = (have >> (2 * c + 1)) & 1u ? rel : 0;
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (j >= (j < 16 ? rel0 : rel1)) r[c][j] = __float_as_uint(-INFINITY);
              }
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
              for (int j = 0; j < 32; j += 2)
                mx[(j >> 1) & 3] =
                    max3_nan(mx[(j >> 1) & 3], __uint_as_float(r[c][j]), __uint_as_float(r[c][j + 1]));
            const float hi = max_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3]);
            const bool over = !(hi <= top);
            float f = 1.f;
            if (over) {
              const float mn = max_nan(m, hi * p.sl2);
              f = ex2(m - mn);
              m = mn;
              top = hi + slack;
              l *= f;
            }
            if (i > from && __any_sync(0xffffffffu, over)) {
              // (these scores were formed after the PV before them was done)
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t o[16];
                tmem_ld16(t_o + c * 16, o);
                tmem_wait_ld_of(o);
#pragma unroll
                for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                tmem_st16(t_o + c * 16, o);
              }
            }
            const float nm = m == -INFINITY ? 0.f : -m;
            const float2 nm2 = make_float2(nm, nm);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t pk[16];
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                const float2 y =
                    fma2(make_float2(__uint_as_float(r[c][2 * j]), __uint_as_float(r[c][2 * j + 1])), sl2, nm2);
                const float2 e = make_float2(ex2(y.x), ex2(y.y));
                sum[j & 1] = add2(sum[j & 1], e);
                pk[j] = pack_bf16(e.x, e.y);
              }
              tmem_st16(t_s + c * 16, pk);
              if (c == 1 && !t.split && lane == 0) mbar_arrive(bar(TURN, 1 - x));
            }
            const float2 s2 = add2(sum[0], sum[1]);
            l += s2.x + s2.y;
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar(P_FULL, x));
          }
        }
        if (!ok) break;
        // the next item's queries, so that its first scores can start
        const It cur = it;
        const Part ct = t;
        more = advance(p, it, end);
        if (more) {
          t = part(p, it, end);
          if (t.count(x) > 0) load_q(it, t);
        }
        // ---------------------------------------------------------- the piece is done
        if (cnt > 0) {
          if (!(ok = warp_wait(bar(O_FULL, x), items & 1, abort, p))) break;
          ++items;
          tc_fence_after();
        }
        const bool starts = cur.u == 0, ends = cur.u + ct.n == cur.units, all = starts && ends;
        float* const slot = ws + (2 * (size_t)blockIdx.x + (starts ? 1 : 0)) * S::kFloats;
        // side b's share of the tiles of split rows goes through the slot's upper half
        const bool other = ct.split && ct.n > 1;
        const int out = other && x == 1 ? kTile + row : rho;
        const bool live = rho < ct.rows && (cnt > 0);
        if (cnt > kSpan) {
          const float2 ml = fold_span<D>(p, t_o, m, l, false, true);
          m = ml.x;
          l = ml.y;
        }
        // side b's rows of a slot may hold what side a has yet to read
        if (x == 1 && shared > 0 && (other || !all) &&
            !(ok = warp_wait(bar(SHARE, 1), (shared - 1) & 1, abort, p)))
          break;
        if (other && x == 1) {
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t r[32];
            tmem_ld32(t_o + c * 32, r);
            tmem_wait_ld_of(r);
            if (live) {
#pragma unroll
              for (int j = 0; j < 32; j += 4)
                *reinterpret_cast<float4*>(slot + (size_t)out * D + c * 32 + j) =
                    make_float4(__uint_as_float(r[j]), __uint_as_float(r[j + 1]), __uint_as_float(r[j + 2]),
                                __uint_as_float(r[j + 3]));
            }
          }
          if (live) S::ml(slot)[out] = make_float2(m, l);
          mbar_arrive(bar(SHARE, 0));
        }
        if (other && x == 0 && !(ok = warp_wait(bar(SHARE, 0), shared & 1, abort, p))) break;
        if (!(ct.split && x == 1) && cnt > 0) {
          float m1 = -INFINITY, l1 = 0.f;
          if (other && live) {
            const float2 ml = S::ml(slot)[kTile + row];
            m1 = ml.x;
            l1 = ml.y;
          }
          const float mm = max_nan(m, m1), mb = mm == -INFINITY ? 0.f : mm;
          const float w0 = ex2(m - mb), w1 = ex2(m1 - mb);
          const float ll = w0 * l + w1 * l1;
          const float inv = all ? inverse(ll) : 1.f;
          const int64_t orow = all && live ? out_row(p, cur.q.begin, cur.h, cur.rb, kRows, rho) : 0;
          const float a0 = w0 * inv, a1 = w1 * inv;
#pragma unroll 1
          for (int c = 0; c < D / 32; ++c) {
            uint32_t r[32];
            tmem_ld32(t_o + c * 32, r);
            tmem_wait_ld_of(r);
            if (live) {
#pragma unroll
              for (int j = 0; j < 32; j += 4) {
                float4 v = make_float4(a0 * __uint_as_float(r[j]), a0 * __uint_as_float(r[j + 1]),
                                       a0 * __uint_as_float(r[j + 2]), a0 * __uint_as_float(r[j + 3]));
                if (other) {
                  const float4 y = *reinterpret_cast<const float4*>(slot + (size_t)(kTile + row) * D + c * 32 + j);
                  v = make_float4(fmaf(a1, y.x, v.x), fmaf(a1, y.y, v.y), fmaf(a1, y.z, v.z), fmaf(a1, y.w, v.w));
                }
                if (all) store4(p, orow, D, c * 32 + j, v);
                else *reinterpret_cast<float4*>(slot + (size_t)rho * D + c * 32 + j) = v;
              }
            }
          }
          if (live) {
            if (!all) S::ml(slot)[rho] = make_float2(mm, ll);
            else store_lse(p, orow, mm, ll);
          }
        }
        if (other) {
          if (x == 0) mbar_arrive(bar(SHARE, 1));  // the slot's upper half may be written again
          ++shared;
        }
        if (cnt > 0) {
          tc_fence_before();
          mbar_arrive(bar(O_FREE, x));
        }
        if (row == 0 && x == 0 && !all) {
          if (!starts) {
            sh.meta.head = ends ? 1 : 2;
          } else {
            sh.meta.tail = 1;
            sh.meta.begin = cur.q.begin;
            sh.meta.nq = cur.q.nq;
            sh.meta.h = cur.h;
            sh.meta.rb = cur.rb;
          }
        }
        base += ct.n;
      }
    }
  }
  // (what follows runs on the registers that each warpgroup has left)
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  if (threadIdx.x == 0) out_meta[blockIdx.x] = sh.meta;
}

// Items that cross CTAs, in a launch of its own: the register split above does not leave the
// first kernel's warps alike enough to do it there.
template <int D>
__global__ void __launch_bounds__(kThreads) join_kernel(const __grid_constant__ Params p) {
  __shared__ __align__(16) uint8_t scratch[kJoinBytes<kThreads>];
  griddep_wait();
  const float* const ws = static_cast<const float*>(p.a.ws);
  join_ctas<D, kRows, kThreads>(
      p, reinterpret_cast<const CtaMeta*>(ws + Work<D>::meta(gridDim.x)), ws, scratch);
}

template <int D, int G>
static cudaError_t launch(Params p, int sms, cudaStream_t st) {
  auto kern = prompt_kernel<D, G>;
  constexpr int kSmem = Smem<D, G>::kBytes;
  static_assert(kSmem + sizeof(Static) <= 227 * 1024, "shared memory");
  static std::atomic<uint64_t> set[2];  // devices that are ready
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev >= 128 || !(set[dev >> 6].load() & bit)) {
    // a split that does not fit what the launch allocates would wait forever: refused
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kern)) != cudaSuccess) return e;
    if (fa.numRegs != kRegsLaunch) return cudaErrorInvalidConfiguration;
    if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) != cudaSuccess)
      return e;
    if (dev < 128) set[dev >> 6].fetch_or(bit);
  }
  const int grid = sms < kMaxSms ? sms : kMaxSms;
  kern<<<grid, kThreads, kSmem, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = kThreads;
  cfg.stream = st;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, join_kernel<D>, p);
}

}  // namespace cprompt

size_t cache_prompt_workspace(int D) {
  using namespace cprompt;
  return sizeof(float) * (D == 128 ? Work<128>::floats(kMaxSms) : Work<64>::floats(kMaxSms));
}

cudaError_t launch_cache_prompt(const cattn::Params& p, int sms, cudaStream_t st) {
  using namespace cprompt;
  if (p.c.D == 128)
    return p.c.G == 128  ? launch<128, 128>(p, sms, st)
           : p.c.G == 64 ? launch<128, 64>(p, sms, st)
                         : launch<128, 32>(p, sms, st);
  return p.c.G == 64 ? launch<64, 64>(p, sms, st) : launch<64, 32>(p, sms, st);
}

}  // namespace cpattn
