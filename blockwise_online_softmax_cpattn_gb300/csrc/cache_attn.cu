// Attention of new tokens over the 4-bit cache, for few query rows per K/V head
// (decoding steps, drafts; float32 always).
//
// A row's answer needs every cached byte once and little else: at D = 128, group 64 a
// token and K/V head is 144 bytes of HBM and 256 channels to turn into numbers, so the
// kernel's two bounds are the memory and, close behind, the instructions that unpack
// codes.  What it does about each:
//
//   Work.  Every warp on the GPU takes an equal run of the line of items (8 NT rows each,
//   units of 32 tokens).  Pieces are joined first among the warps of a CTA in shared
//   memory, then, for items that cross CTAs, by the CTA that began the item from the
//   workspace, with a flag for each piece (a grid barrier in their place cost 2 us more a
//   call, a second launch 4).
//
//   Loads.  A tile of 16 tokens of one K/V head is contiguous (codes and their (a, z)):
//   one bulk copy, of two tiles where a page holds both.  Each warp keeps a ring of
//   its own of them in flight and waits for nobody else.
//
//   Arithmetic.  S^T = K Q^T and O^T = V^T P^T with mma.m16n8k16: the cached operand is
//   the 16-row one, the query rows the 8 columns, so a decoding step's few rows fill
//   the instruction as well as they can.  The cached operand goes from shared memory
//   through registers: the layout of words and rows gives every lane the codes that
//   its operand fragment needs by one wide load a row, without conflicts, and turning
//   a pair of codes into a pair of bf16 values takes a shift, a logic operation and a
//   packed FMA.  The query rows of S^T's fragment become the rows of P^T's by one
//   8x8 transpose (movmatrix) a fragment.  (The fifth-generation MMA wants 64 or more
//   rows and its operands written back to shared memory: a decoding step would fill a
//   sixteenth of it.)
//   The running maximum of a row moves only when a score exceeds it by more than 8 in
//   log2 units; otherwise no lane needs to hear of the others' scores.
//
// float32 (NS = 3): q and P are sums of three bf16 numbers, the cached values are bf16
// numbers anyway, so three MMAs give products of float32 quality.
//
//   Roundings.  In bf16 P becomes bf16, half a step 2^-9 of each term, because the MMA takes no
//   wider operand, as in the library's other tensor-core kernels; l sums P before that.  All else
//   is kept in float32 up to the result; exponentials are the GPU's base-2 one, scores meet
//   scale log2 e in one multiplication.
//
//   Sums.  An MMA cuts its sum off where a float32 addition rounds: up to 2^-23 of the sum so
//   far is lost a step, always downwards, which grows with the tokens that one warp walks (o
//   6e-5 too small after 20000 tokens, 6e-3 after a million).  So O, m and l are kept a span of
//   units at a time and folded into float32 sums in the workspace after each (kSpan).  In
//   float32 a tile's O is an MMA sum of its own besides, which float32 additions join.
//
// Measured (D 128, group 64, 32 query heads and 8 K/V heads where not said):
//   128 requests of 100 to 16000 tokens, 0.94 GB: 191 us, 4.9 TB/s; a copy's rate is 6.8.
//   The arithmetic pipe that does shifts and logic is 63 % busy, 2.5 instructions a clock
//   issue: unpacking and the loads share the time.  (Shifts as high halves of products, on
//   the other pipe, took 238 us: they issue at half the rate.)
//   One request of 4096 tokens 14 us, of 131072 (8 heads each with its own, group 128) 46 us:
//   some 14 us of a call are no work on keys, but a launch, finding the run (3), the first
//   copy, the joins (3) and instructions that are fetched for the first time.
//   32 requests of 500 to 12000 tokens and up to 5 new ones on 4 K/V heads, 40 rows: 79 us,
//   three passes over the codes.  24, 32 and 40 rows at a time, queries in shared memory, took
//   88 to 99: fewer warps, each waiting for itself.
//   float32, 16 requests of 700 to 9000 tokens on 4 K/V heads: 31 us; 4000 new tokens
//   of 4 heads behind 20000: 1.8 ms.
//   The spans and the sums of a tile cost 1 to 4 % of all this (0 where items are short).
#include <math.h>

#include <algorithm>
#include <atomic>
#include <chrono>

#include "cache_work.cuh"

namespace cpattn {
namespace cattn {

constexpr int kUnit = 32;            // cached tokens of a unit: two tiles
// An item's start and end, in units.  1, 2, 3, 5, 8: 256 requests of 3 to 1023 tokens on 12 heads of
// 64 take 56, 49, 47, 50, 53 us; 128 of 100 to 16000 198, 189, 189, 190, 192.
constexpr int kItemCost = 3;

// Units after which the sums are folded (of few tokens: never).  bf16: 512 steps of an MMA, at
// most 2^-14 of the span's sum lost, little beside P's 2^-9 a term.  float32: 64 additions, each
// rounded to nearest, off by at most 2^-18 of it.
template <int NS>
constexpr int kSpan = NS == 1 ? 256 : 32;

// Workspace of a launch of at most `ctas` CTAs: a slot per warp (head pieces that other
// work followed), a head and a tail slot per CTA, the spans' sums per warp, a flag per CTA.
template <int D, int RB, int WARPS>
struct Work {
  static constexpr size_t kSlot = (size_t)Slot<D, RB>::kFloats;
  // a lane's numbers as the registers hold them, (m, l) of its rows and O: float4s side by side
  static constexpr size_t kSums = (size_t)RB / 8 * (1 + D / 16) * 32 * 4;
  static __host__ __device__ size_t cta_slots(int ctas) { return (size_t)ctas * WARPS * kSlot; }
  static __host__ __device__ size_t sums(int ctas) { return (size_t)ctas * (WARPS + 2) * kSlot; }
  static __host__ __device__ size_t flags(int ctas) { return sums(ctas) + (size_t)ctas * WARPS * kSums; }
};

// ---------------------------------------------------------------------------
// MMA fragments
// ---------------------------------------------------------------------------
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// A pair of floats as NS bf16 pairs that sum to it
template <int NS>
__device__ __forceinline__ void split_pair(float x, float y, uint32_t (&u)[NS]) {
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    u[s] = pack_bf16(x, y);
    if (s + 1 < NS) {
      x -= __uint_as_float(u[s] << 16);
      y -= __uint_as_float(u[s] & 0xffff0000u);
    }
  }
}

// What a warp tells the others of its CTA about its open pieces.
struct PieceMeta {
  int head;         // 0 none, 1 ends the item, 2 goes on
  int head_global;  // the head piece is in the workspace, not in shared memory
  int tail;         // 1: open
  int rows, begin, h, rb;      // of the tail's item
  int left;                    // its units behind the warp's run
  int head_rows;
};
template <typename It, int WARPS>
struct Shared {
  int64_t sums[kSums];          // inclusive prefix sums of cost over requests
  int64_t warp_part[WARPS];
  uint64_t bars[WARPS * 8];
  int abort;
  int ctas;                     // that have work
  uint64_t began;               // this CTA, in ns
  int64_t c0, c1, total;        // this CTA's run of the line, the line's length
  PieceMeta meta[WARPS];
  // per warp, what the main loop has no registers for: the items that are being loaded and
  // computed, and the run's end
  It in[WARPS], it[WARPS];
  Place end[WARPS];
};

// Cached tokens up to the end of the run's part of an item.
template <typename It>
__device__ __forceinline__ int piece_end(const It& it, const Place& end) {
  return (it.u + it.left(end)) * kUnit;
}

// Steps an item kept in shared memory to the next one (see cache_work.cuh: out of line).
template <typename It>
__device__ __noinline__ void next_item(const Params& p, It* it, const It* from) {
  It x = *from;
  x.next(p);
  __syncwarp();
  if ((threadIdx.x & 31) == 0) *it = x;
  __syncwarp();
}

// The run of this warp, its first unit and the next warp's, into sh.
template <typename It, int WARPS>
__device__ __forceinline__ void find_run(const Params& p, Shared<It, WARPS>& sh) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (p.a.n_req <= 32) {
    // Few requests: each warp finds its run by itself, a request a lane, with nothing to wait
    // for but the loads, and in 32 bits (the other way takes 1 us more to the first copy).
    Req q = {0, 0, 0};
    if (lane < p.a.n_req) q = request(p, lane);
    const int64_t wide = q.nq > 0 ? It::head_cost(p, q) * p.c.Hkv : 0;
    if (!__any_sync(0xffffffffu, wide >= (1 << 26))) {
      const int mine = (int)wide;
      int inc = mine;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, m);
        if (lane >= m) inc += y;
      }
      const int total = __shfl_sync(0xffffffffu, inc, 31);
      int c0, c1;
      cta_run(total, c0, c1);
      if (threadIdx.x == 0) {
        sh.ctas = max(1, min((int)gridDim.x, total));
        sh.c0 = c0;
        sh.c1 = c1;
        sh.total = max(1, total);
      }
#pragma unroll 1
      for (int e = 0; e < 2; ++e) {
        const int v = c0 + part_of(c1 - c0, warp + e, WARPS);
        const uint32_t past = __ballot_sync(0xffffffffu, inc > v);
        const int from = past ? __ffs(past) - 1 : 31;
        It x;
        x.h = x.rb = x.u = x.seen = x.units = 0;
        x.r = past ? from : p.a.n_req;
        x.q.begin = __shfl_sync(0xffffffffu, q.begin, from);
        x.q.nq = __shfl_sync(0xffffffffu, q.nq, from);
        x.q.len = __shfl_sync(0xffffffffu, q.len, from);
        const int all = __shfl_sync(0xffffffffu, mine, from), first = __shfl_sync(0xffffffffu, inc, from) - all;
        if (past) x.within(p, v - first, all / p.c.Hkv);
        if (lane == 0) {
          if (e == 0) sh.in[warp] = sh.it[warp] = x;
          else sh.end[warp] = x;
        }
      }
      return;
    }
  }
  const int64_t total = sum_costs<It, WARPS * 32>(p, sh.sums, sh.warp_part);
  int64_t c0, c1;
  cta_run(total, c0, c1);
  if (threadIdx.x == 0) {
    sh.ctas = (int)max((int64_t)1, min((int64_t)gridDim.x, total));
    sh.c0 = c0;
    sh.c1 = c1;
    sh.total = max((int64_t)1, total);
  }
  // one half of the lanes looks for each
  const It x = item_at<It>(p, sh.sums, c0 + part_of(c1 - c0, warp + (lane >> 4), WARPS));
  if (lane == 0) sh.in[warp] = sh.it[warp] = x;
  if (lane == 16) sh.end[warp] = x;
}

// The end of the kernel: joins the CTA's open pieces, then the items that cross CTAs.
template <int D, typename It, int WARPS>
__device__ __forceinline__ void finish(const Params& p, const Shared<It, WARPS>& sh, uint8_t* smem, int stage_bytes) {
  constexpr int RB = It::kRows;
  using S = Slot<D, RB>;
  using W = Work<D, RB, WARPS>;
  const int lane = threadIdx.x & 31;
  const PieceMeta* meta = sh.meta;
  float* const ws = static_cast<float*>(p.a.ws);
  uint64_t* const flags = reinterpret_cast<uint64_t*>(ws + W::flags(gridDim.x));
  // ---- the CTA's pieces -------------------------------------------------------
  // Pieces in order: number 2 w is warp w's head, 2 w + 1 its tail.  A tail begins a group
  // of pieces of one item, a head that ends the item closes one.  The rows of the groups are
  // shared out among the warps, 4 channels a lane.
  static_assert(2 * WARPS <= 32, "a bit per piece");
  const int warp = threadIdx.x >> 5;
  const bool mine = lane < 2 * WARPS;
  const int state = !mine ? 0 : (lane & 1) ? meta[lane >> 1].tail : meta[lane >> 1].head;
  const uint32_t pieces = __ballot_sync(0xffffffffu, state != 0);
  const uint32_t tails = __ballot_sync(0xffffffffu, (lane & 1) && state != 0);
  const uint32_t closing = __ballot_sync(0xffffffffu, !(lane & 1) && state == 1);
  const uint32_t leads = tails | (pieces & (0u - pieces));
  float* const cta_slots = ws + W::cta_slots(gridDim.x) + 2 * (size_t)blockIdx.x * S::kFloats;
  int k = 0;
#pragma unroll 1
  for (uint32_t lead = leads; lead; lead &= lead - 1, ++k) {
    const uint32_t first = lead & (0u - lead), rest = lead & (lead - 1);
    const uint32_t ids = pieces & (rest ? (rest & (0u - rest)) - first : 0u - first);
    const bool begun = (first & tails) != 0, ended = (ids & closing) != 0;
    const PieceMeta& own = meta[(__ffs(first) - 1) >> 1];
    const int rows = begun ? own.rows : own.head_rows;
    float* const to = cta_slots + (begun ? S::kFloats : 0);
    // RPW rows at a time: row r of group k is the job of warp (k RB + r) / RPW
    constexpr int V = D / 4, RPW = 32 / V;
#pragma unroll 1
    for (int row = ((warp + 64 * WARPS - k * (RB / RPW)) % WARPS) * RPW + lane / V; row < rows; row += WARPS * RPW) {
      const int ch = lane % V * 4;
      Acc acc;
#pragma unroll 1
      for (uint32_t b = ids; b; b &= b - 1) {
        const int id = __ffs(b) - 1, w = id >> 1;
        const float* s = (id & 1) == 0 && meta[w].head_global
                             ? ws + ((size_t)blockIdx.x * WARPS + w) * S::kFloats
                             : reinterpret_cast<const float*>(smem + (size_t)w * p.stages * stage_bytes);
        acc.add(S::ml(s)[row], *reinterpret_cast<const float4*>(s + row * D + ch));
      }
      if (begun && ended) {
        write_out<D>(p, out_row(p, own.begin, own.h, own.rb, RB, row), ch, acc.m, acc.l, acc.o);
      } else {
        *reinterpret_cast<float4*>(to + row * D + ch) = acc.o;
        if (ch == 0) S::ml(to)[row] = make_float2(acc.m, acc.l);
      }
    }
  }

  // ---- items that cross CTAs ----------------------------------------------------
  // The CTA that began one waits for the head pieces of the CTAs behind it up to the one that
  // ends the item (which wait for nobody before they publish theirs; all CTAs are resident)
  // and joins them with its tail.  How many those are follows from the line.  A flag is this
  // launch's own number, put there by the piece's CTA and taken away by the one that waits.
  __syncthreads();  // the slots are written
  if (sh.abort) return;
  if ((pieces & ~tails & (leads & (0u - leads))) && threadIdx.x == 0) {
    __threadfence();
    asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(flags + blockIdx.x), "l"(p.publish) : "memory");
  }
  const int last = tails ? 31 - __clz(tails) : 0;
  if (!tails || (closing >> last)) return;
  const PieceMeta own = meta[last >> 1];
  const int64_t item_end = sh.c0 + part_of(sh.c1 - sh.c0, (last >> 1) + 1, WARPS) + own.left;
  const int64_t scaled = item_end * sh.ctas + sh.total - 1;
  const int past = scaled <= 0x7fffffff ? (int)((unsigned)scaled / (unsigned)sh.total) : (int)divide(scaled, sh.total);
  const int behind = min(past - 1, sh.ctas - 1) - (int)blockIdx.x;
  // (CTAs begin together and their runs are equal: one that takes as long again has failed)
  bool ok = true;
  for (int i = threadIdx.x; i < behind; i += WARPS * 32) {
    uint64_t* const f = flags + blockIdx.x + 1 + i;
    uint64_t v = 0;
    const uint64_t t0 = globaltimer_ns(), limit = p.timeout_ns + (t0 - sh.began);
    for (uint32_t it = 1;; ++it) {
      asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(f) : "memory");
      if (v == p.nonce || ((it & 63u) == 0 && globaltimer_ns() - t0 > limit)) break;
    }
    ok = ok && v == p.nonce;
    *f = 0;
  }
  if (!__syncthreads_and(ok)) {
    if (threadIdx.x == 0) latch_status(p.a.status, kStatusTimeout);
    return;
  }
  // few numbers leave threads over: those share the pieces and meet in shared memory
  constexpr int V = D / 4, THREADS = WARPS * 32;
  const int parts = own.rows * V, n = behind + 1;
  const int shares = max(1, min(THREADS / parts, n)), share = threadIdx.x / parts;
  Acc* const meet = reinterpret_cast<Acc*>(smem);
#pragma unroll 1
  for (int e = shares > 1 ? threadIdx.x % parts : threadIdx.x; e < parts; e += shares > 1 ? parts : THREADS) {
    const int row = e / V, ch = (e - row * V) * 4;
    Acc acc;
    if (share < shares || shares == 1) {
#pragma unroll 4
      for (int i = shares > 1 ? share : 0; i < n; i += shares) {
        const float* q = cta_slots + (i ? 2 * (size_t)i : 1) * S::kFloats;
        acc.add(__ldcg(S::ml(q) + row), __ldcg(reinterpret_cast<const float4*>(q + row * D + ch)));
      }
    }
    if (shares > 1) meet[threadIdx.x] = acc;
    else write_out<D>(p, out_row(p, own.begin, own.h, own.rb, RB, row), ch, acc.m, acc.l, acc.o);
  }
  if (shares == 1) return;
  __syncthreads();
  if ((int)threadIdx.x >= parts) return;
  Acc acc = meet[threadIdx.x];
#pragma unroll 1
  for (int i = 1; i < shares; ++i) {
    const Acc& x = meet[threadIdx.x + i * parts];
    acc.add(make_float2(x.m, x.l), x.o);
  }
  const int row = threadIdx.x / V, ch = (threadIdx.x - row * V) * 4;
  write_out<D>(p, out_row(p, own.begin, own.h, own.rb, RB, row), ch, acc.m, acc.l, acc.o);
}

template <int D, int G, int NT, int NS, int WARPS, int MINB>
__global__ void __launch_bounds__(WARPS * 32, MINB) attn_kernel(const __grid_constant__ Params p) {
  constexpr int RB = 8 * NT;
  constexpr int KW = D / 32;    // words of a K row per lane (channels 8 KW t4 ..)
  constexpr int VW = D / 64;    // words of a V row per lane (channels 8 VW g ..)
  constexpr int MT = D / 16;    // 16-channel tiles of O^T
  using S = Slot<D, RB>;
  using W = Work<D, RB, WARPS>;
  extern __shared__ __align__(128) uint8_t smem[];
  using It = Item<RB, kUnit, kItemCost>;
  __shared__ Shared<It, WARPS> sh;
  PieceMeta* const meta = sh.meta;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t4 = lane & 3;
  constexpr int par_words = D / G;
  constexpr int half = kCacheTile * (D / 2 + 4 * par_words);
  constexpr int tile_bytes = 2 * half, stage_bytes = 2 * tile_bytes;
  volatile int* abort = &sh.abort;
  if (threadIdx.x == 0) {
    sh.abort = 0;
    sh.began = globaltimer_ns();
  }
  if (lane == 0) {
#pragma unroll 1
    for (int s = 0; s < p.stages; ++s)  // fault hook: one arrival more than there will be
      mbar_init(smem_u32(&sh.bars[warp * 8 + s]), p.c.debug_fault == 1 ? 2 : 1);
    fence_barrier_init();
  }
  __syncthreads();

  find_run(p, sh);
  float* const slot_smem = reinterpret_cast<float*>(smem + (size_t)warp * p.stages * stage_bytes);
  if (lane == 0) {
    meta[warp].head = 0;
    meta[warp].tail = 0;
  }
  __syncwarp();
  bool ok = true;
  int to_issue = sh.in[warp].r < p.a.n_req ? sh.in[warp].left(sh.end[warp]) : 0;  // units of the item
  if (to_issue > 0) {
    const uint32_t ring = smem_u32(slot_smem), bar0 = smem_u32(&sh.bars[warp * 8]);
    int stage_in = 0, stage = 0;
    uint32_t parity = 0, valid = 0;  // two bits a stage: which tiles were loaded
    // Pages of the coming tiles: lane i knows that of the i-th, or where units are inside
    // pages (a page is a multiple of 32 tokens), of the i-th unit.
    const int per_lane = p.unit_in_page ? 1 : 2;
    int tab = 0, tab_k = 32;         // the next unit's first lane
    int w0 = 0;                      // the unit's first tile in its page
    const uint8_t* from = nullptr;   // the item's K/V head in page 0
    // issues the copies of the next unit
    auto issue = [&]() {
      if (tab_k == 32) {
        const It& in = sh.in[warp];
        const int64_t tok = ((int64_t)in.u * per_lane + lane) * (kUnit / per_lane);
        const int64_t at = (int64_t)in.r * p.a.max_pages + tok / p.c.page;
        tab = tok < in.seen && page_at_ok(p, at) ? p.a.table[at] : -1;
        from = p.a.cache + in.h * p.c.block_bytes();
        w0 = (in.u * 2) % p.page_tiles;
        tab_k = 0;
        __syncwarp();
        if (lane == 0) sh.in[warp].u += 32 / per_lane;  // where the next look at the table starts
      }
      const uint32_t bar = bar0 + 8 * stage_in;
      const uint32_t dst = ring + stage_in * stage_bytes;
      const int pg = __shfl_sync(0xffffffffu, tab, p.unit_in_page ? tab_k : tab_k + (lane & 1));
      const bool page_ok = (unsigned)pg < (unsigned)p.c.n_pages;
      uint32_t have;
      if (p.unit_in_page) {
        // (of an item's last unit the second tile may lie past its end: it is masked)
        have = page_ok ? 3u : 0u;
        if (lane == 0) {
          mbar_expect_tx(bar, page_ok ? stage_bytes : 0);
          if (page_ok) bulk_load(dst, from + pg * p.page_bytes + (int64_t)w0 * tile_bytes, stage_bytes, bar);
        }
        w0 = w0 + 2 == p.page_tiles ? 0 : w0 + 2;
      } else {
        // a lane a tile
        have = __ballot_sync(0xffffffffu, page_ok) & 3u;
        if (lane == 0) mbar_expect_tx(bar, __popc(have) * tile_bytes);
        __syncwarp();
        const int w = w0 + (lane & 1);
        if (lane < 2 && page_ok)
          bulk_load(dst + lane * tile_bytes, from + pg * p.page_bytes + (int64_t)(w < p.page_tiles ? w : 0) * tile_bytes,
                    tile_bytes, bar);
        w0 = (w0 + 2) % p.page_tiles;
      }
      tab_k += per_lane;
      valid = (valid & ~(3u << (2 * stage_in))) | have << (2 * stage_in);
      if (++stage_in == p.stages) stage_in = 0;
      if (--to_issue == 0) {
        if (!sh.in[warp].same(sh.end[warp])) {
          next_item(p, &sh.in[warp], &sh.in[warp]);
          to_issue = sh.in[warp].r < p.a.n_req ? sh.in[warp].left(sh.end[warp]) : 0;
          tab_k = 32;
        }
      }
    };
#pragma unroll 1
    for (int s = 0; s < p.stages && to_issue > 0; ++s) issue();

#pragma unroll 1
    for (bool more = true; more;) {
      const int len = sh.it[warp].q.len;
      int tok0 = sh.it[warp].u * kUnit;
      uint32_t qf[NT][NS][KW][4];
      int lim[NT][2], least;
      {
        const It it = sh.it[warp];
        const int rows = block_rows(p, it.q.nq, it.rb, RB);
        // query fragments: column g of every 8, channels 8 KW t4 ..
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int rho = n * 8 + g;
#pragma unroll
          for (int s = 0; s < NS; ++s)
#pragma unroll
            for (int w = 0; w < KW; ++w)
#pragma unroll
              for (int i = 0; i < 4; ++i) qf[n][s][w][i] = 0;
          const unsigned x = (unsigned)it.rb * RB + rho, tok = x / (unsigned)p.n_rep;
          if (rho < rows && token_ok(p, it.q.begin + (int)tok)) {
            const int64_t at = (it.q.begin + (int)tok) * p.a.qs.token +
                               (it.h * p.n_rep + (int)(x - tok * p.n_rep)) * p.a.qs.head + 8 * KW * t4;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
              if constexpr (NS == 1) {
                const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.a.q) + at + 8 * w);
                qf[n][0][w][0] = v.x, qf[n][0][w][1] = v.y, qf[n][0][w][2] = v.z, qf[n][0][w][3] = v.w;
              } else {
                const float* src = static_cast<const float*>(p.a.q) + at + 8 * w;
                const float4 x0 = reinterpret_cast<const float4*>(src)[0], x1 = reinterpret_cast<const float4*>(src)[1];
                const float f[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  uint32_t u[NS];
                  split_pair<NS>(f[2 * i], f[2 * i + 1], u);
#pragma unroll
                  for (int s = 0; s < NS; ++s) qf[n][s][w][i] = u[s];
                }
              }
            }
          }
        }
        // columns 2 t4, 2 t4 + 1 of every 8: how many keys the row sees
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) lim[n][e] = seen_by(p, it.q, it.rb * RB + n * 8 + 2 * t4 + e);
        least = seen_by(p, it.q, it.rb * RB);
      }
      // m: the maximum in log2 units that P is formed against; top: the raw score above
      // which it moves
      const float slack = 8.f / p.sl2;
      float m[NT][2], top[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll 1
      for (;;) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          m[n][0] = m[n][1] = -INFINITY;
          top[n][0] = top[n][1] = -INFINITY;
          l[n][0] = l[n][1] = 0.f;
#pragma unroll
          for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
        }

        const int stop = min(tok0 + kSpan<NS> * kUnit, piece_end(sh.it[warp], sh.end[warp]));
#pragma unroll 1
        for (; tok0 < stop; tok0 += kUnit) {
          ok = mbar_wait(bar0 + 8 * stage, (parity >> stage) & 1u, abort, p.a.status, p.timeout_ns);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          parity ^= 1u << stage;
          const uint32_t have = (valid >> (2 * stage)) & 3u;
          const uint8_t* base = reinterpret_cast<const uint8_t*>(slot_smem) + stage * stage_bytes;
          // every row sees every token of the unit
          const bool whole = have == 3u && tok0 + kUnit <= least;

          // ---- S^T = K Q^T -------------------------------------------------------
          float sc[2][NT][4];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint8_t* kt = base + i * tile_bytes;
            uint32_t w0[KW], w1[KW];
            if constexpr (KW == 4) {
              const uint4 x = *reinterpret_cast<const uint4*>(kt + g * (D / 2) + 16 * t4);
              const uint4 y = *reinterpret_cast<const uint4*>(kt + (g + 8) * (D / 2) + 16 * t4);
              w0[0] = x.x, w0[1] = x.y, w0[2] = x.z, w0[3] = x.w;
              w1[0] = y.x, w1[1] = y.y, w1[2] = y.z, w1[3] = y.w;
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(kt + g * (D / 2) + 8 * t4);
              const uint2 y = *reinterpret_cast<const uint2*>(kt + (g + 8) * (D / 2) + 8 * t4);
              w0[0] = x.x, w0[1] = x.y;
              w1[0] = y.x, w1[1] = y.y;
            }
            const uint32_t* par = reinterpret_cast<const uint32_t*>(kt + kCacheTile * (D / 2));
            const int grp = 8 * KW * t4 / G;
            const uint32_t az0 = par[g * par_words + grp], az1 = par[(g + 8) * par_words + grp];
            const uint32_t a0 = az_a2(az0), z0 = az_z2(az0), a1 = az_a2(az1), z1 = az_z2(az1);
#pragma unroll
            for (int n = 0; n < NT; ++n) sc[i][n][0] = sc[i][n][1] = sc[i][n][2] = sc[i][n][3] = 0.f;
#pragma unroll
            for (int w = 0; w < KW; ++w) {
              uint32_t x[4], y[4];
              codes_to_bf16<true>(w0[w], p.ones, x);
              codes_to_bf16<true>(w1[w], p.ones, y);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                x[q] = bf16x2_fma(x[q], a0, z0);
                y[q] = bf16x2_fma(y[q], a1, z1);
              }
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int s = NS - 1; s >= 0; --s) {
                  mma16816(sc[i][n], x[0], y[0], x[1], y[1], qf[n][s][w][0], qf[n][s][w][1]);
                  mma16816(sc[i][n], x[2], y[2], x[3], y[3], qf[n][s][w][2], qf[n][s][w][3]);
                }
            }
          }

          // ---- softmax -----------------------------------------------------------
          if (!whole) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const int tok = tok0 + i * kCacheTile + g + (j >> 1) * 8;
                  if (!((have >> i) & 1u) || tok >= lim[n][j & 1]) sc[i][n][j] = -INFINITY;
                }
          }
          uint32_t pf[2][NT][NS][2];
          {
            float mx[NT][2];
            bool over = false;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                mx[n][e] = max3_nan(sc[0][n][e], sc[0][n][e + 2], max_nan(sc[1][n][e], sc[1][n][e + 2]));
                over |= !(mx[n][e] <= top[n][e]);
              }
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  float x = mx[n][e];
#pragma unroll
                  for (int q = 4; q < 32; q <<= 1) x = max_nan(x, __shfl_xor_sync(0xffffffffu, x, q));
                  // rows whose maximum did not move that far keep it
                  if (x <= top[n][e]) continue;
                  const float mn = max_nan(m[n][e], x * p.sl2);
                  const float f = ex2(m[n][e] - mn);
                  m[n][e] = mn;
                  top[n][e] = x + slack;
                  l[n][e] *= f;
#pragma unroll
                  for (int t = 0; t < MT; ++t) {
                    o[n][t][e] *= f;
                    o[n][t][e + 2] *= f;
                  }
                }
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
              for (int n = 0; n < NT; ++n) {
                const float2 sl2 = make_float2(p.sl2, p.sl2);
                const float2 nm = make_float2(m[n][0] == -INFINITY ? 0.f : -m[n][0],
                                              m[n][1] == -INFINITY ? 0.f : -m[n][1]);
                const float2 x = fma2(make_float2(sc[i][n][0], sc[i][n][1]), sl2, nm);
                const float2 y = fma2(make_float2(sc[i][n][2], sc[i][n][3]), sl2, nm);
                const float pr[4] = {ex2(x.x), ex2(x.y), ex2(y.x), ex2(y.y)};
                const float2 sum = add2(make_float2(pr[0], pr[1]), make_float2(pr[2], pr[3]));
                const float2 ll = add2(make_float2(l[n][0], l[n][1]), sum);
                l[n][0] = ll.x;
                l[n][1] = ll.y;
                uint32_t u[NS], v[NS];
                split_pair<NS>(pr[0], pr[1], u);
                split_pair<NS>(pr[2], pr[3], v);
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                  pf[i][n][s][0] = transpose8x8(u[s]);
                  pf[i][n][s][1] = transpose8x8(v[s]);
                }
              }
          }

          // ---- O^T += V^T P^T ----------------------------------------------------
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint8_t* vt = base + i * tile_bytes + half;
            const uint32_t* par = reinterpret_cast<const uint32_t*>(vt + kCacheTile * (D / 2));
            const int grp = 8 * VW * g / G;
            // tokens 2 t4, 2 t4 + 1, 2 t4 + 8, 2 t4 + 9 are in rows t4, t4 + 4, t4 + 8, t4 + 12
            uint32_t w[4][VW], az[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int row = t4 + 4 * e;
              if constexpr (VW == 2) {
                const uint2 x = *reinterpret_cast<const uint2*>(vt + row * (D / 2) + 8 * g);
                w[e][0] = x.x, w[e][1] = x.y;
              } else {
                w[e][0] = *reinterpret_cast<const uint32_t*>(vt + row * (D / 2) + 4 * g);
              }
              az[e] = par[row * par_words + grp];
            }
            if (!whole) {
              // rows nothing was appended to, or that were not loaded, hold anything: as zeros
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int tok = tok0 + i * kCacheTile + 2 * t4 + (e & 1) + (e >> 1) * 8;
                if (!((have >> i) & 1u) || tok >= len) az[e] = 0u;
              }
            }
            const uint32_t a0 = __byte_perm(az[0], az[1], 0x5410), z0 = __byte_perm(az[0], az[1], 0x7632);
            const uint32_t a1 = __byte_perm(az[2], az[3], 0x5410), z1 = __byte_perm(az[2], az[3], 0x7632);
#pragma unroll
            for (int j = 0; j < VW; ++j) {
              uint32_t x0[4], x1[4], y0[4], y1[4];  // even and odd channels of tokens t.., of t + 8..
              codes_to_bf16<false>(__byte_perm(w[0][j], w[1][j], 0x5410), p.ones, x0);
              codes_to_bf16<false>(__byte_perm(w[0][j], w[1][j], 0x7632), p.ones, x1);
              codes_to_bf16<false>(__byte_perm(w[2][j], w[3][j], 0x5410), p.ones, y0);
              codes_to_bf16<false>(__byte_perm(w[2][j], w[3][j], 0x7632), p.ones, y1);
#pragma unroll
              for (int q = 0; q < 4; ++q) {
                const uint32_t f0 = bf16x2_fma(x0[q], a0, z0), f1 = bf16x2_fma(x1[q], a0, z0);
                const uint32_t f2 = bf16x2_fma(y0[q], a1, z1), f3 = bf16x2_fma(y1[q], a1, z1);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                  float(&to)[4] = o[n][j * 4 + q];
                  if constexpr (NS == 1) {
                    mma16816(to, f0, f1, f2, f3, pf[i][n][0][0], pf[i][n][0][1]);
                  } else {
                    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int s = NS - 1; s >= 0; --s)
                      mma16816(d, f0, f1, f2, f3, pf[i][n][s][0], pf[i][n][s][1]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) to[e] += d[e];
                  }
                }
              }
            }
          }
          // the stage has been read
          __syncwarp();
          if (++stage == p.stages) stage = 0;
          if (to_issue > 0) issue();
        }
        if (!ok) break;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int q = 4; q < 32; q <<= 1) l[n][e] += __shfl_xor_sync(0xffffffffu, l[n][e], q);
        // ---- the span is done ----------------------------------------------------
        const bool held = sh.it[warp].u * kUnit + kSpan<NS> * kUnit < tok0;   // there were spans before
        const bool more_spans = tok0 < piece_end(sh.it[warp], sh.end[warp]);
        if (held || more_spans) {
          // with the earlier spans' sums, in each lane's own place
          float4* const sum = reinterpret_cast<float4*>(
                                  static_cast<float*>(p.a.ws) + W::sums(gridDim.x) +
                                  ((size_t)blockIdx.x * WARPS + warp) * W::kSums) + lane;
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            float4* const at = sum + n * (1 + MT) * 32;
            const float4 ml = held ? at[0] : make_float4(-INFINITY, -INFINITY, 0.f, 0.f);
            const float mx0 = max_nan(m[n][0], ml.x), mx1 = max_nan(m[n][1], ml.y);
            const float b0 = mx0 == -INFINITY ? 0.f : mx0, b1 = mx1 == -INFINITY ? 0.f : mx1;
            const float f0 = ex2(ml.x - b0), f1 = ex2(ml.y - b1), w0 = ex2(m[n][0] - b0), w1 = ex2(m[n][1] - b1);
            m[n][0] = mx0;
            m[n][1] = mx1;
            l[n][0] = fmaf(ml.z, f0, l[n][0] * w0);
            l[n][1] = fmaf(ml.w, f1, l[n][1] * w1);
            if (more_spans) at[0] = make_float4(m[n][0], m[n][1], l[n][0], l[n][1]);
#pragma unroll
            for (int t = 0; t < MT; ++t) {
              const float4 x = held ? at[(1 + t) * 32] : make_float4(0.f, 0.f, 0.f, 0.f);
              float(&u)[4] = o[n][t];
              u[0] = fmaf(x.x, f0, u[0] * w0);
              u[1] = fmaf(x.y, f1, u[1] * w1);
              u[2] = fmaf(x.z, f0, u[2] * w0);
              u[3] = fmaf(x.w, f1, u[3] * w1);
              if (more_spans) at[(1 + t) * 32] = make_float4(u[0], u[1], u[2], u[3]);
            }
          }
        }
        if (!more_spans) break;
      }
      if (!ok) break;

      // ---- the piece is done ---------------------------------------------------
      const It it = sh.it[warp];
      const bool starts = it.u == 0, ends = it.u + it.left(sh.end[warp]) == it.units;
      const int rows = block_rows(p, it.q.nq, it.rb, RB);
      more = !it.same(sh.end[warp]);
      if (more) {
        next_item(p, &sh.it[warp], &sh.it[warp]);
        more = sh.it[warp].r < p.a.n_req && sh.it[warp].left(sh.end[warp]) > 0;
      }
      const bool whole_item = starts && ends;
      float* const to = more ? static_cast<float*>(p.a.ws) + ((size_t)blockIdx.x * WARPS + warp) * S::kFloats
                             : slot_smem;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int rho = n * 8 + 2 * t4 + e;
          if (rho < rows) {
            const float f = whole_item ? inverse(l[n][e]) : 1.f;
            const int64_t row = whole_item ? out_row(p, it.q.begin, it.h, it.rb, RB, rho) : rho;
            const int ch0 = 8 * VW * g;
#pragma unroll
            for (int t = 0; t < MT; t += 2) {
              const float4 v = make_float4(o[n][t][e] * f, o[n][t][e + 2] * f, o[n][t + 1][e] * f,
                                           o[n][t + 1][e + 2] * f);
              if (whole_item) store4(p, row, D, ch0 + 2 * t, v);
              else *reinterpret_cast<float4*>(to + rho * D + ch0 + 2 * t) = v;
            }
            if (g == 0) {
              if (!whole_item) S::ml(to)[rho] = make_float2(m[n][e], l[n][e]);
              else store_lse(p, row, m[n][e], l[n][e]);
            }
          }
        }
      if (lane == 0 && !whole_item) {
        if (!starts) {
          meta[warp].head = ends ? 1 : 2;
          meta[warp].head_global = more;
          meta[warp].head_rows = rows;
        } else {
          meta[warp].tail = 1;
        }
        // of the last open piece: the tail if there is one
        meta[warp].rows = rows;
        meta[warp].begin = it.q.begin;
        meta[warp].left = it.units - it.u - it.left(sh.end[warp]);
        meta[warp].h = it.h;
        meta[warp].rb = it.rb;
      }
    }
    if (!ok && lane == 0) {
      // never leave with a copy still writing into this CTA's shared memory
      int never = 0;
#pragma unroll 1
      for (int s = 0; s < p.stages; ++s)
        mbar_wait(smem_u32(&sh.bars[warp * 8 + s]), (parity >> s) & 1u, &never, nullptr, p.drain_ns());
    }
  }
  __syncthreads();
  finish<D>(p, sh, smem, stage_bytes);
}

// ---------------------------------------------------------------------------
// variants
// ---------------------------------------------------------------------------
// NT 8-row blocks at a time, NS bf16 parts of q and P, CTAs of WARPS warps, MINB of them
// on an SM: what the accumulators leave of the 64 K registers.
template <int D, int G, int NT, int NS, int WARPS, int MINB>
struct Variant {
  static constexpr int kCtas = kMaxSms * MINB;
  static constexpr int kStatic = 6144;  // room for the static shared memory
  static_assert(sizeof(Shared<Item<8 * NT, kUnit, kItemCost>, WARPS>) <= kStatic, "shared memory");
  using W = Work<D, 8 * NT, WARPS>;
  static size_t workspace() { return W::flags(kCtas) * sizeof(float) + kCtas * sizeof(uint64_t); }
  static cudaError_t launch(Params p, int sms, cudaStream_t st) {
    auto kern = attn_kernel<D, G, NT, NS, WARPS, MINB>;
    const int stage = WARPS * 2 * p.c.tile_bytes();
    const int room = 227 * 1024 / MINB - kStatic;
    p.stages = room / stage < 8 ? room / stage : 8;
    // the ring of a warp also takes the sums of its last piece
    if (p.stages < 1 || (size_t)p.stages * stage < W::kSlot * WARPS * sizeof(float))
      return cudaErrorInvalidConfiguration;
    static std::atomic<uint64_t> set[2];  // devices whose limit is raised
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev >= 128 || !(set[dev >> 6].load() & bit)) {
      if ((e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, room)) != cudaSuccess)
        return e;
      if (dev < 128) set[dev >> 6].fetch_or(bit);
    }
    const int grid = sms * MINB < kCtas ? sms * MINB : kCtas;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = WARPS * 32;
    cfg.dynamicSmemBytes = (size_t)p.stages * stage;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeCooperative;  // CTAs wait for one another
    at.val.cooperative = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, p);
  }
};
// (12 warps where their registers are full, 16 else.  At D 128 Exact8 and Rows16 fill the 168
// registers of 12 warps and spill up to 20 and 120 bytes a thread; with 16 warps Exact8 spilled
// more, 33 us for 29.  At D 64 nothing spills: 16 warps take 92 us for 96, of Rows16 70 for 74.)
template <int D, int G>
using Rows8 = Variant<D, G, 1, 1, 16, 1>;
template <int D, int G>
using Rows16 = Variant<D, G, 2, 1, D == 64 ? 16 : 12, 1>;
template <int D, int G>
using Exact8 = Variant<D, G, 1, 3, D == 64 ? 16 : 12, 1>;

}  // namespace cattn

// The workspace does not depend on the group.
size_t cache_attn_workspace(const Cache& c) {
  using namespace cattn;
  const size_t n = !c.bf16       ? (c.D == 128 ? Exact8<128, 32>::workspace() : Exact8<64, 32>::workspace())
                   : c.D == 128 ? std::max({Rows8<128, 32>::workspace(), Rows16<128, 32>::workspace(),
                                            cache_prompt_workspace(128)})
                                : std::max({Rows8<64, 32>::workspace(), Rows16<64, 32>::workspace(),
                                            cache_prompt_workspace(64)});
  return (n + 255) / 256 * 256;
}

namespace cattn {
// A number that no flag in a workspace holds: unlike any before it, and unlike what memory
// holds by chance (a count through the finaliser of SplitMix64: Steele, Lea, Flood 2014).
// A captured launch keeps its number; its flags are taken away in each run.
static uint64_t next_nonce() {
  static std::atomic<uint64_t> count{(uint64_t)std::chrono::steady_clock::now().time_since_epoch().count()};
  uint64_t x = count.fetch_add(1) * 0x9E3779B97F4A7C15ull;
  x = (x ^ (x >> 30)) * 0xBF58476D1CE4E5B9ull;
  x = (x ^ (x >> 27)) * 0x94D049BB133111EBull;
  return (x ^ (x >> 31)) | 1ull;
}
}  // namespace cattn

template <int D, int G>
static cudaError_t launch_attn(const cattn::Params& p, int sms, cudaStream_t st) {
  using namespace cattn;
  if (!p.c.bf16) return Exact8<D, G>::launch(p, sms, st);
  // 8 rows at a time while that is all a request has, else 16; past three blocks of 16, each
  // of which unpacks the codes again, the tensor memory's kernel.  32 requests of 500 to 12000
  // cached tokens, us (8 rows, 16 rows, tensor memory):
  //   4 K/V heads of 8 query heads: 8 rows 35, 43, 82; then (16 rows, tensor memory) 16 rows 47,
  //     94; 32: 73, 108; 48: 100, 110; 56: 122, 113; 64: 125, 114; 128: 219, 136
  //   8 K/V heads of 4: 8 rows 54, 68, 148; 16 rows 74, 167; 32: 127, 193; 48: 176, 200;
  //     56: 221, 201; 64: 223, 203; 128: 413, 240
  // and 64 requests of 200 to 8000, D 64, 4 K/V heads of 8: 8 rows 33, 36, 80; 16 rows 37, 81;
  // 32: 55, 91; 48: 74, 92; 56: 92, 92; 128: 168, 103.
  // (One kernel a call: the requests with few rows of a call with a long one are slower than in
  // a call of their own, 127 decoding ones beside a chunk of 2048 tokens 1534 us, apart 1034.)
  const int64_t rows = (int64_t)p.a.max_q * p.n_rep;
  if (rows <= 8) return Rows8<D, G>::launch(p, sms, st);
  if (rows <= 48) return Rows16<D, G>::launch(p, sms, st);
  return launch_cache_prompt(p, sms, st);
}

cudaError_t launch_cache_attn(const Cache& c, const CacheAttnArgs& a, cudaStream_t st) {
  cattn::Params p;
  p.c = c;
  p.a = a;
  p.n_rep = c.Hq / c.Hkv;
  p.stages = 0;
  p.per_sum = (a.n_req + cattn::kSums - 1) / cattn::kSums;
  p.page_tiles = c.page / kCacheTile;
  p.unit_in_page = c.page % cattn::kUnit == 0;
  p.page_bytes = c.Hkv * c.block_bytes();
  p.nonce = cattn::next_nonce();
  p.publish = c.debug_fault == 3 ? 0 : p.nonce;
  p.timeout_ns = c.debug_fault ? cattn::kDebugTimeoutNs : cattn::kTimeoutNs;
  p.ones = kOnes;
  p.sl2 = c.scale * 1.44269504088896340736f;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  timing_begin("cache_attn", st);
  if (c.D == 128)
    e = c.G == 128  ? launch_attn<128, 128>(p, sms, st)
        : c.G == 64 ? launch_attn<128, 64>(p, sms, st)
                    : launch_attn<128, 32>(p, sms, st);
  else
    e = c.G == 64 ? launch_attn<64, 64>(p, sms, st) : launch_attn<64, 32>(p, sms, st);
  timing_end(st);
  return e;
}

}  // namespace cpattn
