// Linear attention on the 5th-generation tensor cores (sm_103a): bf16, head dimension 64 or 128.
// The sweep, its runs and its direction are described in layer.cuh; one block takes one run of
// one sweep and head, in chunks of 128 tokens.  Per chunk, with w the powers of the decay:
//
//   S = a b^T            (SS)  P = S * w(i - j), zero where j comes after i, as bf16 into TMEM
//   O1 = P c             (TS)
//   O2 = a M             (SS)  M: what went before, as bf16 in shared memory
//   out_i = mul (O1_i + w(i + 1) O2_i)
//   U = (w(n - 1 - j) b_j)^T c   (SS, both transposed by their descriptors)
//   M = w(n) M + U
//
// M itself stays in float32, in registers (two threads a row, one channel of b).  b is weighted once
// S has read it, as two bf16 numbers, hi in b's place and what is left, lo, in a place of its own,
// and U is the sum of two products: 16 bits, in the runs' sums too.  For a state that is handed out in
// float32, in the sums and in the sequence's last run, it is three, 24 bits.  The smallest part is
// summed first: so the large numbers go through eight steps of the tensor cores' sum (16 terms
// each) and not through all.  As operands P and M are rounded to bf16 once, like the output itself.
// Errors against float64, of the norm: outputs 2.35e-3 whatever the decays, which is sqrt(2) times
// their own rounding of 1.66e-3 (with b in one part in the sums 2.4e-3 to 2.8e-3, the more the longer
// the memory); states 1.0e-7 (8192 tokens; 2.4e-6 in two parts, 5.4e-7 in three with the largest first).  U starts from zero in every chunk: no sum on the tensor cores
// runs longer than 384 terms.
//
// Warp roles (640 threads):
//   warp 0        TMA producer: the tiles a, b, c of a chunk, two stages of a and b and one of c
//                 (which is wanted last; three each at D 64)
//   warp 1        issues S;  warp 2: O1;  warp 3: O2 and U
//   warps 4-11    the output, two threads a row: S -> P, then the epilogue, staged where a lies (S
//                 and O2 have read it) and out by TMA: stored from registers, every instruction
//                 touches 32 lines, and the other warps' loads and stores wait for that (15 % more)
//   warps 12-19   the state, two threads a row: b times its weights, M, its bf16 copy
// Issuers are whole warps with one elected lane, as in tc_fwd.cu.  TMEM: S/P [0, 128),
// O1, O2 and U of D columns each behind it.
//
// The first launch (SUM) only needs U and M: no a; warps 4-11 weigh b, ahead of warps 12-19, and U has
// two places.  At D 128 two parts leave room for three stages of b and two of c (81.8 us for the
// forward pass of 8192 tokens; two of b and three of c 84.3), three parts for two of each.
//
// Measured (GB300, D 128, 8192 tokens of 32 heads: 128 runs of 16 chunks): the sums 35 us, 2.9 TB/s
// on 96 SMs; the sweep 61 us, 6000 cycles a chunk where 128 KB from and to memory would take
// 4700 and the products 3100; 131072 tokens of 8 heads 235 us (152 runs).  It is bound by two chains
// that come to some 6000 cycles each: S -> P -> O1 -> output -> P of the next chunk, and weights ->
// U -> M -> its copy -> weights of the next.  Code that runs once a chunk in each of 20 warps is
// fetched cold, so that a wait for what is there already costs 400.  (lo in a's place and the output
// over M's copy, with two stages of c, linked the chains through O2: 260 us against 235, and the
// backward pass of 8192 tokens 188 against 176, now 166.  Weights a chunk ahead of M, waiting for the
// output's store a chunk later and prefetches into L2 changed it by -3 to 4 %, each for the worse
// in most cases.)  Halving what is loaded, or leaving out seven eighths of the products, changed
// its time by 5 % at most.
// A block takes all of a head's channels: in two halves, for twice the blocks, S and the reads of a
// and b came twice, and shared memory (960 KB a chunk, against 670) was the bound, 135 us.
//
// A barrier that a role may leave behind by a phase comes as a pair, by the chunk's parity.
// Every mbarrier wait is bounded.
#include "layer.cuh"

namespace cpattn {
namespace lintc {

constexpr int kTile = kLinTcChunk;
constexpr int kThreads = 640;
// Registers of the five warpgroups (control, two of the output or the weights, two of the state): at
// most what 640 threads are launched with, 96 each.
constexpr int kRegsControl = 64, kRegsOut = 80, kRegsState = 128, kRegsLaunch = 96;
static_assert(128 * (kRegsControl + 2 * kRegsOut + 2 * kRegsState) <= kThreads * kRegsLaunch, "");

// EXACT: of a SUM, a state is handed out in the end (keys in three parts).
template <int D, bool SUM, bool EXACT>
struct Smem {
  static constexpr int kTileBytes = kTile * D * 2;
  static constexpr int kAS = SUM ? 0 : D == 128 ? 2 : 3;  // stages of a, of b, of c
  static constexpr int kBS = !SUM ? kAS : EXACT ? (D == 128 ? 2 : 4) : D == 128 ? 3 : 5;
  static constexpr int kCS = D == 128 ? (SUM ? 2 : 1) : kBS;
  static constexpr int kXS = !SUM ? 1 : EXACT ? (D == 128 ? 3 : 5) : D == 128 ? 2 : 3;  // smaller parts of the weighted b
  static constexpr int kA = 0;
  static constexpr int kB = kA + kAS * kTileBytes;
  static constexpr int kC = kB + kBS * kTileBytes;
  static constexpr int kX = kC + kCS * kTileBytes;
  // (at D 64 U reads on behind a part's tile, as far as another one)
  static constexpr int kM = kX + (kXS + (SUM && D == 64)) * kTileBytes;
  // the output's staging, 4 KB a warp: at D 128 where a lies, at D 64 that is too small
  static constexpr int kO = kM + (SUM ? 0 : D * D * 2);
  static constexpr int kPow = kO + (SUM || D == 128 ? 0 : 8 * 4096);
  // powers r^e at kPow + 4 (128 + e), zeros for e < 0
  static constexpr int kBar = kPow + 4 * 264;
  static constexpr int kNumBars = 2 * (kAS + kBS + kCS) + 15 + 3 + kXS;
  static constexpr int kMisc = kBar + 8 * kNumBars;
  static constexpr int kBytes = kMisc + 16;
};

struct Maps {
  CUtensorMap a, b, c, o;
};
struct Params {
  Linear p;
  Maps maps[kMaxSweeps];
};

// Every role runs through its code once a chunk, on every sub-partition, and together they overran
// the instruction cache (40 % of its requests missed, 10 % now): loops stay rolled where registers
// allow (but those that issue products: one at a time, eight chunks at D 64 took 26 us and not 22),
// and a wait is a few instructions, bounded by a number of tries of up to 20 us each (the hardware
// suspends the thread meanwhile) instead of by a clock.
constexpr uint32_t kTryNs = 20000;
constexpr uint32_t kTries = 500000;       // 10 s at most, 50 ms if a try takes 100 ns only
constexpr uint32_t kDebugTries = 2500;    // 50 ms at most, under the fault hook
constexpr uint32_t kDrainTries = 10000;

__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(kTryNs)
      : "memory");
  return ok != 0;
}
// Gives up (false) when *abort is set or the tries run out; then it sets *abort itself, so that
// every other role of the block stops too, and latches the device status word.
__device__ __forceinline__ bool thread_wait(uint32_t bar, uint32_t par, volatile int* abort, int* status, uint32_t tries) {
#pragma unroll 1
  while (!try_wait(bar, par)) {
    if (*abort) return false;
    if (--tries == 0) {
      *abort = 1;
      latch_status(status, kStatusTimeout);
      return false;
    }
  }
  return true;
}
// The same with every lane of the warp; all lanes agree on the result.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t par, volatile int* abort, int* status, uint32_t tries) {
  return __all_sync(0xffffffffu, thread_wait(bar, par, abort, status, tries));
}
// Ignores the abort flag (used to drain in-flight copies and products before exit).
__device__ __forceinline__ void drain_wait(uint32_t bar, uint32_t par) {
#pragma unroll 1
  for (uint32_t i = 0; i < kDrainTries && !try_wait(bar, par); ++i) {
  }
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// PIECES: the chunks of a zigzag order off their grid (layer.cuh).  A kernel of its own, since its
// divisions cost the other orders 8 % (T 8192, 32 heads of 128: 62 -> 67 us).
template <int D, bool SUM, bool EXACT, bool PIECES>
__global__ void __launch_bounds__(kThreads, 1)
    sweep_kernel(const __grid_constant__ Params prm) {
  using L = Smem<D, SUM, EXACT>;
  constexpr int AS = L::kAS, BS = L::kBS, CS = L::kCS, XS = L::kXS;
  constexpr uint32_t kTmemCols = SUM ? 2 * D : 512;
  const Linear& p = prm.p;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the layout has no alignment slack
    if (threadIdx.x == 0) latch_status(p.status, kStatusLaunch);
    return;
  }
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bars = sbase + L::kBar;
  auto a_full = [&](int s) { return bars + 8 * s; };
  auto a_empty = [&](int s) { return bars + 8 * (AS + s); };
  auto b_full = [&](int s) { return bars + 8 * (2 * AS + s); };
  auto b_empty = [&](int s) { return bars + 8 * (2 * AS + BS + s); };
  auto c_full = [&](int s) { return bars + 8 * (2 * AS + 2 * BS + s); };
  auto c_empty = [&](int s) { return bars + 8 * (2 * AS + 2 * BS + CS + s); };
  const uint32_t one = bars + 8 * 2 * (AS + BS + CS);
  auto s_full = [&](int i) { return one + 8 * (i & 1); };        // pairs
  auto x_full = [&](int k) { return one + 8 * (2 + (k & 1)); };  // parts written, the k-th time
  auto u_full = [&](int i) { return one + 8 * (4 + (i & 1)); };
  const uint32_t p_full = one + 48, o_full = one + 56, o_free = one + 64, m_full = one + 72,
                 m_free = one + 80, h_done = one + 88, o2_full = one + 96, fin = one + 120;
  auto u_free = [&](int i) { return one + 104 + 8 * (i & 1); };  // SUM, in the place of fixed
  auto fixed = [&](int k) { return one + 104 + 8 * (k & 1); };  // partial chunks, a pair
  auto x_empty = [&](int s) { return one + 144 + 8 * s; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + L::kMisc + 4);
  float* pw = reinterpret_cast<float*>(smem + L::kPow) + 128;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t tmo = p.debug_fault ? kDebugTries : kTries;

  // ---- this block's run
  const int runs = SUM ? p.segs - 1 : p.segs;  // the last run's own sum is nobody's start
  const int bh = blockIdx.x / runs, run = blockIdx.x - bh * runs;
  const LinSweep& w = SUM ? p.sum[blockIdx.y] : p.sweep[blockIdx.y];
  const Maps& maps = prm.maps[blockIdx.y];
  const int n_tok = lin_tokens(p, bh);
  const float ld = lin_decay(p, bh);
  const int back = w.back, late = back;
  // bf16 numbers of a weighted b
  const int parts = (SUM ? EXACT && w.exact : w.exact && run == p.segs - 1) ? 3 : 2;
  const int bb = bh / p.Hq, h = bh - bb * p.Hq;
  const int head_a = bb * (p.Hq / w.rep_a) + h / w.rep_a;
  const int head_b = bb * (p.Hq / w.rep_b) + h / w.rep_b;
  const int head_c = bb * (p.Hq / w.rep_c) + h / w.rep_c;
  const int64_t rows_q = (int64_t)p.B * p.Hq * p.T;  // (for a CPATTN_DEBUG build's checks)
  const int m0 = run * p.cps;
  int n_chunks = min(p.cps, p.nch - m0);
  if (!back) n_chunks = min(n_chunks, lin_chunks<kTile, PIECES>(p, n_tok) - m0);  // (else chunks of padding)
  // The i-th chunk of the run: first position and tokens.
  auto chunk_pos = [&](int i) { return lin_first<kTile, PIECES>(p, lin_chunk(p.nch, back, m0 + i)); };
  auto chunk_n = [&](int i) { return lin_size<kTile, PIECES>(p, n_tok, lin_chunk(p.nch, back, m0 + i)); };

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::kNumBars; ++i) mbar_init(bars + 8 * i, 1);
    // a_empty: the eight warps that stage the output; c_empty: O1 and U; the rest by threads
    for (int i = 0; i < AS; ++i) mbar_init(a_empty(i), 8);
    for (int i = 0; i < CS; ++i) mbar_init(c_empty(i), SUM ? 1 : 2);
    for (int i = 0; i < 2; ++i) {
      mbar_init(x_full(i), 256);
      mbar_init(fixed(i), 256);
    }
    mbar_init(p_full, 256);
    mbar_init(o_free, 256);
    mbar_init(m_full, 256);
    *abort = 0;
    fence_barrier_init();
  }
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  for (int i = threadIdx.x; i < 264; i += blockDim.x) pw[i - 128] = i < 128 ? 0.f : lin_pow(ld, i - 128);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();  // (the next launch's blocks start as this one's end)
  const uint32_t tS = tmem, tO1 = tmem + 128, tO2 = tmem + 128 + D;
  auto tU = [&](int i) { return SUM ? tmem + (i & 1) * D : tmem + 128 + 2 * D; };

  // ---- b times its weights, in its parts: two threads a token, half the channels each
  constexpr int HC = D / 2, DD = D * D;
  const int quad = warp & 3, row = quad * 32 + lane;  // a token of a chunk (for M: a channel of b)
  const int col0 = (warp >> 2 & 1) * HC;              // channels of b (columns of M)
  StageRing<BS> wb;
  StageRing<CS> wc;
  int wk = 0, wx = 0, wf = 0;
  uint32_t xpar = 0;
  auto weigh = [&](int i) -> bool {
    const int n = chunk_n(i);
    // (x_full of the last but one has been seen)
    if (SUM && i > 1 && !warp_wait(u_full(i), (i >> 1 & 1) ^ 1, abort, p.status, tmo)) return false;
    if (!warp_wait(b_full(wb.stage), wb.par, abort, p.status, tmo)) return false;
    uint8_t* const bt = smem + L::kB + wb.stage * L::kTileBytes;
    // this thread's half of its token's row: HC / 8 chunks of eight channels
    uint4* const line = reinterpret_cast<uint4*>(bt + (col0 >> 6) * (kTile * 128) + row * 128);
    const int chunk0 = (col0 & 63) >> 3;
    // Where they lie.  At D 64 the row's other thread has the line's other half, and nothing orders
    // the two in the sums: each clears, reads and writes its own pieces alone.
    auto piece = [&](int j) { return (chunk0 + j) ^ (row & 7); };
    if (n < kTile) {
      // rows behind the last token hold anything: zeros, in b and in c
      if (!warp_wait(c_full(wc.stage), wc.par, abort, p.status, tmo)) return false;
      if (row >= n) {
        uint4* const cline = line + (L::kC - L::kB + (wc.stage - wb.stage) * L::kTileBytes) / 16;
#pragma unroll
        for (int j = 0; j < HC / 8; ++j) line[piece(j)] = cline[piece(j)] = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();
      if (!SUM) mbar_arrive(fixed(wf++));
    }
    // S has read b
    if (!SUM && !warp_wait(s_full(i), (i >> 1) & 1, abort, p.status, tmo)) return false;
    const float uw = row < n ? pw[(back ? row : n - 1 - row) + late] : 0.f;
    const float2 uw2 = make_float2(uw, uw);
    // the parts of eight channels
    auto split = [&](uint4 x, uint4& hi, uint4& mid, uint4& lo, bool three) {
      const uint32_t in[4] = {x.x, x.y, x.z, x.w};
      uint32_t h[4], m[4], l[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float2 v = mul2(make_float2(bf16_lo(in[q]), bf16_hi(in[q])), uw2);
        h[q] = pack_bf16(v.x, v.y);
        v = fma2(make_float2(bf16_lo(h[q]), bf16_hi(h[q])), make_float2(-1.f, -1.f), v);
        m[q] = pack_bf16(v.x, v.y);
        if (three) l[q] = pack_bf16(v.x - bf16_lo(m[q]), v.y - bf16_hi(m[q]));
      }
      hi = make_uint4(h[0], h[1], h[2], h[3]);
      mid = make_uint4(m[0], m[1], m[2], m[3]);
      if (three) lo = make_uint4(l[0], l[1], l[2], l[3]);
    };
    // a place for each of the smaller parts, two numbers ahead of the product; or (!SUM) for the smallest
    // alone, which U of the last chunk has read
    uint4* const xline = line + (L::kX - L::kB - wb.stage * L::kTileBytes) / 16;
    if (SUM) {
      auto place = [&](uint4*& l) -> bool {
        if (!warp_wait(x_empty(wx), xpar ^ 1u, abort, p.status, tmo)) return false;
        l = xline + wx * (L::kTileBytes / 16);
        if (++wx == XS) wx = 0, xpar ^= 1u;
        return true;
      };
      uint4 *l0, *l1;  // the smallest part's, the middle one's (of two parts: l0)
      if (!place(l0)) return false;
      if (EXACT && parts == 3) {
        if (!place(l1)) return false;
#pragma unroll 2
        for (int j = 0; j < HC / 8; ++j) {
          const int at = piece(j);
          uint4 hi;
          split(line[at], hi, l1[at], l0[at], true);
          line[at] = hi;
        }
      } else {
#pragma unroll 2
        for (int j = 0; j < HC / 8; ++j) {
          const int at = piece(j);
          uint4 hi, lo;
          split(line[at], hi, l0[at], lo, false);
          line[at] = hi;
        }
      }
    } else if (parts == 2) {
#pragma unroll 2
      for (int j = 0; j < HC / 8; ++j) {
        const int at = piece(j);
        uint4 hi, mid, lo;
        split(line[at], hi, mid, lo, false);
        line[at] = hi;
        xline[at] = mid;
      }
    } else {
      uint4 hi[HC / 8];
#pragma unroll
      for (int j = 0; j < HC / 8; ++j) {
        const int at = piece(j);
        uint4 mid, lo;
        split(line[at], hi[j], mid, lo, true);
        line[at] = mid;
        xline[at] = lo;
      }
      fence_proxy_async_smem();
      mbar_arrive(x_full(wk++));
      if (!warp_wait(h_done, i & 1, abort, p.status, tmo)) return false;
#pragma unroll
      for (int j = 0; j < HC / 8; ++j) line[piece(j)] = hi[j];
    }
    fence_proxy_async_smem();
    mbar_arrive(x_full(wk++));
    wb.advance();
    wc.advance();
    return true;
  };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == 0) {
      // ---------------------------------------------------------- producer
      if (lane == 0) {
        StageRing<AS == 0 ? 1 : AS> ra;
        StageRing<BS> rb;
        StageRing<CS> rc;
        bool ok = true;
        for (int i = 0; i < n_chunks && ok; ++i) {
          const int slot = p.m.slot(chunk_pos(i));
          auto load = [&](auto& ring, uint32_t full, uint32_t empty, int base, const CUtensorMap* tm, int head,
                          int heads) {
            if (!ok || !(ok = thread_wait(empty, ring.par ^ 1, abort, p.status, tmo))) return;
            mbar_expect_tx(full, L::kTileBytes);
            const int row = head * p.T + slot;
            // (a partial chunk reads on into the next head, or zeros behind the tensor)
            if (in_bounds(row, 1, (int64_t)heads * p.T, p.status) && !(p.debug_fault && i == 0)) {
              for (int kb = 0; kb < D / 64; ++kb)
                tma_load_2d(sbase + base + ring.stage * L::kTileBytes + kb * (kTile * 128), tm, kb * 64, row, full);
              ring.mark_issued();
            }
            ring.advance();
          };
          load(rb, b_full(rb.stage), b_empty(rb.stage), L::kB, &maps.b, head_b, p.B * (p.Hq / w.rep_b));
          if (!SUM) load(ra, a_full(ra.stage), a_empty(ra.stage), L::kA, &maps.a, head_a, p.B * (p.Hq / w.rep_a));
          load(rc, c_full(rc.stage), c_empty(rc.stage), L::kC, &maps.c, head_c, p.B * (p.Hq / w.rep_c));
        }
        // never leave with a copy still writing into this block's shared memory
        for (int s = 0; s < AS; ++s)
          if (ra.was_issued(s)) drain_wait(a_full(s), ra.issued_parity(s));
        for (int s = 0; s < BS; ++s)
          if (rb.was_issued(s)) drain_wait(b_full(s), rb.issued_parity(s));
        for (int s = 0; s < CS; ++s)
          if (rc.was_issued(s)) drain_wait(c_full(s), rc.issued_parity(s));
      }
    } else if (warp == 1) {
      if constexpr (!SUM) {
        // -------------------------------------------------------- S = a b^T
        const bool leader = elect_one();
        constexpr uint32_t kId = idesc_bf16(128, 128, false, false);
        const uint64_t ad0 = sdesc_sw128(sbase + L::kA, 16, 1024), bd0 = sdesc_sw128(sbase + L::kB, 16, 1024);
        StageRing<AS> ra;
        int nf = 0;  // partial chunks
        for (int i = 0; i < n_chunks; ++i) {
          if (!warp_wait(a_full(ra.stage), ra.par, abort, p.status, tmo) ||
              !warp_wait(b_full(ra.stage), ra.par, abort, p.status, tmo))
            break;
          // (everyone has seen s_full of the last but one; what comes last is waited for last)
          if (i > 1 && !warp_wait(u_full(i), (i >> 1 & 1) ^ 1, abort, p.status, tmo)) break;
          // a partial chunk's rows of b and c behind its end are zeroed first
          if (chunk_n(i) < kTile) {
            if (!warp_wait(fixed(nf), nf >> 1 & 1, abort, p.status, tmo)) break;
            ++nf;
          }
          // S's place is free once O1 of the last chunk has read P there
          if (i > 0 && !warp_wait(o_full, (i - 1) & 1, abort, p.status, tmo)) break;
          tc_fence_after();
          const uint32_t st = ra.stage * (L::kTileBytes >> 4);
          if (leader) {
#pragma unroll 4
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = st + (kk >> 2) * 1024 + (kk & 3) * 2;  // 16 KiB blocks, 32 B steps
              mma_ss(tS, ad0 + off, bd0 + off, kId, kk > 0);
            }
            mma_commit(s_full(i));
          }
          __syncwarp();
          ra.advance();
        }
        if (leader) mma_commit(fin);
        __syncwarp();
        drain_wait(fin, 0);
      }
    } else if (warp == 2) {
      if constexpr (!SUM) {
        // -------------------------------------------------------- O1 = P c
        const bool leader = elect_one();
        constexpr uint32_t kId = idesc_bf16(128, D, false, true);
        const uint64_t cd0 = sdesc_sw128(sbase + L::kC, kTile * 128, 1024);
        StageRing<CS> rc;
        int nf = 0;
        for (int i = 0; i < n_chunks; ++i) {
          if (!warp_wait(c_full(rc.stage), rc.par, abort, p.status, tmo)) break;
          if (chunk_n(i) < kTile) {
            if (!warp_wait(fixed(nf), nf >> 1 & 1, abort, p.status, tmo)) break;
            ++nf;
          }
          // the epilogue of the last chunk has read O1
          if (i > 0 && !warp_wait(o_free, (i - 1) & 1, abort, p.status, tmo)) break;
          if (!warp_wait(p_full, i & 1, abort, p.status, tmo)) break;
          tc_fence_after();
          const uint32_t st = rc.stage * (L::kTileBytes >> 4);
          if (leader) {
#pragma unroll 4
            for (int kk = 0; kk < kTile / 16; ++kk)
              mma_ts(tO1, tS + (kk >> 2) * 64 + (kk & 3) * 8, cd0 + st + (uint64_t)(kk * 128), kId, kk > 0);
            mma_commit(o_full);
            mma_commit(c_empty(rc.stage));
          }
          __syncwarp();
          rc.advance();
        }
        if (leader) mma_commit(fin + 8);
        __syncwarp();
        drain_wait(fin + 8, 0);
      }
    } else {
      // --------------- O2 = a M, and U = (weighted b)^T c, part after part
      const bool leader = elect_one();
      constexpr uint32_t kId = idesc_bf16(128, D, true, true), kId2 = idesc_bf16(128, D, false, true);
      // (at D 64 U's lower 64 rows read what lies behind the tile: nobody reads them)
      const uint64_t bd0 = sdesc_sw128(sbase + L::kB, kTile * 128, 1024);
      const uint64_t cd0 = sdesc_sw128(sbase + L::kC, kTile * 128, 1024);
      const uint64_t ad0 = sdesc_sw128(sbase + L::kA, 16, 1024);
      const uint64_t md = sdesc_sw128(sbase + L::kM, D * 128, 1024);
      const uint64_t xd0 = sdesc_sw128(sbase + L::kX, kTile * 128, 1024);
      StageRing<BS> rb;
      StageRing<CS> rc;
      bool ok = true;
      int k = 0, x = 0;
      for (int i = 0; i < n_chunks && ok; ++i) {
        const uint32_t st = rb.stage * (L::kTileBytes >> 4), stc = rc.stage * (L::kTileBytes >> 4);
        if constexpr (!SUM) {
          // the epilogue of the last chunk has read O2
          if (!(ok = warp_wait(a_full(rb.stage), rb.par, abort, p.status, tmo) &&
                     warp_wait(m_full, i & 1, abort, p.status, tmo) &&
                     (i == 0 || warp_wait(o_free, (i - 1) & 1, abort, p.status, tmo))))
            break;
          tc_fence_after();
          if (leader) {
#pragma unroll 4
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ss(tO2, ad0 + st + (kk >> 2) * 1024 + (kk & 3) * 2, md + (uint64_t)(kk * 128), kId2, kk > 0);
            mma_commit(m_free);
            mma_commit(o2_full);
          }
          __syncwarp();
        }
        if (!(ok = warp_wait(c_full(rc.stage), rc.par, abort, p.status, tmo))) break;
        // a part: b's place, or one of its own
        auto product = [&](uint64_t pd, bool first) {
          if (leader)
#pragma unroll 4
            for (int kk = 0; kk < kTile / 16; ++kk)
              mma_ss(tU(i), pd + (uint64_t)(kk * 128), cd0 + stc + (uint64_t)(kk * 128), kId, !first || kk > 0);
        };
        // U's place has been read
        if (SUM && i > 1 && !(ok = warp_wait(u_free(i), (i >> 1 & 1) ^ 1, abort, p.status, tmo))) break;
        if (!(ok = warp_wait(x_full(k), (k >> 1) & 1, abort, p.status, tmo))) break;
        ++k;
        tc_fence_after();
        if (!SUM) {
#pragma unroll 1
          for (int part = 0; part < 2; ++part) product(part ? bd0 + st : xd0, part == 0);
        } else {
#pragma unroll 1
          for (int part = 0; part < parts - 1; ++part) {
            product(xd0 + x * (L::kTileBytes >> 4), part == 0);
            if (leader) mma_commit(x_empty(x));
            __syncwarp();
            if (++x == XS) x = 0;
          }
        }
        if (SUM) product(bd0 + st, false);
        if (!SUM && parts == 3) {
          if (leader) mma_commit(h_done);
          __syncwarp();
          if (!(ok = warp_wait(x_full(k), (k >> 1) & 1, abort, p.status, tmo))) break;
          ++k;
          tc_fence_after();
          product(bd0 + st, false);
        }
        if (leader) {
          mma_commit(u_full(i));
          mma_commit(b_empty(rb.stage));
          mma_commit(c_empty(rc.stage));
        }
        __syncwarp();
        rb.advance();
        rc.advance();
      }
      if (leader) mma_commit(fin + 16);
      __syncwarp();
      drain_wait(fin + 16, 0);
    }
  } else if (warp < 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOut));
    if constexpr (SUM) {
      for (int i = 0; i < n_chunks; ++i)
        if (!weigh(i)) break;
    } else {
      // ------------------------------------------------ P and the epilogue
      const int half = warp >> 2 & 1;
      const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
      int sa = 0;  // stage of a
      for (int i = 0; i < n_chunks; ++i) {
        if (!warp_wait(s_full(i), (i >> 1) & 1, abort, p.status, tmo)) break;
        tc_fence_after();
        // 32 columns at a time, two times a half: weights from the table (zero for columns that come
        // after the row; wholly such columns are not read).  P of half h lies over S's columns
        // [64 h, 64 h + 32), which this thread has read by then.
        const float* wr = back ? pw - row + half * 64 : pw + row - half * 64;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[16];
          const int col = 2 * half + c;
          if (back ? col < quad : col > quad) {
#pragma unroll
            for (int j = 0; j < 16; ++j) pk[j] = 0u;
          } else {
            uint32_t r[32];
            tmem_ld32(tS + lane_off + col * 32, r);
            float f[32];
            if (back) {
#pragma unroll
              for (int j = 0; j < 32; ++j) f[j] = wr[j];
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) f[j] = wr[-j];
            }
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              pk[j] = pack_bf16(__uint_as_float(r[2 * j]) * f[2 * j], __uint_as_float(r[2 * j + 1]) * f[2 * j + 1]);
          }
          tmem_st16(tS + lane_off + half * 64 + c * 16, pk);
          wr += back ? 32 : -32;
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(p_full);

        // (while O1 runs)
        const int n = chunk_n(i);
        const float ow = pw[(back ? n - 1 - min(row, n - 1) : row) + 1 - late] * w.mul;
        const float2 ow2 = make_float2(ow, ow), mul2v = make_float2(w.mul, w.mul);
        const int64_t tile_row0 = (int64_t)bh * p.T + p.m.slot(chunk_pos(i));
        const bool store = row < n && in_bounds(tile_row0 + row, 1, rows_q, p.status);
        const int64_t at = (tile_row0 + row) * D + half * HC;
        if (!warp_wait(o2_full, i & 1, abort, p.status, tmo) || !warp_wait(o_full, i & 1, abort, p.status, tmo)) break;
        tc_fence_after();
        // whole chunks go by way of shared memory: this warp's 32 lines of 64 bf16 or 32 float32
        // columns (at D 64 of 32 bf16: half lines), swizzled as the tensor map has it
        const bool staged = n == kTile;
        const int area = (D == 128 ? L::kA + sa * L::kTileBytes : L::kO) + (quad * 2 + half) * 4096;
        const int lchunks = D == 64 && !w.out_f32 ? 4 : 8, lswz = D == 64 && !w.out_f32 ? lane >> 1 & 3 : lane & 7;
        uint4* const line = reinterpret_cast<uint4*>(smem + area) + lane * lchunks;
        auto leave = [&](int col) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (in_bounds(tile_row0 + quad * 32, 32, rows_q, p.status))
              tma_store_2d(&maps.o, half * HC + col, (int)(tile_row0 + quad * 32), sbase + area);
            bulk_commit_group();
          }
          __syncwarp();
        };
        auto left = [&]() {
          if (lane == 0) bulk_wait_read_all();
          __syncwarp();
        };
#pragma unroll 1
        for (int c = 0; c < HC / 16; ++c) {
          uint32_t o1[16], o2[16];
          tmem_ld16(tO1 + lane_off + half * HC + c * 16, o1);
          tmem_ld16(tO2 + lane_off + half * HC + c * 16, o2);
          tmem_wait_ld();
          if (c == HC / 16 - 1) {  // O1 and O2 have been read
            tc_fence_before();
            mbar_arrive(o_free);
          }
          float2 v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j)
            v[j] = fma2(ow2, make_float2(__uint_as_float(o2[2 * j]), __uint_as_float(o2[2 * j + 1])),
                        mul2(mul2v, make_float2(__uint_as_float(o1[2 * j]), __uint_as_float(o1[2 * j + 1]))));
          if (D == 64 && c == 0 && staged) left();  // the last chunk's
          if (w.out_f32) {
            if (c == 2 && staged) left();  // the first 32 columns
            float4* const dst = reinterpret_cast<float4*>(static_cast<float*>(w.out) + at) + c * 4;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float4 x = make_float4(v[2 * j].x, v[2 * j].y, v[2 * j + 1].x, v[2 * j + 1].y);
              if (staged) reinterpret_cast<float4*>(line)[((c & 1) * 4 + j) ^ lswz] = x;
              else if (store) dst[j] = x;
            }
            if (staged && (c & 1)) leave((c >> 1) * 32);
          } else {
            uint4* const dst = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(w.out) + at) + c * 2;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint4 x = make_uint4(pack_bf16(v[4 * j].x, v[4 * j].y), pack_bf16(v[4 * j + 1].x, v[4 * j + 1].y),
                                         pack_bf16(v[4 * j + 2].x, v[4 * j + 2].y), pack_bf16(v[4 * j + 3].x, v[4 * j + 3].y));
              if (staged) line[(c * 2 + j) ^ lswz] = x;
              else if (store) dst[j] = x;
            }
          }
        }
        if (staged && !w.out_f32) leave(0);
        if (D == 128) left();  // (before a comes there; at D 64 the store has until the next output)
        if (lane == 0) mbar_arrive(a_empty(sa));
        if (++sa == AS) sa = 0;
      }
      if (lane == 0) bulk_wait_all();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsState));
    // -------------------------------------------------------- the state
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const bool mine = D == 128 || row < D;
    float M[HC];
#pragma unroll
    for (int c = 0; c < HC; ++c) M[c] = 0.f;
    if (!SUM && mine) {
      if (w.init) {
        const float* src = w.init + (int64_t)bh * DD;
        if (w.trans) {
#pragma unroll
          for (int c = 0; c < HC; ++c) M[c] = src[(col0 + c) * D + row] * w.init_mul;
        } else {
#pragma unroll
          for (int c = 0; c < HC; c += 4) {
            const float4 x = *reinterpret_cast<const float4*>(src + row * D + col0 + c);
            M[c] = x.x * w.init_mul, M[c + 1] = x.y * w.init_mul;
            M[c + 2] = x.z * w.init_mul, M[c + 3] = x.w * w.init_mul;
          }
        }
      }
      // the runs before this one, folded in order, once the launch that sums them is through
      if (run > 0) griddep_wait();
      for (int s = 0; s < run; ++s) {
        const float f = lin_pow(ld, lin_run_tokens<kTile, PIECES>(p, n_tok, back, s));
        const float* src = w.sums + ((int64_t)bh * p.segs + s) * DD;
        if (!w.trans) {  // a run's sum lies with its columns first (see below)
#pragma unroll
          for (int c = 0; c < HC; ++c) M[c] = fmaf(f, M[c], src[(col0 + c) * D + row]);
        } else {
#pragma unroll
          for (int c = 0; c < HC; c += 4) {
            const float4 x = *reinterpret_cast<const float4*>(src + row * D + col0 + c);
            M[c] = fmaf(f, M[c], x.x), M[c + 1] = fmaf(f, M[c + 1], x.y);
            M[c + 2] = fmaf(f, M[c + 2], x.z), M[c + 3] = fmaf(f, M[c + 3], x.w);
          }
        }
      }
    }
    // M as bf16, the operand of O2: rows of b's channels, 128-byte lines of 64 columns, swizzled
    auto publish = [&]() {
      if (mine) {
        uint4* const line = reinterpret_cast<uint4*>(smem + L::kM + (col0 >> 6) * (D * 128) + row * 128);
#pragma unroll
        for (int c = 0; c < HC; c += 8)
          line[(((col0 & 63) + c) >> 3) ^ (row & 7)] =
              make_uint4(pack_bf16(M[c], M[c + 1]), pack_bf16(M[c + 2], M[c + 3]),
                         pack_bf16(M[c + 4], M[c + 5]), pack_bf16(M[c + 6], M[c + 7]));
      }
      fence_proxy_async_smem();
      mbar_arrive(m_full);
    };
    // M = r^n M + U of chunk i
    auto take = [&](int i) -> bool {
      if (!warp_wait(u_full(i), (i >> 1) & 1, abort, p.status, tmo)) return false;
      tc_fence_after();
      const float f = pw[chunk_n(i)];
      const float2 f2 = make_float2(f, f);
#pragma unroll
      for (int c = 0; c < HC / 32; ++c) {
        uint32_t u[32];
        tmem_ld32(tU(i) + lane_off + col0 + c * 32, u);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float2 x = fma2(f2, make_float2(M[c * 32 + j], M[c * 32 + j + 1]),
                                make_float2(__uint_as_float(u[j]), __uint_as_float(u[j + 1])));
          M[c * 32 + j] = x.x, M[c * 32 + j + 1] = x.y;
        }
      }
      tc_fence_before();
      if (SUM) mbar_arrive(u_free(i));
      return true;
    };
    if (!SUM && n_chunks > 0) publish();
    bool ok = true;
    for (int i = 0; i < n_chunks && ok; ++i) {
      if constexpr (!SUM)
        if (!(ok = weigh(i))) break;
      if (!(ok = take(i))) break;
      if (!SUM && i + 1 < n_chunks) {
        // O2 of this chunk has read the old copy
        if (!(ok = warp_wait(m_free, i & 1, abort, p.status, tmo))) break;
        publish();
      }
    }
    if (ok && mine) {
      if constexpr (SUM) {
        // columns first: the threads of a warp write, and in most sweeps read, consecutive numbers
        float* dst = w.sums + ((int64_t)bh * p.segs + run) * DD;
#pragma unroll
        for (int c = 0; c < HC; ++c) dst[(col0 + c) * D + row] = M[c];
      } else if (run == p.segs - 1 && w.fin) {
        float* dst = w.fin + (int64_t)bh * DD;
#pragma unroll
        for (int c = 0; c < HC; c += 4)
          *reinterpret_cast<float4*>(dst + row * D + col0 + c) = make_float4(
              M[c] * w.fin_mul, M[c + 1] * w.fin_mul, M[c + 2] * w.fin_mul, M[c + 3] * w.fin_mul);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

static bool make_map(CUtensorMap* m, const void* t, int64_t heads, int T, int D) {
  return encode_tmap_2d_bf16(m, t, D, (uint64_t)heads * T, 64, kTile) == CUDA_SUCCESS;
}

template <int D, bool SUM, bool EXACT, bool PIECES>
static cudaError_t run(const Linear& p, int n, const LinSweep* sweeps, bool dependent, cudaStream_t st) {
  Params prm;
  prm.p = p;
  for (int i = 0; i < n; ++i) {
    const LinSweep& w = sweeps[i];
    Maps& m = prm.maps[i];
    const int64_t hq = (int64_t)p.B * p.Hq;
    if (!make_map(&m.b, w.b, hq / w.rep_b, p.T, D) || !make_map(&m.c, w.c, hq / w.rep_c, p.T, D))
      return cudaErrorInvalidValue;
    m.a = m.o = m.b;
    if (!SUM && !make_map(&m.a, w.a, hq / w.rep_a, p.T, D)) return cudaErrorInvalidValue;
  }
  if (!SUM)  // the output's boxes: one warp's 32 rows, a line of 128 bytes each (bf16 at D 64: 64)
    for (int i = 0; i < n; ++i) {
      const LinSweep& w = sweeps[i];
      const uint64_t rows = (uint64_t)p.B * p.Hq * p.T;
      if ((w.out_f32 ? encode_tmap_2d_f32(&prm.maps[i].o, w.out, D, rows, 32, 32)
                     : encode_tmap_2d_bf16(&prm.maps[i].o, w.out, D, rows, D / 2, 32)) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    }
  constexpr int kSmem = Smem<D, SUM, EXACT>::kBytes;
  auto kern = sweep_kernel<D, SUM, EXACT, PIECES>;
  static ReadyDevices ready;
  const cudaError_t e = ready.once([&] {
    cudaFuncAttributes at;  // a split that does not fit what the launch allocates would wait forever
    const cudaError_t r = cudaFuncGetAttributes(&at, kern);
    if (r != cudaSuccess) return r;
    if (at.numRegs < kRegsLaunch) return cudaErrorInvalidConfiguration;
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  if (e != cudaSuccess) return e;
  const unsigned blocks = (unsigned)(p.B * p.Hq * (SUM ? p.segs - 1 : p.segs));
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, n);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = dependent ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, prm);
}

}  // namespace lintc

bool linear_tc_supported(const Ring& R) {
  if (!R.bf16 || (R.D != 64 && R.D != 128)) return false;
  // A chunk's positions are consecutive slots, so a zigzag half of h tokens takes h / 128 chunks,
  // rounded up, and a chunk costs the same whatever it holds; float32 arithmetic packs its chunks.
  // Forward and backward pass here against there, us, 32 ranks with halves of 12, 16 and 64 tokens:
  // 32 heads of 128 105 and 231 against 123 and 274, 161 and 437, 774 and 1784; of 64 75 and 172
  // against 59 and 131, 77 and 209, 291 and 778; 4 heads of 128 56 and 63 against 58 and 66, 63 and
  // 96, 120 and 252; of 64 37 and 37 against 26 and 29, 28 and 45, 51 and 117.  From 16 on all but the
  // last's forward pass are faster here.
  if (R.zz && R.T / R.cp / 2 < 16) return false;
  return (double)R.B * R.Hq * R.T < 2147483647.0 - kLinTcChunk;
}

template <bool SUM, bool EXACT>
static cudaError_t run(const Linear& p, int n, const LinSweep* sweeps, bool dependent, cudaStream_t st) {
  if (p.seg < p.T)
    return p.D == 128 ? lintc::run<128, SUM, EXACT, true>(p, n, sweeps, dependent, st)
                      : lintc::run<64, SUM, EXACT, true>(p, n, sweeps, dependent, st);
  return p.D == 128 ? lintc::run<128, SUM, EXACT, false>(p, n, sweeps, dependent, st)
                    : lintc::run<64, SUM, EXACT, false>(p, n, sweeps, dependent, st);
}

cudaError_t launch_linear_tc(const Linear& p, cudaStream_t st, bool backward) {
  cudaError_t e;
  if (p.segs > 1) {
    timing_begin(backward ? "linear_bwd_sums" : "linear_fwd_sums", st);
    e = p.sum[0].exact || p.sum[1].exact ? run<true, true>(p, p.n_sums, p.sum, false, st)
                                         : run<true, false>(p, p.n_sums, p.sum, false, st);
    timing_end(st);
    if (e != cudaSuccess) return e;
  }
  timing_begin(backward ? "linear_bwd" : "linear_fwd", st);
  e = run<false, false>(p, p.n_sweeps, p.sweep, p.segs > 1, st);
  timing_end(st);
  return e;
}

}  // namespace cpattn
