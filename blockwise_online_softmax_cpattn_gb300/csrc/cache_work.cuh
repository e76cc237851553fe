// How the 4-bit cache's attention kernels divide their work and join its pieces (device
// code, internal to libcpattn).
//
// An item is RB query rows (new tokens x the heads of a K/V group) of one request and K/V
// head; it is cut into units of UNIT cached tokens.  The items of all requests stand in
// one line, by row block, K/V head and request, each with a cost: its units and COST for
// its start and end (the request's numbers and its query rows come from memory, its
// result goes there).  A worker takes an equal run of that line, so neither ragged
// lengths nor few requests leave SMs idle, and nothing about lengths has to be known on
// the host.  A run ends anywhere: what its worker knows of an item that it did not see
// whole is a piece (O, m, l), and pieces are joined in their order by the (O, LSE) merge.
#pragma once

#include <math.h>

#include "cache.cuh"

namespace cpattn {
namespace cattn {

constexpr int kSums = 256;           // entries of the prefix sums over requests
constexpr int kMaxSms = 160;         // of a GB300, and a few: the workspace's size
constexpr float kLn2 = 0.69314718055994530942f;
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr uint64_t kDebugTimeoutNs = 50000000ull;  // under the fault hook

struct Params {
  Cache c;
  CacheAttnArgs a;
  int n_rep, stages;                 // stages: of a ring of copies
  int per_sum;                       // requests per entry of the prefix sums
  int page_tiles, unit_in_page;      // tiles of a page; units do not straddle pages
  int64_t page_bytes;                // of all K/V heads
  float sl2;                         // scale * log2(e)
  uint32_t ones;                     // kOnes
  uint64_t nonce;                    // of this launch's flags
  uint64_t publish;                  // what a piece's flag is set to: nonce, but for the fault hook
  uint64_t timeout_ns;               // of a wait
  // ... for copies and MMAs in flight, before a CTA that gave up leaves
  __device__ __forceinline__ uint64_t drain_ns() const { return timeout_ns / 10; }
};

// ---------------------------------------------------------------------------
// items
// ---------------------------------------------------------------------------
struct Req {
  int begin, nq, len;
};
__device__ __forceinline__ Req request(const Params& p, int r) {
  Req q;
  const int b = min(max(p.a.q_start[r], 0), p.a.n_tokens);
  const int e = min(max(p.a.q_start[r + 1], b), p.a.n_tokens);
  q.begin = b;
  q.nq = e - b;
  q.len = min(max(p.a.kv_len[r], 0), p.a.max_pages * p.c.page);
  return q;
}
// Rows of q are fewer than 2^31 (checked on the host), and so are a request's.
// cached tokens that row x of the request sees
__device__ __forceinline__ int seen_by(const Params& p, const Req& q, int x) {
  if (!p.c.causal) return q.len;
  return min(max(q.len - q.nq + (int)((unsigned)x / (unsigned)p.n_rep) + 1, 0), q.len);
}
// ... that row block rb (RB rows) sees, and its units
__device__ __forceinline__ int block_seen(const Params& p, const Req& q, int rb, int RB) {
  // the last block's last row is the last token's, which sees all
  if (!p.c.causal || (int64_t)(rb + 1) * RB >= (int64_t)q.nq * p.n_rep) return q.len;
  return seen_by(p, q, (rb + 1) * RB - 1);
}
__device__ __forceinline__ int units_of(int seen, int unit) { return max(1, (seen + unit - 1) / unit); }
__device__ __forceinline__ int blocks_of(const Params& p, const Req& q, int RB) {
  return (int)(((unsigned)(q.nq * p.n_rep) + RB - 1) / RB);
}
// Most of these kernels' instructions run once a launch, and an instruction that has to be
// fetched takes as long as many that are there: what runs once is kept small, its loops
// rolled, 64-bit divisions and steps from item to item out of line.
static __device__ __noinline__ int64_t divide(int64_t x, int64_t y) { return x / y; }

// i / n of x, rounded down (in 32 bits where they do; i <= n < 2^8)
__device__ __forceinline__ int part_of(int x, int i, int n) {
  const unsigned q = (unsigned)x / (unsigned)n, r = (unsigned)x - q * n;
  return (int)(q * i + r * i / (unsigned)n);
}
__device__ __forceinline__ int64_t part_of(int64_t x, int i, int n) {
  return x <= 0x7fffffff ? part_of((int)x, i, n) : divide(x * i, n);
}

// Request, K/V head and row block of an item, and a unit in it.  Items follow each other by
// row block, K/V head, request.
struct Place {
  int r, h, rb, u;
};
template <int RB, int UNIT, int COST>
struct Item : Place {
  static constexpr int kRows = RB;
  Req q;
  int seen, units;
  __device__ __forceinline__ void settle(const Params& p) {
    seen = block_seen(p, q, rb, RB);
    units = units_of(seen, UNIT);
  }
  // cost of one K/V head of a request
  static __device__ __forceinline__ int64_t head_cost(const Params& p, const Req& q) {
    const int nb = blocks_of(p, q, RB);
    int64_t n = 0;
#pragma unroll 1
    for (int b = 0; b < nb; ++b) n += units_of(block_seen(p, q, b, RB), UNIT) + COST;
    return n;
  }
  __device__ __forceinline__ bool same(const Place& o) const { return r == o.r && h == o.h && rb == o.rb; }
  // units of this item before `end`, from u on
  __device__ __forceinline__ int left(const Place& end) const { return (same(end) ? end.u : units) - u; }
  // The place at `x` in the numbering of cost that starts with request r0: an item's first
  // COST numbers are its first unit's.  (The bounds of the searches matter only if lengths
  // change under the kernel.)
  __device__ __forceinline__ void locate(const Params& p, int r0, int64_t x) {
    h = rb = u = 0;
#pragma unroll 1
    for (r = r0; r < p.a.n_req; ++r) {
      q = request(p, r);
      if (q.nq == 0) continue;
      const int64_t all = head_cost(p, q) * p.c.Hkv;
      if (x < all) break;
      x -= all;
    }
    if (r < p.a.n_req) within(p, x);  // else behind the last item
  }
  // ... that starts with this request, which is not empty
  __device__ __forceinline__ void within(const Params& p, int64_t x) {
    const int64_t c = head_cost(p, q);
    if (c > 0x7fffffff || x > 0x7fffffff) {
      h = (int)divide(x, c);
      within_head(p, x - h * c);
    } else {
      within(p, (int)x, (int)c);
    }
  }
  // c: the cost of one of its K/V heads
  __device__ __forceinline__ void within(const Params& p, int x, int c) {
    h = (unsigned)x / (unsigned)c;
    within_head(p, x - h * c);
  }
  template <typename Int>
  __device__ __forceinline__ void within_head(const Params& p, Int x) {
    const int nb = blocks_of(p, q, RB);
#pragma unroll 1
    for (rb = 0;; ++rb) {
      settle(p);
      if (rb == nb - 1 || x < units + COST) break;
      x -= units + COST;
    }
    u = max(0, min((int)x - COST, units - 1));
  }
  __device__ __forceinline__ void next(const Params& p) {
    u = 0;
    if (++rb >= blocks_of(p, q, RB)) {
      rb = 0;
      if (++h == p.c.Hkv) {
        h = 0;
#pragma unroll 1
        do {
          if (++r >= p.a.n_req) return;
          q = request(p, r);
        } while (q.nq == 0);
      }
    }
    settle(p);
  }
};

// ---------------------------------------------------------------------------
// pieces: O (not divided by l), m and l of an item's rows
// ---------------------------------------------------------------------------
// slot: [rows][D] floats, then [rows] (m, l)
template <int D, int RB>
struct Slot {
  static constexpr int kFloats = RB * (D + 2);
  static __device__ __forceinline__ float2* ml(float* s) { return reinterpret_cast<float2*>(s + RB * D); }
  static __device__ __forceinline__ const float2* ml(const float* s) {
    return reinterpret_cast<const float2*>(s + RB * D);
  }
};
// What a CTA leaves for the joining of items that cross CTAs: the state of its head piece
// (the part of an item that an earlier CTA began) and whether a tail piece (of an item
// begun here) is open.
struct CtaMeta {
  int head;   // 0 none, 1 ends the item, 2 the item goes on
  int tail;   // 1: open
  int begin, nq, h, rb;  // the tail's item
};

// Row rho of a block -> its row of q and o
__device__ __forceinline__ int64_t out_row(const Params& p, int begin, int h, int rb, int RB, int rho) {
  const unsigned x = (unsigned)rb * RB + rho, tok = x / (unsigned)p.n_rep;
  return (int64_t)(begin + (int)tok) * p.c.Hq + h * p.n_rep + (int)(x - tok * p.n_rep);
}
__device__ __forceinline__ int block_rows(const Params& p, int nq, int rb, int RB) {
  return (int)min((int64_t)RB, (int64_t)nq * p.n_rep - (int64_t)rb * RB);
}

// (rows are checked in a CPATTN_DEBUG build, as everywhere in the library)
__device__ __forceinline__ bool row_ok(const Params& p, int64_t row) {
  return in_bounds(row, 1, (int64_t)p.a.n_tokens * p.c.Hq, p.a.status);
}
__device__ __forceinline__ bool token_ok(const Params& p, int64_t token) {
  return in_bounds(token, 1, p.a.n_tokens, p.a.status);
}
__device__ __forceinline__ bool page_at_ok(const Params& p, int64_t at) {  // an entry of the table
  return in_bounds(at, 1, (int64_t)p.a.n_req * p.a.max_pages, p.a.status);
}
__device__ __forceinline__ void store4(const Params& p, int64_t row, int D, int ch, float4 v) {
  if (!row_ok(p, row)) return;
  if (p.c.bf16 && !p.c.o_f32)
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.a.o) + row * D + ch) =
        make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
  else
    *reinterpret_cast<float4*>(static_cast<float*>(p.a.o) + row * D + ch) = v;
}
// 1 / l for the rows that saw a key (NaN for those that met one)
__device__ __forceinline__ float inverse(float l) { return l == 0.f ? 0.f : 1.f / l; }
__device__ __forceinline__ float lse_of(float m, float l) {
  return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

__device__ __forceinline__ void store_lse(const Params& p, int64_t row, float m, float l) {
  if (p.a.lse && row_ok(p, row)) p.a.lse[row] = lse_of(m, l);
}

// An item's rows from their sums: divided and written, 4 channels a thread.
template <int D>
__device__ __forceinline__ void write_out(const Params& p, int64_t row, int ch, float m, float l, float4 o) {
  const float inv = inverse(l);
  store4(p, row, D, ch, make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
  if (ch == 0) store_lse(p, row, m, l);
}

// The sums of 4 channels of one row over pieces.  add() keeps the maximum so far.
struct Acc {
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void add(float2 ml, float4 x) {
    const float mn = max_nan(m, ml.x);
    const float base = mn == -INFINITY ? 0.f : mn;
    const float f = ex2(m - base), w = ex2(ml.x - base);
    m = mn;
    l = fmaf(l, f, w * ml.y);
    o.x = fmaf(o.x, f, w * x.x);
    o.y = fmaf(o.y, f, w * x.y);
    o.z = fmaf(o.z, f, w * x.z);
    o.w = fmaf(o.w, f, w * x.w);
  }
};

// ---------------------------------------------------------------------------
// finding a run
// ---------------------------------------------------------------------------
// Inclusive prefix sums of cost over the requests, per_sum of them an entry, and the total.
// Every thread of the CTA takes part.
template <typename It, int THREADS>
__device__ __forceinline__ int64_t sum_costs(const Params& p, int64_t* sums, int64_t* warp_part) {
  constexpr int PT = kSums / THREADS > 0 ? kSums / THREADS : 1, WARPS = THREADS / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // thread t's entries are PT neighbours, so one scan over threads gives all sums (threads
  // past the last entry have no requests)
  int64_t mine[PT], run = 0;
#pragma unroll
  for (int i = 0; i < PT; ++i) {
    const int64_t r0 = (int64_t)(threadIdx.x * PT + i) * p.per_sum;
#pragma unroll 1
    for (int64_t r = r0; r < r0 + p.per_sum && r < p.a.n_req; ++r) {
      const Req q = request(p, (int)r);
      if (q.nq > 0) run += It::head_cost(p, q) * p.c.Hkv;
    }
    mine[i] = run;
  }
  int64_t inc = run;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, inc, m);
    if (lane >= m) inc += y;
  }
  if (lane == 31) warp_part[warp] = inc;
  __syncthreads();
  int64_t before = 0, total = 0;
#pragma unroll 4
  for (int w = 0; w < WARPS; ++w) {
    if (w < warp) before += warp_part[w];
    total += warp_part[w];
  }
#pragma unroll
  for (int i = 0; i < PT; ++i)
    if (threadIdx.x * PT + i < kSums) sums[threadIdx.x * PT + i] = before + inc - run + mine[i];
  __syncthreads();
  return total;
}
// This CTA's run of the line.  CTAs that would get nothing are not counted, so an item's
// CTAs are neighbours.
template <typename Int>
__device__ __forceinline__ void cta_run(Int total, Int& c0, Int& c1) {
  const int ctas = (int)max((Int)1, min((Int)gridDim.x, total));
  const int cta = min((int)blockIdx.x, ctas);
  c0 = part_of(total, cta, ctas);
  c1 = part_of(total, min(cta + 1, ctas), ctas);
}
// The item and unit at place v of the line (r = n_req behind its end).  Called by a whole warp;
// each half looks for a place of its own.
template <typename It>
__device__ __forceinline__ It item_at(const Params& p, const int64_t* sums, int64_t v) {
  static_assert(kSums == 256, "16 entries of 16");
  // first entry whose sum is past v: first its sixteen, then it
  const int lane = threadIdx.x & 31, i = lane & 15, half = lane & 16;
  const uint32_t b0 = __ballot_sync(0xffffffffu, sums[16 * i + 15] > v) >> half & 0xffffu;
  const int g = b0 ? __ffs(b0) - 1 : 15;
  const uint32_t b1 = __ballot_sync(0xffffffffu, sums[16 * g + i] > v) >> half & 0xffffu;
  const int lo = b1 ? 16 * g + __ffs(b1) - 1 : kSums;
  It x;
  x.seen = x.units = 0;
  x.q = {0, 0, 0};
  x.locate(p, lo * p.per_sum, lo < kSums ? v - (lo ? sums[lo - 1] : 0) : 0);
  return x;
}

// ---------------------------------------------------------------------------
// items that cross CTAs (in a launch of its own, behind the one that left the pieces)
// ---------------------------------------------------------------------------
// An item's CTAs are the one that began it (its tail piece) and those behind it up to the one
// that ends it (their head pieces); each joins a part of the item's numbers.  slots: a head
// and a tail slot per CTA; smem: kJoinBytes.  The states come in one load; few numbers leave
// threads over: those share the pieces and meet in shared memory.
template <int THREADS>
constexpr int kJoinBytes = THREADS * (int)sizeof(Acc) + kMaxSms * (int)sizeof(CtaMeta);
template <int D, int RB, int THREADS>
__device__ __forceinline__ void join_ctas(const Params& p, const CtaMeta* states, const float* slots, void* smem) {
  using S = Slot<D, RB>;
  constexpr int V = D / 4;
  static_assert(THREADS >= kMaxSms, "a state a thread");
  Acc* const scratch = static_cast<Acc*>(smem);
  CtaMeta* const meta = reinterpret_cast<CtaMeta*>(scratch + THREADS);
  const int lane = threadIdx.x & 31, me = blockIdx.x, ctas = gridDim.x;
  if ((int)threadIdx.x < ctas) meta[threadIdx.x] = states[threadIdx.x];
  __syncthreads();
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {  // the item of this CTA's head, that of its tail
    int owner = me;
    if (which == 0) {
      if (meta[me].head == 0) continue;
      owner = -1;
      for (int i = me - 1; i >= 0 && owner < 0; i -= 32) {
        const uint32_t b = __ballot_sync(0xffffffffu, i - lane >= 0 && meta[max(i - lane, 0)].tail != 0);
        if (b) owner = i - (__ffs(b) - 1);
      }
      if (owner < 0) continue;  // (only if a CTA gave up)
    } else if (meta[me].tail == 0) {
      continue;
    }
    int n = ctas - owner;  // the item's CTAs
    for (int i = owner + 1; i < ctas; i += 32) {
      const uint32_t b = __ballot_sync(0xffffffffu, i + lane < ctas && meta[min(i + lane, ctas - 1)].head != 2);
      if (b) {
        n = i - owner + __ffs(b);
        break;
      }
    }
    n = min(n, ctas - owner);
    const CtaMeta cm = meta[owner];
    const int all = block_rows(p, cm.nq, cm.rb, RB) * V;
    const int e0 = all * (me - owner) / n, e1 = all * (me - owner + 1) / n;
    const int parts = e1 - e0;
    if (parts <= 0) continue;
    const int shares = max(1, min(THREADS / parts, n)), share = threadIdx.x / parts;
    const float* const first = slots + 2 * (size_t)owner * S::kFloats;
    if (shares == 1) {
      // four numbers' loads at a time (the stores in between might alias them otherwise)
      for (int i0 = threadIdx.x; i0 < parts; i0 += 4 * THREADS) {
        Acc acc[4];
        for (int i = 0; i < n; ++i) {
          const float* s = first + (i ? 2 * (size_t)i : 1) * S::kFloats;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const int e = e0 + min(i0 + u * THREADS, parts - 1), row = e / V, ch = (e - row * V) * 4;
            acc[u].add(S::ml(s)[row], *reinterpret_cast<const float4*>(s + row * D + ch));
          }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (i0 + u * THREADS >= parts) break;
          const int e = e0 + i0 + u * THREADS, row = e / V, ch = (e - row * V) * 4;
          write_out<D>(p, out_row(p, cm.begin, cm.h, cm.rb, RB, row), ch, acc[u].m, acc[u].l, acc[u].o);
        }
      }
      continue;
    }
    __syncthreads();  // the scratch of the item before
    {
      const int e = e0 + threadIdx.x % parts, row = e / V, ch = (e - row * V) * 4;
      Acc acc;
      if (share < shares) {
#pragma unroll 4
        for (int i = share; i < n; i += shares) {
          const float* s = first + (i ? 2 * (size_t)i : 1) * S::kFloats;
          acc.add(S::ml(s)[row], *reinterpret_cast<const float4*>(s + row * D + ch));
        }
      }
      scratch[threadIdx.x] = acc;
    }
    __syncthreads();
    if ((int)threadIdx.x < parts) {
      Acc acc = scratch[threadIdx.x];
      for (int i = 1; i < shares; ++i) {
        const Acc& x = scratch[threadIdx.x + i * parts];
        acc.add(make_float2(x.m, x.l), x.o);
      }
      const int e = e0 + threadIdx.x, row = e / V, ch = (e - row * V) * 4;
      write_out<D>(p, out_row(p, cm.begin, cm.h, cm.rb, RB, row), ch, acc.m, acc.l, acc.o);
    }
  }
}

}  // namespace cattn

// ---- cache_prompt.cu: many query rows per K/V head, bf16 --------------------
size_t cache_prompt_workspace(int D);
cudaError_t launch_cache_prompt(const cattn::Params& p, int sms, cudaStream_t st);

}  // namespace cpattn
