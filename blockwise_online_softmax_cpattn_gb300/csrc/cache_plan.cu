// Block tables, query offsets and slots of the 4-bit cache from request lengths.
//
// With P = page and c(x) = ceil(x / P): request r needs n_r = max(c(new) - c(old), 0)
// pages, gives back g_r = max(c(old) - c(new), 0) and brings t_r = max(new - old, 0)
// tokens.  Three prefix sums over the requests settle everything else:
//   returned page number i of the call (in request order) goes to free_list[F + i],
//     F the pages free before;
//   with A = F + sum g the pages there are then, request r is served iff its prefix
//     sum of n through r is at most A, and taken page number i is the list's entry
//     A - 1 - i: a free one below F, above it a returned one, read from its request's
//     table row, which nothing writes -- so taking needs no wait for returning;
//   new token i belongs to the request whose run of the sums of t holds i.
// A binary search in the sums gives every page and token its request.
//
// A step of a running server has a few dozen requests and tokens: bound by latency, so
// all of it is one launch of one CTA with the sums in shared memory.  A batch of prompts
// has more tokens than one SM writes quickly: there the sums stay in the workspace and
// a second launch, a programmatic dependent of the first, spreads pages and tokens over
// the GPU.  Measured: 64 requests that each add a token 7 us; 700 requests, 240 000 tokens,
// 15 us, of which the second launch is 10 (a chain of loads: sums, the search, the request's
// numbers, the table; the sums in shared memory instead changed nothing).
#include "cache.cuh"

namespace cpattn {
namespace plan {

constexpr int kScanThreads = 1024;
constexpr int kFillThreads = 256;
constexpr int kSmallReq = 1024;       // the sums of this many requests stay on chip
// Tokens that one CTA fills about as fast as a second launch starts, us (one CTA, two
// launches): 64 requests, 512 tokens 6.2, 8.3; 2048: 8.3, 8.6; 4096: 9.4, 8.3; 512 requests, 4096:
// 10.3, 10.8; 1024 requests, 4096: 11.4, 12.3.
// Pages taken or returned are not counted: the rule would need the lengths, or a bound that most
// decoding steps exceed.  So many pages with few tokens are slow, all right though they are: 64 slots
// and 700 requests that return 250 pages each 139 us, 1000 that return 500 each 396; past 1024
// requests the second launch has a CTA per 256 slots, and 1500 that return 500 each take 2170 us
// with 64 slots, 158 with 5000, 3000 that return 100 each 967 with none, 17 with 300000.
constexpr int kSmallItems = 4096;

// The per-request results of the sums: exclusive prefix sums of t, n (of the served: a
// request that is not adds nothing) and g, and what pages and tokens are found from.
struct Sums {
  int *start, *need, *back, *old_len, *new_pages;
  __device__ static Sums at(int* base, int n_req) {
    const int n = n_req + 1;
    return {base, base + n, base + 2 * n, base + 3 * n, base + 4 * n};
  }
};
constexpr int kArrays = 5, kTotals = 4;  // totals: F, A, pages taken, pages returned

__device__ __forceinline__ int clampi(int x, int lo, int hi) { return x < lo ? lo : x > hi ? hi : x; }

// last r in [0, n) with sum[r] <= i, for sum[0] = 0 <= i < sum[n]: in a run of equal sums
// the last is the one that adds something
__device__ __forceinline__ int find(const int* sum, int n, int i) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sum[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}
struct View {
  PlanArgs a;
  Sums s;
  int F, A, taken, returned;
  __device__ __forceinline__ int pages_old(int r) const { return (s.old_len[r] + a.page - 1) / a.page; }
  // returned page number i
  __device__ __forceinline__ int back_page(int i) const {
    const int r = find(s.back, a.n_req, i);
    return a.table[(int64_t)r * a.max_pages + s.new_pages[r] + (i - s.back[r])];
  }
  // taken page number i
  __device__ __forceinline__ int take_page(int i) const {
    const int at = A - 1 - i;
    return at >= F ? back_page(at - F) : a.free_list[at];
  }
};

__device__ void fill(const View& v, int64_t first, int64_t stride) {
  const PlanArgs& a = v.a;
  for (int64_t i = first; i < v.returned; i += stride)
    if (v.F + i < a.n_pages) a.free_list[v.F + i] = v.back_page((int)i);
  for (int64_t i = first; i < v.taken; i += stride) {
    const int r = find(v.s.need, a.n_req, (int)i);
    a.table[(int64_t)r * a.max_pages + v.pages_old(r) + ((int)i - v.s.need[r])] = v.take_page((int)i);
  }
  const int tokens = v.s.start[a.n_req];
  for (int64_t i = first; i < a.n_slots; i += stride) {
    int slot = -1;
    if (i < tokens) {
      const int r = find(v.s.start, a.n_req, (int)i);
      const int pos = v.s.old_len[r] + ((int)i - v.s.start[r]);
      const int pg = pos / a.page, have = v.pages_old(r);
      const int need = v.s.need[r + 1] - v.s.need[r];
      const bool served = v.s.new_pages[r] <= have || need > 0;
      if (served) {
        const int id = pg < have ? a.table[(int64_t)r * a.max_pages + pg]
                                 : v.take_page(v.s.need[r] + pg - have);
        if (id >= 0 && id < a.n_pages) slot = id * a.page + (pos - pg * a.page);
      }
    }
    a.slots[i] = slot;
  }
}

__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, m);
    if (lane >= m) x += y;
  }
  return x;
}

// One CTA: the sums (in shared memory, SMALL, or the workspace), lengths and offsets out,
// and with SMALL the pages and slots too.
template <bool SMALL>
__global__ void __launch_bounds__(kScanThreads) scan_kernel(PlanArgs a) {
  __shared__ int sums_smem[SMALL ? kArrays * (kSmallReq + 1) : 1];
  __shared__ int64_t part[3][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Sums s = Sums::at(SMALL ? sums_smem : a.ws + kTotals, a.n_req);
  const int F = clampi(*a.n_free, 0, a.n_pages);
  const int most = a.max_pages * a.page;
  // sums of need and back (each below 2^31: at most the table's entries) in one 64-bit
  // word, of tokens in another
  int64_t run_nb = 0, run_t = 0;
  if (!SMALL) griddep_launch_dependents();  // fill_kernel waits for this grid's end itself
  // how many pages come back decides who is served
  int64_t returned = 0;
  for (int base = 0; base < a.n_req; base += kScanThreads) {
    const int r = base + threadIdx.x;
    int g = 0;
    if (r < a.n_req) {
      const int po = (clampi(a.len_old[r], 0, most) + a.page - 1) / a.page;
      const int pn = (clampi(a.len_new[r], 0, most) + a.page - 1) / a.page;
      g = po > pn ? po - pn : 0;
    }
    returned += g;
  }
  {
    const int64_t w = warp_scan(returned, lane);
    if (lane == 31) part[2][warp] = w;
    __syncthreads();
    const int64_t x = warp_scan(lane < kScanThreads / 32 ? part[2][lane] : 0, lane);
    returned = __shfl_sync(0xffffffffu, x, 31);
  }
  const int64_t have = F + returned;
  const int A = (int)(have < a.n_pages ? have : a.n_pages);
  int64_t taken = 0;  // this thread's
  for (int base = 0; base < a.n_req; base += kScanThreads) {
    const int r = base + threadIdx.x;
    int o = 0, w = 0, n = 0, g = 0, t = 0, po = 0, pn = 0;
    if (r < a.n_req) {
      o = clampi(a.len_old[r], 0, most);
      w = clampi(a.len_new[r], 0, most);
      po = (o + a.page - 1) / a.page;
      pn = (w + a.page - 1) / a.page;
      n = pn > po ? pn - po : 0;
      g = po > pn ? po - pn : 0;
      t = w > o ? w - o : 0;
    }
    const int64_t nb = ((int64_t)g << 32) | n;
    const int64_t inb = warp_scan(nb, lane), it = warp_scan(t, lane);
    if (lane == 31) part[0][warp] = inb, part[1][warp] = it;
    __syncthreads();
    const int64_t cn = warp_scan(part[0][lane], lane), ct = warp_scan(part[1][lane], lane);
    const int64_t before_n = __shfl_sync(0xffffffffu, cn, (warp + 31) & 31);
    const int64_t before_t = __shfl_sync(0xffffffffu, ct, (warp + 31) & 31);
    const int64_t xnb = run_nb + (warp ? before_n : 0) + inb - nb;  // exclusive
    const int64_t xt = run_t + (warp ? before_t : 0) + it - t;
    run_nb += __shfl_sync(0xffffffffu, cn, 31);
    run_t += __shfl_sync(0xffffffffu, ct, 31);
    __syncthreads();  // part is written again in the next round
    if (r < a.n_req) {
      const int64_t xn = xnb & 0xffffffff;
      const bool served = n == 0 || xn + n <= A;
      if (served) taken += n;
      s.start[r] = (int)(xt < 0x7fffffff ? xt : 0x7fffffff);
      s.need[r] = (int)xn;
      s.back[r] = (int)(xnb >> 32);
      s.old_len[r] = o;
      s.new_pages[r] = pn;
      a.q_start[r] = s.start[r];
      a.len_out[r] = served ? w : o;
    }
  }
  {
    const int64_t w = warp_scan(taken, lane);
    if (lane == 31) part[2][warp] = w;
    __syncthreads();
    const int64_t x = warp_scan(part[2][lane], lane);
    taken = __shfl_sync(0xffffffffu, x, 31);
  }
  // the served that need pages are the first of them: past those the sum stays
  for (int r = threadIdx.x; r < a.n_req; r += kScanThreads)
    if (s.need[r] > taken) s.need[r] = (int)taken;
  if (threadIdx.x == 0) {
    const int total = (int)(run_t < 0x7fffffff ? run_t : 0x7fffffff);
    s.start[a.n_req] = total;
    s.need[a.n_req] = (int)taken;
    s.back[a.n_req] = (int)returned;
    a.q_start[a.n_req] = total;
    *a.n_free_out = A - (int)taken;
    if (!SMALL) {
      a.ws[0] = F;
      a.ws[1] = A;
      a.ws[2] = (int)taken;
      a.ws[3] = (int)returned;
    }
  }
  if (SMALL) {
    __syncthreads();
    fill(View{a, s, F, A, (int)taken, (int)returned}, threadIdx.x, kScanThreads);
  }
}

__global__ void __launch_bounds__(kFillThreads) fill_kernel(PlanArgs a) {
  griddep_wait();
  const View v{a, Sums::at(a.ws + kTotals, a.n_req), a.ws[0], a.ws[1], a.ws[2], a.ws[3]};
  fill(v, (int64_t)blockIdx.x * kFillThreads + threadIdx.x, (int64_t)gridDim.x * kFillThreads);
}

}  // namespace plan

size_t cache_plan_workspace(int n_req) {
  const size_t ints = plan::kTotals + (size_t)plan::kArrays * ((size_t)n_req + 1);
  return (ints * sizeof(int) + 255) / 256 * 256;
}

cudaError_t launch_cache_plan(const PlanArgs& a, cudaStream_t st) {
  using namespace plan;
  timing_begin("cache_plan", st);
  if (a.n_req <= kSmallReq && a.n_slots <= kSmallItems) {
    scan_kernel<true><<<1, kScanThreads, 0, st>>>(a);
  } else {
    scan_kernel<false><<<1, kScanThreads, 0, st>>>(a);
    cudaLaunchConfig_t cfg = {};
    // one item a thread where that many fit on the GPU at once, else a few each
    const int64_t want = ((int64_t)a.n_slots + kFillThreads - 1) / kFillThreads;
    cfg.gridDim = (unsigned)(want < 1 ? 1 : want > 152 * 8 ? 152 * 8 : want);
    cfg.blockDim = kFillThreads;
    cfg.stream = st;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, fill_kernel, a);
    if (e != cudaSuccess) {
      timing_end(st);
      return e;
    }
  }
  timing_end(st);
  return cudaGetLastError();
}

}  // namespace cpattn
