// Attention of new tokens over the 4-bit cache.
//
// One warp per query row and head: the row's keys one after the other, each lane D / 32
// channels, the running maximum and sum of the softmax in float32.
#include <math.h>

#include "cache.cuh"

namespace cpattn {
namespace cattn {

constexpr int kThreads = 128;
constexpr float kLn2 = 0.69314718055994530942f;

template <int D, typename T, bool OF32>
__global__ void __launch_bounds__(kThreads) simple_kernel(Cache c, CacheAttnArgs a) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int64_t id = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (id >= (int64_t)a.n_tokens * c.Hq) return;
  const int row = (int)(id / c.Hq), hq = (int)(id - (int64_t)row * c.Hq);
  const int h = hq / (c.Hq / c.Hkv);
  if (row >= a.q_start[a.n_req]) return;
  int lo = 0, hi = a.n_req;  // last request that starts at or before the row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.q_start[mid] <= row) lo = mid;
    else hi = mid;
  }
  const int r = lo;
  const int begin = a.q_start[r], nq = a.q_start[r + 1] - begin;
  if (row < begin || row >= begin + nq) return;
  const int64_t most = (int64_t)a.max_pages * c.page;
  int len = a.kv_len[r];
  len = len < 0 ? 0 : len > most ? (int)most : len;
  const int64_t seen = c.causal ? (int64_t)len - nq + (row - begin) + 1 : len;
  float q[E], o[E], m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; ++e) {
    q[e] = (float)static_cast<const T*>(a.q)[row * a.qs.token + hq * a.qs.head + lane * E + e];
    o[e] = 0.f;
  }
  const float sl2 = c.scale * 1.44269504088896340736f;
  const int w = lane * E / 8;        // word of this lane's channels
  for (int64_t p = 0; p < seen; ++p) {
    const int pg = a.table[(int64_t)r * a.max_pages + p / c.page];
    if (pg < 0 || pg >= c.n_pages) continue;
    const int off = (int)(p % c.page), t = off % kCacheTile;
    const uint8_t* tile = a.cache + c.tile_at(pg, h, off / kCacheTile);
    float kv[2][E];
    for (int x = 0; x < 2; ++x) {
      const uint8_t* half = tile + x * c.half_tile();
      const int rr = x ? cache_v_row(t) : t;
      const uint32_t word = reinterpret_cast<const uint32_t*>(half)[rr * (D / 8) + w];
      const uint32_t az = reinterpret_cast<const uint32_t*>(
          half + kCacheTile * c.row_bytes())[rr * c.groups() + w * 8 / c.G];
      uint32_t u[4];
      if (x) codes_to_bf16<false>(word, u);
      else codes_to_bf16<true>(word, u);
      for (int e = 0; e < E; ++e) {
        const int ch = (lane * E + e) & 7;
        uint32_t y = 0;
        for (int i = 0; i < 4; ++i)
          if (i == ch >> 1) y = bf16x2_fma(u[i], az_a2(az), az_z2(az));
        kv[x][e] = __uint_as_float((ch & 1) ? y & 0xffff0000u : y << 16);
      }
    }
    float s = 0.f;
    for (int e = 0; e < E; ++e) s = fmaf(q[e], kv[0][e], s);
    for (int i = 16; i; i >>= 1) s += __shfl_xor_sync(0xffffffffu, s, i);
    s *= sl2;
    const float mn = max_nan(m, s);  // a NaN score makes its row NaN
    const float f = mn == -INFINITY ? 1.f : exp2f(m - mn), pr = mn == -INFINITY ? 0.f : exp2f(s - mn);
    l = l * f + pr;
    for (int e = 0; e < E; ++e) o[e] = o[e] * f + pr * kv[1][e];
    m = mn;
  }
  const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
  using O = std::conditional_t<OF32, float, T>;
  for (int e = 0; e < E; ++e)
    static_cast<O*>(a.o)[((int64_t)row * c.Hq + hq) * D + lane * E + e] = (O)(o[e] * inv);
  if (lane == 0 && a.lse)
    a.lse[(int64_t)row * c.Hq + hq] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

}  // namespace cattn

size_t cache_attn_workspace(const Cache&) { return 256; }

template <int D>
static void launch_simple(const Cache& c, const CacheAttnArgs& a, cudaStream_t st) {
  const int64_t rows = (int64_t)a.n_tokens * c.Hq;
  const unsigned grid = (unsigned)((rows + 3) / 4);
  if (!c.bf16)
    cattn::simple_kernel<D, float, true><<<grid, cattn::kThreads, 0, st>>>(c, a);
  else if (c.o_f32)
    cattn::simple_kernel<D, __nv_bfloat16, true><<<grid, cattn::kThreads, 0, st>>>(c, a);
  else
    cattn::simple_kernel<D, __nv_bfloat16, false><<<grid, cattn::kThreads, 0, st>>>(c, a);
}

cudaError_t launch_cache_attn(const Cache& c, const CacheAttnArgs& a, cudaStream_t st) {
  timing_begin("cache_attn", st);
  if (c.D == 128) launch_simple<128>(c, a, st);
  else launch_simple<64>(c, a, st);
  timing_end(st);
  return cudaGetLastError();
}

}  // namespace cpattn
