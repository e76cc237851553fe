// Rows into the 4-bit cache and out of it.
//
// Both are copies that convert: a thread takes 8 channels of one row (16 or 32 bytes of
// a tensor, one 32-bit word of codes), the D / 8 threads of a row sit side by side in a
// warp, and the D / G groups of the row are runs of G / 8 of them, which find their
// minimum and maximum with shuffles.  Bound by HBM: 2 (or 4) bytes in and 0.56 out a
// channel at group 64.
#include "cache.cuh"

namespace cpattn {
namespace rows {

constexpr int kThreads = 256;

// 8 channels of a row as floats
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w;
  x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
}
__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&x)[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(p);
  x[0] = lo_f(a.x), x[1] = hi_f(a.x), x[2] = lo_f(a.y), x[3] = hi_f(a.y);
  x[4] = lo_f(a.z), x[5] = hi_f(a.z), x[6] = lo_f(a.w), x[7] = hi_f(a.w);
}

// The code word of 8 channels (channel 2p + e in bits 4(p + 4e)) and the group's (a, z);
// `lanes` threads share a group.  The code is the number of borders a (33 + 2j) / 32
// that d = x - z is above: j near 16 d / a - 16.5 is found by a multiplication with the
// rounded 16 / a, at most one off, and d is then compared with border j itself, whose
// product is exact in float32 (8 + 6 bits).
__device__ __forceinline__ uint32_t quantise8(float (&x)[8], int lanes, uint32_t& az, int* status) {
  float lo = x[0], hi = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min_nan(lo, x[i]);
    hi = max_nan(hi, x[i]);
  }
  if (!(lo >= -kCacheHuge && hi <= kCacheHuge)) {  // also true of a NaN
    latch_status(status, kStatusRange);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i] = isnan(x[i]) ? 0.f : fminf(fmaxf(x[i], -kCacheHuge), kCacheHuge);
      lo = i == 0 ? x[0] : fminf(lo, x[i]);
      hi = i == 0 ? x[0] : fmaxf(hi, x[i]);
    }
  }
  for (int m = 1; m < lanes; m <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
  }
  const __nv_bfloat16 ab = __float2bfloat16_rn(__fmul_rn(hi - lo, 16.f / 15.f));
  float a = __bfloat162float(ab);
  if (a < kCacheTiny) a = 0.f;
  const __nv_bfloat16 zb = __float2bfloat16_rn(__fsub_rn(lo, a));
  const float z = __bfloat162float(zb);
  az = (a == 0.f ? 0u : (uint32_t)__bfloat16_as_ushort(ab)) | (uint32_t)__bfloat16_as_ushort(zb) << 16;
  if (a == 0.f) return 0u;
  const float r = 16.f / a, a16 = a * 0.0625f, b0 = a * 1.03125f;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float d = __fsub_rn(x[i], z);
    const float t = fminf(fmaxf(fmaf(d, r, -16.5f), 0.f), 14.f);
    const float m = t + 12582912.f;  // rounds t to a whole number j, in the low bits too
    const float j = m - 12582912.f;
    const uint32_t code = (__float_as_uint(m) & 15u) + (d > fmaf(j, a16, b0) ? 1u : 0u);
    w |= code << (4 * ((i >> 1) + 4 * (i & 1)));
  }
  return w;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    append_kernel(Cache c, int64_t n_rows, int n, const T* k, RowStrides ks, const T* v, RowStrides vs,
                  const int* slots, uint8_t* cache, int* status) {
  const int tpr = c.D / 8;  // threads per row
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t row = id / tpr;
  const int w = (int)(id % tpr);
  // rows of tokens side by side, then heads, then keys and values
  const int64_t hv = row / n;
  const int tok = (int)(row - hv * n);
  const int is_v = hv >= c.Hkv;
  const int h = (int)hv - is_v * c.Hkv;
  const bool in = row < n_rows;
  const int slot = in ? slots[tok] : -1;
  const bool live = slot >= 0 && slot < c.slots();
  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (live) {
    const RowStrides s = is_v ? vs : ks;
    load8((is_v ? v : k) + tok * s.token + h * s.head + w * 8, x);
  }
  uint32_t az;
  uint32_t word = quantise8(x, c.G / 8, az, status);  // whole warps: shuffles inside
  if (!live) return;
  const int pg = slot / c.page, off = slot - pg * c.page;
  const int t = off % kCacheTile;
  uint8_t* half = cache + c.tile_at(pg, h, off / kCacheTile) + (is_v ? c.half_tile() : 0);
  const int r = is_v ? cache_v_row(t) : t;
  if (!is_v) word = __funnelshift_l(word, word, 3);
  reinterpret_cast<uint32_t*>(half)[r * tpr + w] = word;
  const int lanes = c.G / 8;
  if (w % lanes == 0)
    reinterpret_cast<uint32_t*>(half + kCacheTile * c.row_bytes())[r * c.groups() + w / lanes] = az;
}

__device__ __forceinline__ void store8(float* p, const uint32_t (&u)[4]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(lo_f(u[0]), hi_f(u[0]), lo_f(u[1]), hi_f(u[1]));
  reinterpret_cast<float4*>(p)[1] = make_float4(lo_f(u[2]), hi_f(u[2]), lo_f(u[3]), hi_f(u[3]));
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const uint32_t (&u)[4]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    read_kernel(Cache c, int64_t n_rows, int n, const int* slots, const uint8_t* cache, T* k,
                RowStrides ks, T* v, RowStrides vs) {
  const int tpr = c.D / 8;
  const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  const int64_t row = id / tpr;
  if (row >= n_rows) return;
  const int w = (int)(id % tpr);
  const int64_t hv = row / n;
  const int tok = (int)(row - hv * n);
  const int is_v = hv >= c.Hkv;
  const int h = (int)hv - is_v * c.Hkv;
  const int slot = slots[tok];
  uint32_t u[4] = {0u, 0u, 0u, 0u};
  if (slot >= 0 && slot < c.slots()) {
    const int pg = slot / c.page, off = slot - pg * c.page;
    const int t = off % kCacheTile;
    const uint8_t* half = cache + c.tile_at(pg, h, off / kCacheTile) + (is_v ? c.half_tile() : 0);
    const int r = is_v ? cache_v_row(t) : t;
    const uint32_t word = reinterpret_cast<const uint32_t*>(half)[r * tpr + w];
    const uint32_t az =
        reinterpret_cast<const uint32_t*>(half + kCacheTile * c.row_bytes())[r * c.groups() + w * 8 / c.G];
    if (is_v) codes_to_bf16<false>(word, kOnes, u);
    else codes_to_bf16<true>(word, kOnes, u);
#pragma unroll
    for (int p = 0; p < 4; ++p) u[p] = bf16x2_fma(u[p], az_a2(az), az_z2(az));
  }
  const RowStrides s = is_v ? vs : ks;
  store8((is_v ? v : k) + tok * s.token + h * s.head + w * 8, u);
}

}  // namespace rows

static cudaError_t row_grid(const Cache& c, int n, int64_t* rows_out, unsigned* grid) {
  const int64_t n_rows = (int64_t)2 * c.Hkv * n;
  const int64_t blocks = (n_rows * (c.D / 8) + rows::kThreads - 1) / rows::kThreads;
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  *rows_out = n_rows;
  *grid = (unsigned)blocks;
  return cudaSuccess;
}

cudaError_t launch_cache_append(const Cache& c, int n, const void* k, RowStrides ks, const void* v,
                                RowStrides vs, const int* slots, void* cache, int* status,
                                cudaStream_t st) {
  int64_t n_rows;
  unsigned grid;
  cudaError_t e = row_grid(c, n, &n_rows, &grid);
  if (e != cudaSuccess) return e;
  timing_begin("cache_append", st);
  if (c.bf16)
    rows::append_kernel<<<grid, rows::kThreads, 0, st>>>(
        c, n_rows, n, static_cast<const __nv_bfloat16*>(k), ks, static_cast<const __nv_bfloat16*>(v),
        vs, slots, static_cast<uint8_t*>(cache), status);
  else
    rows::append_kernel<<<grid, rows::kThreads, 0, st>>>(
        c, n_rows, n, static_cast<const float*>(k), ks, static_cast<const float*>(v), vs, slots,
        static_cast<uint8_t*>(cache), status);
  timing_end(st);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const Cache& c, int n, const int* slots, const void* cache, void* k,
                              RowStrides ks, void* v, RowStrides vs, cudaStream_t st) {
  int64_t n_rows;
  unsigned grid;
  cudaError_t e = row_grid(c, n, &n_rows, &grid);
  if (e != cudaSuccess) return e;
  timing_begin("cache_read", st);
  const uint8_t* cb = static_cast<const uint8_t*>(cache);
  if (c.bf16)
    rows::read_kernel<<<grid, rows::kThreads, 0, st>>>(c, n_rows, n, slots, cb,
                                                       static_cast<__nv_bfloat16*>(k), ks,
                                                       static_cast<__nv_bfloat16*>(v), vs);
  else
    rows::read_kernel<<<grid, rows::kThreads, 0, st>>>(c, n_rows, n, slots, cb, static_cast<float*>(k),
                                                       ks, static_cast<float*>(v), vs);
  timing_end(st);
  return cudaGetLastError();
}

}  // namespace cpattn
