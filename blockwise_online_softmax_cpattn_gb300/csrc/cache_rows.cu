// Rows into the 4-bit cache and out of it.
//
// Both are copies that convert: a thread takes 16 channels of a row (32 or 64 bytes of a
// tensor, two 32-bit words of codes), the D / 16 threads of a row sit side by side in a
// warp, and the D / G groups of the row are runs of G / 16 of them, which find their
// minimum and maximum with shuffles.  (With 8 channels a thread the work per group and
// address made it 30 % slower.)  Each thread does so for kRows tokens, all loads first.
// Bound by HBM: 2 (or 4) bytes in and 0.56 out a channel at group 64, and the other way
// round; close behind, appending, by its instructions, so pairs of channels go through the
// two-lane float32 operations.
// Measured (32768 tokens of 8 heads, D 128, group 64, bf16; 172 MB each): append 39 us, 4.4
// TB/s, 3.0 instructions a clock issue, 15 a value; read 33 us, 5.2 TB/s.  The same in float32
// (306 MB each): append 51 us, 6.0 TB/s, read 51.  float32, 5003 tokens of 12 heads of 64, group
// 32: append 10, read 9.
#include "cache.cuh"

namespace cpattn {
namespace rows {

constexpr int kThreads = 256;
constexpr int kReadRows = 4;  // of cpattn_cache_read
// tokens a thread works on: 64 bytes of loads in flight
template <typename T>
constexpr int kRows = sizeof(T) == 2 ? 2 : 1;

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 16 channels of a row
template <typename T>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 w[2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    w[0] = reinterpret_cast<const uint4*>(p)[0];
    w[1] = reinterpret_cast<const uint4*>(p)[1];
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ void floats(float2 (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[4 * i] = make_float2(lo_f(w[i].x), hi_f(w[i].x));
      x[4 * i + 1] = make_float2(lo_f(w[i].y), hi_f(w[i].y));
      x[4 * i + 2] = make_float2(lo_f(w[i].z), hi_f(w[i].z));
      x[4 * i + 3] = make_float2(lo_f(w[i].w), hi_f(w[i].w));
    }
  }
};
template <>
struct Raw<float> {
  float4 w[4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = reinterpret_cast<const float4*>(p)[i];
  }
  __device__ __forceinline__ void zero() { w[0] = w[1] = w[2] = w[3] = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void floats(float2 (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = make_float2(w[i].x, w[i].y);
      x[2 * i + 1] = make_float2(w[i].z, w[i].w);
    }
  }
};

// The code words of 16 channels (channel 2p + e of 8 in bits 4(p + 4e)) and the group's
// (a, z); LANES threads share a group.  The code is the number of borders a (33 + 2j) / 32 that
// d = x - z is above.  16 d / a - 16.5, held to [0, 14] and rounded, is a j such that the
// code is j or j + 1 (the float32 error of 16 / a matters nowhere near); d is compared with
// border j itself, whose product is exact in float32 (8 + 6 bits), so the code is exact.
// The four codes of a half word are summed as float32 numbers: below 2^16, so exactly.
template <int LANES>
__device__ __forceinline__ uint2 quantise16(float2 (&x)[8], uint32_t& az, int* range) {
  float lo = min_nan(x[0].x, x[0].y), hi = max_nan(x[0].x, x[0].y);
#pragma unroll
  for (int i = 1; i < 8; ++i) {
    lo = min3_nan(lo, x[i].x, x[i].y);
    hi = max3_nan(hi, x[i].x, x[i].y);
  }
  if (!(lo >= -kCacheHuge && hi <= kCacheHuge)) {  // also true of a NaN
    latch_status(range, kStatusRange);
    lo = INFINITY;
    hi = -INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[i].x = isnan(x[i].x) ? 0.f : fminf(fmaxf(x[i].x, -kCacheHuge), kCacheHuge);
      x[i].y = isnan(x[i].y) ? 0.f : fminf(fmaxf(x[i].y, -kCacheHuge), kCacheHuge);
      lo = fminf(lo, fminf(x[i].x, x[i].y));
      hi = fmaxf(hi, fmaxf(x[i].x, x[i].y));
    }
  }
#pragma unroll
  for (int m = 1; m < LANES; m <<= 1) {
    lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, m));
    hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, m));
  }
  const __nv_bfloat16 ab = __float2bfloat16_rn(__fmul_rn(hi - lo, 16.f / 15.f));
  float a = __bfloat162float(ab);
  const bool flat = a < kCacheTiny;
  if (flat) a = 0.f;
  const __nv_bfloat16 zb = __float2bfloat16_rn(__fsub_rn(lo, a));
  const float nz = -__bfloat162float(zb);
  az = (flat ? 0u : (uint32_t)__bfloat16_as_ushort(ab)) | (uint32_t)__bfloat16_as_ushort(zb) << 16;
  const float r = __fdividef(16.f / 14.f, a);  // of a flat group not used
  const float2 a16 = make_float2(a * 0.0625f, a * 0.0625f), b0 = make_float2(a * 1.03125f, a * 1.03125f);
  const float2 magic = make_float2(12582912.f, 12582912.f), nmagic = make_float2(-12582912.f, -12582912.f);
  const float2 k14 = make_float2(14.f, 14.f);
  uint32_t w[2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    float2 sum = make_float2(0.f, 0.f);
    float scale = 1.f;
#pragma unroll
    for (int i = 4 * half; i < 4 * half + 4; ++i) {
      const float2 d = add2(x[i], make_float2(nz, nz));
      const float2 t =
          make_float2(__saturatef(fmaf(d.x, r, -16.5f / 14.f)), __saturatef(fmaf(d.y, r, -16.5f / 14.f)));
      const float2 j = add2(fma2(t, k14, magic), nmagic);  // rounded to a whole number
      const float2 border = fma2(j, a16, b0);
      const float2 code = add2(j, make_float2(d.x > border.x ? 1.f : 0.f, d.y > border.y ? 1.f : 0.f));
      sum = fma2(code, make_float2(scale, scale), sum);
      scale *= 16.f;
    }
    w[half] = __byte_perm(__float_as_uint(sum.x + 8388608.f), __float_as_uint(sum.y + 8388608.f), 0x5410);
  }
  return flat ? make_uint2(0u, 0u) : make_uint2(w[0], w[1]);
}

// (16.f / 15.f and the roundings above are the format's; add2 rounds to nearest.)

// The cache of one K/V head's keys or values (block: that of page 0).
template <int D, int G>
struct Rows {
  static constexpr int kHalf = kCacheTile * (D / 2 + 4 * (D / G));
  Divider page;
  int64_t page_bytes;   // of all heads
  int64_t block_bytes;
  unsigned slots;
  int heads;
  static Rows of(const Cache& c) {
    return {Divider::of(c.page), c.Hkv * c.block_bytes(), c.block_bytes(), (unsigned)c.slots(), c.Hkv};
  }
  __device__ __forceinline__ int64_t first(int h, int is_v) const { return h * block_bytes + is_v * kHalf; }
  // the half tile of a slot, from the first, and the slot's row in it
  __device__ __forceinline__ int64_t half(int slot, int is_v, int& row) const {
    const int pg = page.div(slot), off = slot - pg * (int)page.d, t = off & (kCacheTile - 1);
    row = is_v ? cache_v_row(t) : t;
    return pg * page_bytes + (int64_t)(off / kCacheTile) * (2 * kHalf);
  }
};

template <typename T, int D, int G>
__global__ void __launch_bounds__(kThreads)
    append_kernel(const Rows<D, G> c, int n, const T* k, RowStrides ks, const T* v, RowStrides vs,
                  const int* slots, uint8_t* cache, int* range) {
  constexpr int TPR = D / 16, LANES = G / 16, STEP = kThreads / TPR, N = kRows<T>;
  const int w = threadIdx.x % TPR;
  const int is_v = blockIdx.y >= (unsigned)c.heads;
  const int h = blockIdx.y - is_v * c.heads;
  const RowStrides st = is_v ? vs : ks;
  const T* src = (is_v ? v : k) + h * st.head + w * 16;
  // tokens of a CTA: STEP neighbours at a time
  const int64_t tok0 = (int64_t)blockIdx.x * (STEP * N) + threadIdx.x / TPR;
  int slot[N];
  Raw<T> raw[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t tok = tok0 + i * STEP;
    slot[i] = tok < n ? slots[tok] : -1;
    if ((unsigned)slot[i] >= c.slots) slot[i] = -1;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    raw[i].zero();
    if (slot[i] >= 0) raw[i].load(src + (tok0 + i * STEP) * st.token);
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float2 x[8];
    raw[i].floats(x);
    uint32_t az;
    uint2 word = quantise16<LANES>(x, az, range);  // whole warps: shuffles inside
    if (slot[i] < 0) continue;
    int r;
    uint8_t* half = cache + c.first(h, is_v) + c.half(slot[i], is_v, r);
    if (!is_v) word = make_uint2(__funnelshift_l(word.x, word.x, 3), __funnelshift_l(word.y, word.y, 3));
    reinterpret_cast<uint2*>(half)[r * TPR + w] = word;
    if (w % LANES == 0)
      reinterpret_cast<uint32_t*>(half + kCacheTile * (D / 2))[r * (D / G) + w / LANES] = az;
  }
}

// wide: rows lie on 32-byte boundaries
__device__ __forceinline__ void store8(float* p, const uint32_t (&u)[4], int wide) {
  if (wide) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(lo_f(u[0])),
                 "f"(hi_f(u[0])), "f"(lo_f(u[1])), "f"(hi_f(u[1])), "f"(lo_f(u[2])), "f"(hi_f(u[2])),
                 "f"(lo_f(u[3])), "f"(hi_f(u[3]))
                 : "memory");
  } else {
    reinterpret_cast<float4*>(p)[0] = make_float4(lo_f(u[0]), hi_f(u[0]), lo_f(u[1]), hi_f(u[1]));
    reinterpret_cast<float4*>(p)[1] = make_float4(lo_f(u[2]), hi_f(u[2]), lo_f(u[3]), hi_f(u[3]));
  }
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const uint32_t (&u)[4], int) {
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

// (8 channels a thread here: what a warp stores at a time is then contiguous.)
template <typename T, int D, int G>
__global__ void __launch_bounds__(kThreads)
    read_kernel(const Rows<D, G> c, const uint32_t ones, const int wide, int n, const int* slots,
                const uint8_t* cache, T* k, RowStrides ks, T* v, RowStrides vs) {
  constexpr int TPR = D / 8, LANES = G / 8, STEP = kThreads / TPR, N = kReadRows;
  const int w = threadIdx.x % TPR;
  const int is_v = blockIdx.y >= (unsigned)c.heads;
  const int h = blockIdx.y - is_v * c.heads;
  const RowStrides st = is_v ? vs : ks;
  T* dst = (is_v ? v : k) + h * st.head + w * 8;
  const int64_t tok0 = (int64_t)blockIdx.x * (STEP * N) + threadIdx.x / TPR;
  int slot[N];
  uint32_t word[N], az[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t tok = tok0 + i * STEP;
    slot[i] = tok < n ? slots[tok] : -1;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    word[i] = az[i] = 0u;
    if ((unsigned)slot[i] < c.slots) {
      int r;
      const uint8_t* half = cache + c.first(h, is_v) + c.half(slot[i], is_v, r);
      word[i] = reinterpret_cast<const uint32_t*>(half)[r * TPR + w];
      az[i] = reinterpret_cast<const uint32_t*>(half + kCacheTile * (D / 2))[r * (D / G) + w / LANES];
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int64_t tok = tok0 + i * STEP;
    if (tok >= n) return;
    uint32_t u[4];
    if (is_v) codes_to_bf16<false>(word[i], ones, u);
    else codes_to_bf16<true>(word[i], ones, u);
#pragma unroll
    for (int p = 0; p < 4; ++p) u[p] = bf16x2_fma(u[p], az_a2(az[i]), az_z2(az[i]));  // (0, 0): zeros
    store8(dst + tok * st.token, u, wide);
  }
}

// f(T, D, G) for the cache's
template <typename F>
static cudaError_t dispatch(const Cache& c, F f) {
  auto by_format = [&](auto t) {
    using T = decltype(t);
    if (c.D == 128) {
      if (c.G == 128) return f(T(), std::integral_constant<int, 128>(), std::integral_constant<int, 128>());
      if (c.G == 64) return f(T(), std::integral_constant<int, 128>(), std::integral_constant<int, 64>());
      return f(T(), std::integral_constant<int, 128>(), std::integral_constant<int, 32>());
    }
    if (c.G == 64) return f(T(), std::integral_constant<int, 64>(), std::integral_constant<int, 64>());
    return f(T(), std::integral_constant<int, 64>(), std::integral_constant<int, 32>());
  };
  return c.bf16 ? by_format(__nv_bfloat16()) : by_format(0.f);
}

static dim3 grid_of(const Cache& c, int n, int rows, int channels) {
  const int step = kThreads / (c.D / channels) * rows;
  return dim3((unsigned)(((int64_t)n + step - 1) / step), 2 * c.Hkv);
}

}  // namespace rows

cudaError_t launch_cache_append(const Cache& c, int n, const void* k, RowStrides ks, const void* v,
                                RowStrides vs, const int* slots, void* cache, int* range,
                                cudaStream_t st) {
  timing_begin("cache_append", st);
  const cudaError_t e = rows::dispatch(c, [&](auto t, auto d, auto g) {
    using T = decltype(t);
    rows::append_kernel<T, decltype(d)::value, decltype(g)::value>
        <<<rows::grid_of(c, n, rows::kRows<T>, 16), rows::kThreads, 0, st>>>(
            rows::Rows<decltype(d)::value, decltype(g)::value>::of(c), n, static_cast<const T*>(k), ks,
            static_cast<const T*>(v), vs, slots, static_cast<uint8_t*>(cache), range);
    return cudaGetLastError();
  });
  timing_end(st);
  return e;
}

cudaError_t launch_cache_read(const Cache& c, int n, const int* slots, const void* cache, void* k,
                              RowStrides ks, void* v, RowStrides vs, cudaStream_t st) {
  // Rows on 32-byte boundaries take one store a thread in float32, others two of 16 bytes
  // (32768 tokens of 12 heads of 64: 40 us, 77 us for rows 16 bytes off.  Of those 8 us go when a
  // row's threads write side by side, but then aligned ones take 10 us in place of 8 for 5003
  // tokens; the rest is sectors that are written in parts.)
  const int wide = !(((uintptr_t)k | (uintptr_t)v) & 31) && !((ks.token | ks.head | vs.token | vs.head) & 7);
  timing_begin("cache_read", st);
  const cudaError_t e = rows::dispatch(c, [&](auto t, auto d, auto g) {
    using T = decltype(t);
    rows::read_kernel<T, decltype(d)::value, decltype(g)::value>
        <<<rows::grid_of(c, n, rows::kReadRows, 8), rows::kThreads, 0, st>>>(
            rows::Rows<decltype(d)::value, decltype(g)::value>::of(c), kOnes, wide, n, slots,
            static_cast<const uint8_t*>(cache), static_cast<T*>(k), ks, static_cast<T*>(v), vs);
    return cudaGetLastError();
  });
  timing_end(st);
  return e;
}

}  // namespace cpattn
