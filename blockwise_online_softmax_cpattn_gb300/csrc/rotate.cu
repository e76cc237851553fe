// What stands between a layer's projections and its attention, in one pass over the rows:
// RMS norm of each head of the queries and keys, rotation by position, the move into the
// attention's token order; values move along.  And its backward pass.
//
// A row of D channels belongs to D / 2P lanes, rounded up to a power of two, with P = 8 in bf16 (8
// lanes at D 128, four rows a warp), or 4 where D or the rotation is no multiple of 16 or rows are few
// (cut, below), and 4 in float32: vectors of 16 bytes.  Lane l owns
// pairs P l .. P l + P-1 of the rotation, as two vectors of P channels: at P l and rot/2 + P l when
// pairs lie half a rotation apart, else 2P channels in a row.  So a pair never crosses lanes, the
// only exchange is the norm's sum (three shuffles at D 128), and each row is read and written
// once.  (With P 4 the shuffles and what each head costs anyway take 58.8 us in the backward pass of
// 8000 tokens of 40 heads, with P 8 47.7.)
//
// A warp takes the same slots (four at D 128) of a run of heads, one head after the other: a
// slot's angles are the same in every head, so a lane forms the cosines and sines of its pairs
// once and keeps them in registers.  The rows of the next heads are on their way into shared memory
// meanwhile (cp.async, each lane its own 16-byte pieces, so nothing has to be synchronised): some
// 70 to 90 KB an SM, more than what 7 TB/s at a microsecond's latency takes, and no registers.
// The angle p f is formed in whole numbers, as 64 binary places of a turn: at position 10^5 a
// float32 product alone is off by 2^-8 of a radian, and the float64 units, two lanes an SM, took
// 2 us of a decoding step's 6.6.  Only what is left by whole quarter turns becomes a float32.
//
// Bound by memory: 64 bytes a lane and row against some 130 instructions.  32768 tokens of 40 heads
// of 128 (bf16): 107 us, 6.3 TB/s, 92 % of a copy's rate.  Backward, 8192 tokens of 48 heads: 56 us,
// 5.1 TB/s (75 %); 16 warps an SM at 128 registers leave a dependent instruction's wait (2.2 cycles
// of 7.6 an issue) as its largest stall.  A decoding step's 64 tokens: 4.1 us.
#include "layer.cuh"

namespace cpattn {
namespace rotate {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// P channels in a row as they lie in memory, and as numbers.
template <typename E, int P>
struct Vec;
template <int P>
struct Vec<__nv_bfloat16, P> {
  uint32_t w[P / 2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    if constexpr (P == 8) {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x, w[1] = x.y;
    }
  }
  __device__ __forceinline__ float at(int i) const {
    return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
};
template <int P>
struct Vec<float, P> {
  float w[P];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < P; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(p + i);
      w[i] = x.x, w[i + 1] = x.y, w[i + 2] = x.z, w[i + 3] = x.w;
    }
  }
  __device__ __forceinline__ float at(int i) const { return w[i]; }
};

template <int P>
__device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[P]) {
  if constexpr (P == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                              pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
  else
    *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}
template <int P>
__device__ __forceinline__ void store(float* p, const float (&x)[P]) {
#pragma unroll
  for (int i = 0; i < P; i += 4)
    *reinterpret_cast<float4*>(p + i) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
}

// A lane's two vectors as (first, second) of its pairs, and back.
template <bool NEAR, typename E, int P>
__device__ __forceinline__ void to_pairs(const Vec<E, P>& x, const Vec<E, P>& y, float (&a)[P], float (&b)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    if constexpr (NEAR) {
      a[i] = i < P / 2 ? x.at(2 * i) : y.at(2 * i - P);
      b[i] = i < P / 2 ? x.at(2 * i + 1) : y.at(2 * i + 1 - P);
    } else {
      a[i] = x.at(i), b[i] = y.at(i);
    }
  }
}
template <bool NEAR, typename E, int P>
__device__ __forceinline__ void store_pairs(E* row, int c0, int c1, const float (&a)[P], const float (&b)[P]) {
  if constexpr (NEAR) {
    float x[P], y[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      x[i] = i & 1 ? b[i / 2] : a[i / 2];
      y[i] = i & 1 ? b[(P + i) / 2] : a[(P + i) / 2];
    }
    store<P>(row + c0, x);
    store<P>(row + c1, y);
  } else {
    store<P>(row + c0, a);
    store<P>(row + c1, b);
  }
}

__device__ __forceinline__ float row_sum(float s, int lanes) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
    if (o < lanes) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Channels of a lane: its two vectors begin at c0 and c1.  Past the rotated pairs its 2P channels
// follow each other in either pairing, and are not turned.
template <bool NEAR, int P>
__device__ __forceinline__ void lane_channels(const Rotate& p, int l, int* c0, int* c1) {
  *c0 = 2 * P * l;
  *c1 = 2 * P * l + P;
  if (!NEAR && P * l < p.rot / 2) {
    *c0 = P * l;
    *c1 = P * l + p.rot / 2;
  }
}

// f / (2 pi) as 64 binary places of a turn (f = m 2^(e - 1075); whole turns fall away), so that
// p times it, modulo 2^64, is where position p stands.  Off by 2^-64 for f < 2.
__device__ __forceinline__ uint64_t turns_of(double f) {
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int e = (int)(bits >> 52) & 0x7FF;
  const uint64_t m = e ? (bits << 11) | 0x8000000000000000ull : 0;  // 64 binary places
  uint64_t g = __umul64hi(m, 0xA2F9836E4E441529ull);                 // 2^66 / (2 pi)
  const int s = e - 1024;
  g = s >= 64 || s <= -64 ? 0 : s >= 0 ? g << s : g >> -s;
  return bits >> 63 ? 0 - g : g;
}

// Sine and cosine of `at` 2^-64 turns.  The nearest quarter turn is taken off in whole numbers: the
// rest, an eighth at most, is rounded to a float32 off by less than 2^-25 radians (a float32 over a
// half turn: 2^-23.3).
__device__ __forceinline__ void sin_cos(uint64_t at, float* si, float* co) {
  const uint64_t up = at + (1ull << 61);
  const uint32_t q = (uint32_t)(up >> 62);
  const int64_t rest = (int64_t)(at - ((uint64_t)q << 62));
  float s, c;
  sincospif((float)(int32_t)(rest >> 30) * 1.16415321826934814453125e-10f, &s, &c);  // 2^-33
  const float x = q & 1 ? s : c, y = q & 1 ? c : s;
  *co = __uint_as_float(__float_as_uint(x) ^ ((q + 1) & 2) << 30);
  *si = __uint_as_float(__float_as_uint(y) ^ (q & 2) << 30);
}

// What a lane keeps for its slot: the two tokens (attention's and projection's side) and the turns.
template <int P>
struct Slot {
  int b, t, from;
  bool live;
  float co[P], si[P];
};

// Slots of the `group`'th group, 32 / lanes of them, counted over the whole batch.  dir -1 turns back.
template <int P>
__device__ __forceinline__ Slot<P> make_slot(const Rotate& p, int group, int sub, int l, float dir) {
  Slot<P> s;
  const int g = group * (32 / p.lanes) + sub;
  s.live = g < p.B * p.T && 2 * P * l < p.D;
  s.b = s.live ? g / p.T : 0;
  s.t = s.live ? g - s.b * p.T : 0;
  const int nat = p.m.pos(s.t), j0 = P * l;
  s.from = p.natural_in ? nat : s.t;
  const bool turned = s.live && j0 < p.rot / 2;
  const int pos = turned && p.positions ? p.positions[g] : nat;
#pragma unroll
  for (int i = 0; i < P; ++i) {
    s.co[i] = 1.f;
    s.si[i] = 0.f;
    if (turned) {
      const uint64_t at = (uint64_t)(int64_t)pos * turns_of(p.inv_freq[j0 + i]);
      sin_cos(at, &s.si[i], &s.co[i]);
      s.si[i] *= dir;
    }
  }
  return s;
}

// The rows of a warp's next K heads, in shared memory: [head % K][vector][piece][lane], a vector's
// P channels in pieces of 16 bytes (8: four bf16).  V vectors a row: two of the row itself, in the
// backward pass with the norm two of x.
template <typename E, int P, int V>
struct Ring {
  static constexpr int kBytes = P * (int)sizeof(E), kPiece = kBytes < 16 ? kBytes : 16;
  static constexpr int kPieces = kBytes / kPiece;
  static constexpr int K = V * kBytes > 64 ? 2 : 4;  // heads
  static constexpr int kWarpBytes = K * V * kBytes * 32;

  uint32_t base;  // of this lane
  __device__ __forceinline__ uint32_t at(int head, int v) const {
    return base + ((head & (K - 1)) * V + v) * (kBytes * 32);
  }
  __device__ __forceinline__ void fetch(int head, int v, const E* src) const {
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const char* from = reinterpret_cast<const char*>(src) + i * kPiece;
      if constexpr (kPiece == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at(head, v) + i * 512), "l"(from) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at(head, v)), "l"(from) : "memory");
    }
  }
  __device__ __forceinline__ void commit() const { asm volatile("cp.async.commit_group;" ::: "memory"); }
  // all but the last K - 1 heads have come
  __device__ __forceinline__ void wait() const { asm volatile("cp.async.wait_group %0;" ::"n"(K - 1) : "memory"); }
  __device__ __forceinline__ Vec<E, P> get(int head, int v) const {
    Vec<E, P> x;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if constexpr (kPiece == 16)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(word(x, 4 * i)), "=r"(word(x, 4 * i + 1)), "=r"(word(x, 4 * i + 2)), "=r"(word(x, 4 * i + 3))
                     : "r"(at(head, v) + i * 512)
                     : "memory");
      else
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(word(x, 0)), "=r"(word(x, 1)) : "r"(at(head, v)) : "memory");
    }
    return x;
  }
  __device__ __forceinline__ void clear() const {
#pragma unroll
    for (int i = 0; i < K * V * kPieces; ++i)
#pragma unroll
      for (int j = 0; j < kPiece / 4; ++j)
        asm volatile("st.shared.b32 [%0], %1;" ::"r"(base + i * (kPiece * 32) + 4 * j), "r"(0) : "memory");
  }
  static __device__ __forceinline__ uint32_t& word(Vec<E, P>& x, int i) {
    return reinterpret_cast<uint32_t*>(x.w)[i];
  }
};

// Rows of all heads (queries, keys, values in this order) by number.
template <typename E>
__device__ __forceinline__ E* head_row(const Rotate& p, const RowView (&v)[3], int b, int t, int head) {
  const int j = head < p.Hq ? 0 : head < p.Hq + p.Hkv ? 1 : 2;
  const int h = j == 0 ? head : j == 1 ? head - p.Hq : head - p.Hq - p.Hkv;
  const RowView& x = v[j];
  return static_cast<E*>(x.p) + b * x.sb + h * x.sh + t * x.st;
}

// (two pairs an instruction: the backward pass with the norm is close to issue-bound without)
template <int P>
__device__ __forceinline__ float2 two(const float (&x)[P], int i) {
  return make_float2(x[i], x[i + 1]);
}
template <int P>
__device__ __forceinline__ void put(float (&x)[P], int i, float2 v) {
  x[i] = v.x, x[i + 1] = v.y;
}

template <int P>
__device__ __forceinline__ void turn(const Slot<P>& s, float (&a)[P], float (&b)[P]) {
#pragma unroll
  for (int i = 0; i < P; i += 2) {
    const float2 x = two(a, i), y = two(b, i), co = two(s.co, i), si = two(s.si, i);
    const float2 ny = make_float2(-y.x, -y.y);
    put(a, i, fma2(x, co, mul2(ny, si)));
    put(b, i, fma2(x, si, mul2(y, co)));
  }
}

template <bool NEAR, typename E, int P>
__device__ __forceinline__ void load_weights(const Rotate& p, const void* w, int c0, int c1, float (&a)[P],
                                             float (&b)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) a[i] = b[i] = 1.f;
  if (w && c0 < p.D) {
    Vec<E, P> x, y;
    x.load(static_cast<const E*>(w) + c0);
    y.load(static_cast<const E*>(w) + c1);
    to_pairs<NEAR>(x, y, a, b);
  }
}

// An item is a group of slots and a part of all heads; parts of a group lie far apart, so that
// warps of a block write neighbouring slots of the same heads.
__device__ __forceinline__ void item_of(const Rotate& p, int item, int heads, int* group, int* h0, int* h1) {
  const int part = item / p.groups;
  *group = item - part * p.groups;
  *h0 = (int)((int64_t)heads * part / p.splits);
  *h1 = (int)((int64_t)heads * (part + 1) / p.splits);
}

template <typename E, bool NEAR, bool NORM, int P>
__global__ void __launch_bounds__(kThreads, sizeof(E) == 2 ? 3 : 2) fwd_kernel(const Rotate p) {
  extern __shared__ __align__(16) uint8_t smem[];
  using R = Ring<E, P, 2>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & (p.lanes - 1);
  const int item = blockIdx.x * kWarps + warp;
  if (item >= p.groups * p.splits) return;
  const R ring{smem_u32(smem) + warp * R::kWarpBytes + lane * R::kPiece};
  const int heads = p.Hq + p.Hkv + (p.in[2].p ? p.Hkv : 0);
  int group, h0, h1;
  item_of(p, item, heads, &group, &h0, &h1);
  const Slot<P> s = make_slot<P>(p, group, lane / p.lanes, l, 1.f);
  int c0, c1;
  lane_channels<NEAR, P>(p, l, &c0, &c1);
  if (!s.live) ring.clear();
  auto fetch = [&](int h) {
    if (s.live && h < h1) {
      const E* row = head_row<const E>(p, p.in, s.b, s.from, h);
      ring.fetch(h, 0, row + c0);
      ring.fetch(h, 1, row + c1);
    }
    ring.commit();
  };
#pragma unroll
  for (int u = 0; u < R::K; ++u) fetch(h0 + u);
  float wa[P], wb[P];
  for (int h = h0; h < h1; ++h) {
    if constexpr (NORM)
      if (h == h0 || h == p.Hq) load_weights<NEAR, E, P>(p, h < p.Hq ? p.w[0] : p.w[1], c0, c1, wa, wb);
    ring.wait();
    float a[P], b[P];
    to_pairs<NEAR>(ring.get(h, 0), ring.get(h, 1), a, b);
    fetch(h + R::K);
    if (h < p.Hq + p.Hkv) {
      if constexpr (NORM) {
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < P; i += 2) sum = fma2(two(a, i), two(a, i), fma2(two(b, i), two(b, i), sum));
        const float rs = rsqrtf(row_sum(sum.x + sum.y, p.lanes) * p.inv_d + p.eps);
        const float2 rs2 = make_float2(rs, rs);
#pragma unroll
        for (int i = 0; i < P; i += 2) {
          put(a, i, mul2(two(a, i), mul2(rs2, two(wa, i))));
          put(b, i, mul2(two(b, i), mul2(rs2, two(wb, i))));
        }
      }
      turn(s, a, b);
    }
    if (s.live) store_pairs<NEAR>(head_row<E>(p, p.out, s.b, s.t, h), c0, c1, a, b);
  }
}

// Backward: dY turned back (in: attention's side), with the norm also x.  Blocks are persistent and
// a warp takes an equal stretch of all (group, head) pairs, a group's heads first; each block
// keeps its share of the weights' gradients in registers and leaves one row of sums in the
// workspace; a second, small kernel adds the rows in order.
template <typename E, bool NEAR, bool NORM, int P>
__global__ void __launch_bounds__(kThreads, 2) bwd_kernel(const Rotate p) {
  extern __shared__ __align__(16) uint8_t smem[];
  using R = Ring<E, P, NORM ? 4 : 2>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & (p.lanes - 1), sub = lane / p.lanes;
  const R ring{smem_u32(smem) + warp * R::kWarpBytes + lane * R::kPiece};
  const int heads = p.Hq + p.Hkv + (p.in[2].p ? p.Hkv : 0);
  int c0, c1;
  lane_channels<NEAR, P>(p, l, &c0, &c1);
  // this thread's share of the weights' gradients, queries then keys: in shared memory, so that
  // only one tensor's is in registers at a time
  float4* const mine = reinterpret_cast<float4*>(smem + kWarps * R::kWarpBytes) + threadIdx.x;
  constexpr int kQuads = P / 2;  // 2 P numbers
  if constexpr (NORM) {
#pragma unroll
    for (int i = 0; i < 2 * kQuads; ++i) mine[i * kThreads] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  const int64_t pairs = (int64_t)p.groups * heads, warps = (int64_t)gridDim.x * kWarps;
  const int64_t w0 = (int64_t)blockIdx.x * kWarps + warp, end = pairs * (w0 + 1) / warps;
  for (int64_t at = pairs * w0 / warps; at < end;) {
    const int group = (int)(at / heads), h0 = (int)(at - (int64_t)group * heads);
    const int h1 = (int)min((int64_t)heads, h0 + (end - at));
    at += h1 - h0;
    const Slot<P> s = make_slot<P>(p, group, sub, l, -1.f);
    if (!s.live) ring.clear();
    auto fetch = [&](int h) {
      if (s.live && h < h1) {
        const E* row = head_row<const E>(p, p.in, s.b, s.t, h);
        ring.fetch(h, 0, row + c0);
        ring.fetch(h, 1, row + c1);
        if constexpr (NORM)
          if (h < p.Hq + p.Hkv) {
            const E* x = head_row<const E>(p, p.x, s.b, s.from, h);
            ring.fetch(h, 2, x + c0);
            ring.fetch(h, 3, x + c1);
          }
      }
      ring.commit();
    };
#pragma unroll
    for (int u = 0; u < R::K; ++u) fetch(h0 + u);
    auto tensor = [&](int lo, int hi, auto move, int j) {
      constexpr bool N = NORM && !decltype(move)::value;
      if (lo >= hi) return;
      float wa[P], wb[P], da[P], db[P];
      if constexpr (N) {
        load_weights<NEAR, E, P>(p, p.w[j], c0, c1, wa, wb);
#pragma unroll
        for (int i = 0; i < P; ++i) da[i] = db[i] = 0.f;
      }
      for (int h = lo; h < hi; ++h) {
        ring.wait();
        float a[P], b[P], xa[P], xb[P];
        to_pairs<NEAR>(ring.get(h, 0), ring.get(h, 1), a, b);
        if constexpr (N) to_pairs<NEAR>(ring.get(h, 2), ring.get(h, 3), xa, xb);
        fetch(h + R::K);
        if constexpr (!decltype(move)::value) turn(s, a, b);
        if constexpr (N) {
          float2 sum = make_float2(0.f, 0.f), dot = sum;
#pragma unroll
          for (int i = 0; i < P; i += 2) {
            const float2 x = two(xa, i), y = two(xb, i);
            sum = fma2(x, x, fma2(y, y, sum));
            dot = fma2(mul2(two(a, i), two(wa, i)), x, fma2(mul2(two(b, i), two(wb, i)), y, dot));
          }
          // with r = 1 / sqrt(..): dw += g (r x),  dx = r w g - x (r^3 mean(w g x))
          // (lanes without a row add nothing, also where eps is 0)
          const float all = row_sum(sum.x + sum.y, p.lanes) * p.inv_d + p.eps;
          const float rs = s.live ? rsqrtf(all) : 0.f;
          const float m = -row_sum(dot.x + dot.y, p.lanes) * p.inv_d * rs * rs;
          const float2 rs2 = make_float2(rs, rs), m2 = make_float2(m, m);
#pragma unroll
          for (int i = 0; i < P; i += 2) {
            const float2 x = mul2(two(xa, i), rs2), y = mul2(two(xb, i), rs2);
            const float2 ga = two(a, i), gb = two(b, i);
            put(da, i, fma2(ga, x, two(da, i)));
            put(db, i, fma2(gb, y, two(db, i)));
            put(a, i, fma2(mul2(ga, two(wa, i)), rs2, mul2(x, m2)));
            put(b, i, fma2(mul2(gb, two(wb, i)), rs2, mul2(y, m2)));
          }
        }
        if (s.live) store_pairs<NEAR>(head_row<E>(p, p.out, s.b, s.from, h), c0, c1, a, b);
      }
      if constexpr (N) {
#pragma unroll
        for (int i = 0; i < kQuads; ++i) {
          float4* const at = mine + (j * kQuads + i) * kThreads;
          const float* d = i < P / 4 ? da + 4 * i : db + 4 * i - P;
          float4 v = *at;
          v.x += d[0], v.y += d[1], v.z += d[2], v.w += d[3];
          *at = v;
        }
      }
    };
    tensor(h0, min(h1, p.Hq), std::false_type{}, 0);
    tensor(max(h0, p.Hq), min(h1, p.Hq + p.Hkv), std::false_type{}, 1);
    tensor(max(h0, p.Hq + p.Hkv), h1, std::true_type{}, 2);
  }
  if constexpr (NORM) {
    // the lanes of a warp that hold the same channels, then the warps in order; the ring is done
    griddep_launch_dependents();
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    float* part = reinterpret_cast<float*>(smem);  // [warp][2][D]
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int q = 0; q < kQuads; ++q) {
        const float4 d = mine[(j * kQuads + q) * kThreads];
        const float x[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = 4 * q + k;
          float v = x[k];
          for (int o = p.lanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
          const int c = NEAR ? c0 + 2 * (i % P) + (i >= P) : i < P ? c0 + i : c1 + i - P;
          if (sub == 0 && c < p.D) part[(warp * 2 + j) * p.D + c] = v;
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.D; i += kThreads) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += part[w * 2 * p.D + i];
      p.sums[(int64_t)blockIdx.x * 2 * p.D + i] = v;
    }
  }
}

// dw[j][c] = the sum of n rows of 2 D numbers.  A block takes eight columns, a thread every 128th
// row of one, then a warp its threads of a column and the first warp the warps, in order.
__global__ void __launch_bounds__(1024) sum_kernel(const float* sums, int n, int D, float* dq,
                                                   float* dk) {
  __shared__ float part[32][8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 8 + (lane & 7);
  float v = 0.f;
  griddep_wait();
#pragma unroll 4
  for (int r = threadIdx.x >> 3; r < n; r += 128) v += sums[(int64_t)r * 2 * D + c];
  v += __shfl_xor_sync(0xffffffffu, v, 8);
  v += __shfl_xor_sync(0xffffffffu, v, 16);
  if (lane < 8) part[warp][lane] = v;
  __syncthreads();
  if (threadIdx.x < 8) {
    v = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) v += part[w][lane];
    float* out = c < D ? dq : dk;
    if (out) out[c < D ? c : c - D] = v;
  }
}

template <auto KERN>
static cudaError_t launch_kernel(const Rotate& p, int grid, int bytes, cudaStream_t st) {
  if (bytes > 48 * 1024) {  // (one size a kernel)
    static ReadyDevices ready;
    const cudaError_t e =
        ready.once([&] { return cudaFuncSetAttribute(KERN, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes); });
    if (e != cudaSuccess) return e;
  }
  KERN<<<grid, kThreads, bytes, st>>>(p);
  return cudaGetLastError();
}
template <typename E, bool NEAR, bool NORM, int P>
static cudaError_t launch_one(const Rotate& p, int grid, bool backward, cudaStream_t st) {
  // (the ring's space, at least 16 KB with the norm, later takes 8 KB of sums)
  constexpr int V = NORM ? 4 : 2, kSums = NORM ? 2 * 2 * P * kThreads * 4 : 0;
  return backward ? launch_kernel<bwd_kernel<E, NEAR, NORM, P>>(p, grid, kWarps * Ring<E, P, V>::kWarpBytes + kSums, st)
                  : launch_kernel<fwd_kernel<E, NEAR, NORM, P>>(p, grid, kWarps * Ring<E, P, 2>::kWarpBytes, st);
}
template <typename E, bool NEAR>
static cudaError_t launch_pairs(const Rotate& p, int grid, bool backward, cudaStream_t st) {
  if constexpr (sizeof(E) == 2)
    if (p.P == 8) return p.norm ? launch_one<E, NEAR, true, 8>(p, grid, backward, st) : launch_one<E, NEAR, false, 8>(p, grid, backward, st);
  return p.norm ? launch_one<E, NEAR, true, 4>(p, grid, backward, st) : launch_one<E, NEAR, false, 4>(p, grid, backward, st);
}
static cudaError_t launch(const Rotate& p, int grid, bool backward, cudaStream_t st) {
  timing_begin(backward ? "rotate_bwd" : "rotate_fwd", st);
  const cudaError_t e = p.bf16 ? p.near ? launch_pairs<__nv_bfloat16, true>(p, grid, backward, st)
                                        : launch_pairs<__nv_bfloat16, false>(p, grid, backward, st)
                        : p.near ? launch_pairs<float, true>(p, grid, backward, st)
                                 : launch_pairs<float, false>(p, grid, backward, st);
  timing_end(st);
  return e;
}

// Pairs a lane, groups of slots, and parts that the heads are cut into: one part shares a slot's
// angles among all its heads, but a decoding step's few tokens want every SM, down to a head a
// warp.  Eight pairs a lane cost half the warps and shuffles a row, but twice the angles one after
// the other, and half the warps are there to wait for memory: they pay from 8 warps' rows (of four pairs
// a lane) a warp on, in the backward pass from 4.  Four and eight, us, forward / backward, 40 heads of
// 128: 64 tokens 4.3 / 7.2 and 4.8 / 9.1; 975 12.7 / 14.0 and 16.2 / 15.1; 2000 16.6 / 20.6 and 18.9 /
// 19.5; 3250 21.3 / 28.3 and 21.6 / 24.7; 5000 28.5 / 40.5 and 26.9 / 35.0.  48 heads of 64, half the
// lanes a row: 1666 12.9 / 14.4 and 16.4 / 15.6; 3333 16.2 / 20.2 and 18.7 / 19.9; 6666 23.7 / 32.6
// and 23.4 / 29.3.
static int cut(Rotate* p, bool backward) {
  const int heads = p->Hq + p->Hkv + (p->in[2].p ? p->Hkv : 0);
  const int64_t want = (int64_t)kSms * 64;  // warps
  auto set_pairs = [&](int P) {
    p->P = P;
    p->lanes = 1;
    while (p->lanes * 2 * P < p->D) p->lanes *= 2;
  };
  set_pairs(4);
  if (p->bf16 && p->D % 16 == 0 && p->rot % 16 == 0 &&
      (int64_t)p->B * p->T * heads * p->lanes / 32 > (backward ? 4 : 8) * want)
    set_pairs(8);
  p->inv_d = 1.f / p->D;
  const int per = 32 / p->lanes;
  p->groups = (p->B * p->T + per - 1) / per;
  int64_t splits = (want + p->groups - 1) / p->groups;
  if (splits > heads) splits = heads;
  p->splits = (int)splits;
  return (int)(((int64_t)p->groups * splits + kWarps - 1) / kWarps);  // blocks
}

}  // namespace rotate

using namespace rotate;

size_t rotate_bwd_workspace(int D, int norm) {
  return norm ? (size_t)kBwdBlocks * 2 * D * sizeof(float) : 16;
}

cudaError_t launch_rotate_fwd(Rotate p, cudaStream_t st) {
  const int grid = cut(&p, false);
  return launch(p, grid, false, st);
}

cudaError_t launch_rotate_bwd(Rotate p, float* dqw, float* dkw, cudaStream_t st) {
  // two blocks an SM, but no more warps than there are heads of groups
  const int blocks = cut(&p, true), grid = blocks < kBwdBlocks ? blocks : kBwdBlocks;
  cudaError_t e = launch(p, grid, true, st);
  if (e != cudaSuccess || !p.norm || (!dqw && !dkw)) return e;
  timing_begin("rotate_bwd_sum", st);
  // (started while the blocks before it finish; it waits for them before it reads)
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * p.D / 8);
  cfg.blockDim = dim3(1024);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, sum_kernel, (const float*)p.sums, grid, p.D, dqw, dkw);
  timing_end(st);
  return e;
}

}  // namespace cpattn
