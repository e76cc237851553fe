// What stands between a layer's projections and its attention, in one pass over the rows:
// RMS norm of each head of the queries and keys, rotation by position, the move into the
// attention's token order; values move along.  And its backward pass.
//
// A row of D channels belongs to D / 8 lanes (rounded up to a power of two: 16 at D 128, so a
// warp holds two rows).  Lane l owns pairs 4l .. 4l+3 of the rotation, as two vectors of four
// channels: (4l .., rot/2 + 4l ..) when pairs lie half a rotation apart, else eight channels
// in a row.  So a pair never crosses lanes, the only exchange is the norm's sum (four shuffles
// at D 128), and each row is read and written once.
//
// A block takes `tile` consecutive slots and all (or, with few tokens, some) of their heads:
// the angles of a slot are the same in every head, so their cosines and sines are computed
// once a block, into shared memory.  The angle p f is formed in float64 and reduced to a
// fraction of a turn there: at position 10^5 a float32 product alone is off by 2^-8 of a
// radian.
//
// Bound by memory: 32 (bf16) to 64 (float32) bytes a lane and row against some 70 instructions.
#include "layer.cuh"

namespace cpattn {
namespace rotate {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTile = 16;
constexpr int kMaxPairs = 64;

struct V4 {
  float v[4];
};

__device__ __forceinline__ V4 load4(const __nv_bfloat16* p) {
  const uint2 r = __ldcs(reinterpret_cast<const uint2*>(p));
  V4 x;
  x.v[0] = __uint_as_float(r.x << 16);
  x.v[1] = __uint_as_float(r.x & 0xFFFF0000u);
  x.v[2] = __uint_as_float(r.y << 16);
  x.v[3] = __uint_as_float(r.y & 0xFFFF0000u);
  return x;
}
__device__ __forceinline__ V4 load4(const float* p) {
  const float4 r = __ldcs(reinterpret_cast<const float4*>(p));
  return V4{{r.x, r.y, r.z, r.w}};
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float* x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
}
__device__ __forceinline__ void store4(float* p, const float* x) {
  *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
}

// Eight channels of a lane as (first, second) of its four pairs, and back.
template <bool NEAR>
__device__ __forceinline__ void to_pairs(const V4& x, const V4& y, float (&a)[4], float (&b)[4]) {
  if constexpr (NEAR) {
    a[0] = x.v[0], b[0] = x.v[1], a[1] = x.v[2], b[1] = x.v[3];
    a[2] = y.v[0], b[2] = y.v[1], a[3] = y.v[2], b[3] = y.v[3];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = x.v[i], b[i] = y.v[i];
  }
}
template <bool NEAR, typename E>
__device__ __forceinline__ void store_pairs(E* row, int c0, int c1, const float (&a)[4],
                                            const float (&b)[4]) {
  if constexpr (NEAR) {
    const float x[4] = {a[0], b[0], a[1], b[1]}, y[4] = {a[2], b[2], a[3], b[3]};
    store4(row + c0, x);
    store4(row + c1, y);
  } else {
    store4(row + c0, a);
    store4(row + c1, b);
  }
}

__device__ __forceinline__ float row_sum(float s, int lanes) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
    if (o < lanes) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

// Channels of a lane: two vectors of four, at c0 and c1.  Past the rotated pairs a lane's
// eight channels follow each other in either pairing, and the table holds no turn (1, 0).
template <bool NEAR>
__device__ __forceinline__ void lane_channels(const Rotate& p, int l, int* c0, int* c1) {
  *c0 = 8 * l;
  *c1 = 8 * l + 4;
  if (!NEAR && 4 * l < p.rot / 2) {
    *c0 = 4 * l;
    *c1 = 4 * l + p.rot / 2;
  }
}
// (past the rotated pairs the two vectors hold channels as they come: pairs do not matter)

struct __align__(16) Shared {
  float2 cs[kMaxTile][kMaxPairs];  // cos, sin of every pair of every slot of the tile
  int from[kMaxTile];              // token of the projection's side
};

// Fills the tile's table.  tile slots from t0 on, of batch row b.
__device__ __forceinline__ void fill_table(const Rotate& p, int b, int t0, int nt, float dir,
                                           Shared* s) {
  const int pairs = p.D / 2;
  for (int i = threadIdx.x; i < nt * pairs; i += kThreads) {
    const int t = i / pairs, j = i - t * pairs;
    float2 v = make_float2(1.f, 0.f);
    if (j < p.rot / 2) {
      const int slot = t0 + t;
      const int pos = p.positions ? p.positions[(int64_t)b * p.T + slot] : p.m.pos(slot);
      const double turns = (double)pos * (p.inv_freq[j] * 0.15915494309189533577);  // 1 / (2 pi)
      const float f = (float)(turns - rint(turns));
      sincospif(2.f * f, &v.y, &v.x);
      v.y *= dir;
    }
    s->cs[t][j] = v;
  }
  for (int t = threadIdx.x; t < nt; t += kThreads)
    s->from[t] = p.natural_in ? p.m.pos(t0 + t) : t0 + t;
}

template <typename E>
__device__ __forceinline__ E* row_ptr(const RowView& v, int b, int h, int t) {
  return static_cast<E*>(v.p) + b * v.sb + h * v.sh + t * v.st;
}

// Row r of the block's rows, heads outermost: head and token.  Whole tiles are a power of two.
__device__ __forceinline__ void split_row(const Rotate& p, int r, int nt, int* head, int* t) {
  if (nt == p.tile) *head = r >> p.tile_log2;
  else *head = r / nt;
  *t = r - *head * nt;
}

// The head'th of all heads: queries, keys, then values.
__device__ __forceinline__ int which(const Rotate& p, int head, int* h) {
  if (head < p.Hq) {
    *h = head;
    return 0;
  }
  if (head < p.Hq + p.Hkv) {
    *h = head - p.Hq;
    return 1;
  }
  *h = head - p.Hq - p.Hkv;
  return 2;
}

// Four rows a lane in flight: with 32 to 48 registers of loads outstanding and six blocks an SM
// some 48 KB are under way, what 7 TB/s at a microsecond's latency takes.
constexpr int kRows = 4;

template <typename E, bool NEAR, bool NORM>
__global__ void __launch_bounds__(kThreads) fwd_kernel(const Rotate p) {
  __shared__ Shared s;
  const int tiles = (p.T + p.tile - 1) / p.tile;
  const int b = blockIdx.x / tiles, t0 = (blockIdx.x - b * tiles) * p.tile;
  const int nt = min(p.tile, p.T - t0);
  fill_table(p, b, t0, nt, 1.f, &s);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane & (p.lanes - 1), sub = lane / p.lanes, per_warp = 32 / p.lanes;
  const bool live = 8 * l < p.D;
  int c0, c1;
  lane_channels<NEAR>(p, l, &c0, &c1);
  float wa[2][4], wb[2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    V4 x{{1.f, 1.f, 1.f, 1.f}}, y = x;
    if (NORM && p.w[j] && live) {
      x = load4(static_cast<const E*>(p.w[j]) + c0);
      y = load4(static_cast<const E*>(p.w[j]) + c1);
    }
    to_pairs<NEAR>(x, y, wa[j], wb[j]);
  }
  const int heads = p.Hq + p.Hkv + (p.in[2].p ? p.Hkv : 0);
  const int h0 = (int)((int64_t)heads * blockIdx.y / gridDim.y);
  const int h1 = (int)((int64_t)heads * (blockIdx.y + 1) / gridDim.y);
  const int rows = (h1 - h0) * nt, step = kWarps * per_warp;
  __syncthreads();
  for (int base = warp * per_warp + sub; __any_sync(0xffffffffu, base < rows); base += kRows * step) {
    V4 x[kRows], y[kRows];
    int kind[kRows], hh[kRows], tt[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      const int r = base + u * step;
      kind[u] = -1;
      hh[u] = tt[u] = 0;
      x[u] = y[u] = V4{{0.f, 0.f, 0.f, 0.f}};
      if (r < rows && live) {
        int head;
        split_row(p, r, nt, &head, &tt[u]);
        kind[u] = which(p, h0 + head, &hh[u]);
        const E* row = row_ptr<const E>(p.in[kind[u]], b, hh[u], s.from[tt[u]]);
        x[u] = load4(row + c0);
        y[u] = load4(row + c1);
      }
    }
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
      float a[4], c[4];
      to_pairs<NEAR>(x[u], y[u], a, c);
      if (NORM) {
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) sum = fmaf(a[i], a[i], fmaf(c[i], c[i], sum));
        const float rs = rsqrtf(row_sum(sum, p.lanes) * p.inv_d + p.eps);
        if (kind[u] < 2) {
          const bool k = kind[u] == 1;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            a[i] *= rs * (k ? wa[1][i] : wa[0][i]);
            c[i] *= rs * (k ? wb[1][i] : wb[0][i]);
          }
        }
      }
      if (kind[u] < 0) continue;
      if (kind[u] < 2) {
        const float4* cs = reinterpret_cast<const float4*>(&s.cs[tt[u]][4 * l]);
        const float4 t01 = cs[0], t23 = cs[1];
        const float co[4] = {t01.x, t01.z, t23.x, t23.z}, si[4] = {t01.y, t01.w, t23.y, t23.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float y0 = a[i] * co[i] - c[i] * si[i];
          c[i] = a[i] * si[i] + c[i] * co[i];
          a[i] = y0;
        }
      }
      E* out = row_ptr<E>(p.out[kind[u]], b, hh[u], t0 + tt[u]);
      store_pairs<NEAR>(out, c0, c1, a, c);
    }
  }
}

// The backward pass of a row: dY turned back (in: attention's side), with the norm also x.
// Blocks are persistent: each keeps its share of the weights' gradients in registers (eight
// channels a lane, queries and keys apart) and leaves one row of sums in the workspace; a
// second, small kernel adds the rows in order.
constexpr int kBwdRows = 2;  // rows a lane in flight, two loads each with the norm

template <typename E, bool NEAR, bool NORM>
__global__ void __launch_bounds__(kThreads) bwd_kernel(const Rotate p) {
  __shared__ Shared s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int l = lane & (p.lanes - 1), sub = lane / p.lanes, per_warp = 32 / p.lanes;
  const bool live = 8 * l < p.D;
  int c0, c1;
  lane_channels<NEAR>(p, l, &c0, &c1);
  float wa[2][4], wb[2][4], da[2][4], db[2][4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    V4 x{{1.f, 1.f, 1.f, 1.f}}, y = x;
    if (NORM && p.w[j] && live) {
      x = load4(static_cast<const E*>(p.w[j]) + c0);
      y = load4(static_cast<const E*>(p.w[j]) + c1);
    }
    to_pairs<NEAR>(x, y, wa[j], wb[j]);
#pragma unroll
    for (int i = 0; i < 4; ++i) da[j][i] = db[j][i] = 0.f;
  }
  const int heads = p.Hq + p.Hkv + (p.in[2].p ? p.Hkv : 0);
  const int tiles = (p.T + p.tile - 1) / p.tile, step = kWarps * per_warp;
  const int n_items = p.B * tiles * p.splits;
  for (int item = blockIdx.x; item < n_items; item += gridDim.x) {
    const int tl = item / p.splits, part = item - tl * p.splits;
    const int b = tl / tiles, t0 = (tl - b * tiles) * p.tile;
    const int nt = min(p.tile, p.T - t0);
    const int h0 = (int)((int64_t)heads * part / p.splits);
    const int h1 = (int)((int64_t)heads * (part + 1) / p.splits);
    const int rows = (h1 - h0) * nt;
    __syncthreads();  // the last item's table has been read
    fill_table(p, b, t0, nt, -1.f, &s);
    __syncthreads();
    for (int base = warp * per_warp + sub; __any_sync(0xffffffffu, base < rows);
         base += kBwdRows * step) {
      V4 x[kBwdRows], y[kBwdRows], gx[kBwdRows], gy[kBwdRows];
      int kind[kBwdRows], hh[kBwdRows], tt[kBwdRows];
#pragma unroll
      for (int u = 0; u < kBwdRows; ++u) {
        const int r = base + u * step;
        kind[u] = -1;
        hh[u] = tt[u] = 0;
        x[u] = y[u] = gx[u] = gy[u] = V4{{0.f, 0.f, 0.f, 0.f}};
        if (r < rows && live) {
          int head;
          split_row(p, r, nt, &head, &tt[u]);
          kind[u] = which(p, h0 + head, &hh[u]);
          const E* row = row_ptr<const E>(p.in[kind[u]], b, hh[u], t0 + tt[u]);
          gx[u] = load4(row + c0);
          gy[u] = load4(row + c1);
          if (NORM && kind[u] < 2) {
            const E* xr = row_ptr<const E>(p.x[kind[u]], b, hh[u], s.from[tt[u]]);
            x[u] = load4(xr + c0);
            y[u] = load4(xr + c1);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < kBwdRows; ++u) {
        float ga[4], gb[4];
        to_pairs<NEAR>(gx[u], gy[u], ga, gb);
        if (kind[u] == 0 || kind[u] == 1) {
          const float4* cs = reinterpret_cast<const float4*>(&s.cs[tt[u]][4 * l]);
          const float4 t01 = cs[0], t23 = cs[1];
          const float co[4] = {t01.x, t01.z, t23.x, t23.z}, si[4] = {t01.y, t01.w, t23.y, t23.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float y0 = ga[i] * co[i] - gb[i] * si[i];
            gb[i] = ga[i] * si[i] + gb[i] * co[i];
            ga[i] = y0;
          }
        }
        if (NORM) {
          float xa[4], xb[4], sum = 0.f, dot = 0.f;
          to_pairs<NEAR>(x[u], y[u], xa, xb);
          const bool k = kind[u] == 1;
#pragma unroll
          for (int i = 0; i < 4; ++i) sum = fmaf(xa[i], xa[i], fmaf(xb[i], xb[i], sum));
          const float rs = rsqrtf(row_sum(sum, p.lanes) * p.inv_d + p.eps);
          float na[4], nb[4], ha[4], hb[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            na[i] = xa[i] * rs;
            nb[i] = xb[i] * rs;
            ha[i] = ga[i] * (k ? wa[1][i] : wa[0][i]);
            hb[i] = gb[i] * (k ? wb[1][i] : wb[0][i]);
            dot = fmaf(ha[i], na[i], fmaf(hb[i], nb[i], dot));
          }
          dot = row_sum(dot, p.lanes) * p.inv_d;
          if (kind[u] == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) da[0][i] += ga[i] * na[i], db[0][i] += gb[i] * nb[i];
          } else if (kind[u] == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) da[1][i] += ga[i] * na[i], db[1][i] += gb[i] * nb[i];
          }
          if (kind[u] == 0 || kind[u] == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              ga[i] = rs * (ha[i] - na[i] * dot);
              gb[i] = rs * (hb[i] - nb[i] * dot);
            }
          }
        }
        if (kind[u] < 0) continue;
        E* out = row_ptr<E>(p.out[kind[u]], b, hh[u], s.from[tt[u]]);
        store_pairs<NEAR>(out, c0, c1, ga, gb);
      }
    }
  }
  if constexpr (NORM) {
    // the lanes of a warp that hold the same channels, then the warps in order
    __shared__ float part[kWarps][2][128];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v = i < 4 ? da[j][i & 3] : db[j][i & 3];
        for (int o = p.lanes; o < 32; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        const int c = NEAR ? (i < 4 ? 8 * l + 2 * i : 8 * l + 2 * (i - 4) + 1)
                           : (i < 4 ? c0 + i : c1 + i - 4);
        if (sub == 0 && live) part[warp][j][c] = v;
      }
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * p.D; i += kThreads) {
      const int j = i / p.D, c = i - j * p.D;
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) v += part[w][j][c];
      p.sums[(int64_t)blockIdx.x * 2 * p.D + i] = v;
    }
  }
}

// dw[j][c] = the sum of n rows of 2 D numbers; a block takes 32 columns, its warps every 32nd
// row, then the warps in order.
__global__ void __launch_bounds__(1024) sum_kernel(const float* sums, int n, int D, float* dq,
                                                   float* dk) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float v = 0.f;
  if (c < 2 * D)
    for (int r = warp; r < n; r += 32) v += sums[(int64_t)r * 2 * D + c];
  part[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && c < 2 * D) {
    v = 0.f;
#pragma unroll
    for (int w = 0; w < 32; ++w) v += part[w][lane];
    float* out = c < D ? dq : dk;
    if (out) out[c < D ? c : c - D] = v;
  }
}

template <typename E, bool NEAR>
static void launch_fwd(const Rotate& p, dim3 grid, cudaStream_t st) {
  if (p.norm) fwd_kernel<E, NEAR, true><<<grid, kThreads, 0, st>>>(p);
  else fwd_kernel<E, NEAR, false><<<grid, kThreads, 0, st>>>(p);
}
template <typename E, bool NEAR>
static void launch_bwd(const Rotate& p, int grid, cudaStream_t st) {
  if (p.norm) bwd_kernel<E, NEAR, true><<<grid, kThreads, 0, st>>>(p);
  else bwd_kernel<E, NEAR, false><<<grid, kThreads, 0, st>>>(p);
}

// Slots a block takes, and parts that the heads are cut into: 16 slots share what a block does
// once, but a decoding step's few tokens want every SM.
static void cut(Rotate* p) {
  p->lanes = 1;
  while (p->lanes * 8 < p->D) p->lanes *= 2;
  p->inv_d = 1.f / p->D;
  const int64_t tokens = (int64_t)p->B * p->T;
  p->tile = kMaxTile;
  while (p->tile > 1 && (tokens + p->tile - 1) / p->tile < 2 * kSms) p->tile /= 2;
  p->tile_log2 = 0;
  while ((1 << p->tile_log2) < p->tile) ++p->tile_log2;
  const int heads = p->Hq + p->Hkv + (p->in[2].p ? p->Hkv : 0);
  const int64_t blocks = (int64_t)p->B * ((p->T + p->tile - 1) / p->tile);
  const int rows_pass = kWarps * (32 / p->lanes);
  int64_t splits = blocks < 2 * kSms ? (2 * kSms + blocks - 1) / blocks : 1;
  const int64_t most = ((int64_t)heads * p->tile + rows_pass - 1) / rows_pass;
  if (splits > most) splits = most;
  if (splits > heads) splits = heads;
  p->splits = (int)splits;
}

}  // namespace rotate

using namespace rotate;

size_t rotate_bwd_workspace(int D, int norm) {
  return norm ? (size_t)kBwdBlocks * 2 * D * sizeof(float) : 16;
}

cudaError_t launch_rotate_fwd(Rotate p, cudaStream_t st) {
  cut(&p);
  const int64_t blocks = (int64_t)p.B * ((p.T + p.tile - 1) / p.tile);
  const dim3 grid((unsigned)blocks, (unsigned)p.splits);
  timing_begin("rotate_fwd", st);
  if (p.bf16) {
    if (p.near) launch_fwd<__nv_bfloat16, true>(p, grid, st);
    else launch_fwd<__nv_bfloat16, false>(p, grid, st);
  } else {
    if (p.near) launch_fwd<float, true>(p, grid, st);
    else launch_fwd<float, false>(p, grid, st);
  }
  const cudaError_t e = cudaGetLastError();
  timing_end(st);
  return e;
}

cudaError_t launch_rotate_bwd(Rotate p, float* dqw, float* dkw, cudaStream_t st) {
  cut(&p);
  const int64_t items = (int64_t)p.B * ((p.T + p.tile - 1) / p.tile) * p.splits;
  const int grid = (int)(items < kBwdBlocks ? items : kBwdBlocks);
  timing_begin("rotate_bwd", st);
  if (p.bf16) {
    if (p.near) launch_bwd<__nv_bfloat16, true>(p, grid, st);
    else launch_bwd<__nv_bfloat16, false>(p, grid, st);
  } else {
    if (p.near) launch_bwd<float, true>(p, grid, st);
    else launch_bwd<float, false>(p, grid, st);
  }
  cudaError_t e = cudaGetLastError();
  timing_end(st);
  if (e != cudaSuccess || !p.norm || (!dqw && !dkw)) return e;
  timing_begin("rotate_bwd_sum", st);
  sum_kernel<<<(2 * p.D + 31) / 32, 1024, 0, st>>>(p.sums, grid, p.D, dqw, dkw);
  e = cudaGetLastError();
  timing_end(st);
  return e;
}

}  // namespace cpattn
