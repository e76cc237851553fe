// Linear attention in float32 on the ordinary units: every type, head dimension and layout that
// linear_tc.cu does not take (float32 tensors, other head dimensions, zigzag chunks of fewer
// than 16 tokens).  The sweep, its runs and its direction are described in layer.cuh.
//
// A block takes one run of one sweep and head in chunks of 64 tokens: scores a b^T weighted by
// the decay into shared memory, then out = P c + r^.. (a M), then U = b^T c and M = r^n M + U, all as
// register tiles over shared memory.  M lives in registers (8 x 8 a thread at D 128) with a copy
// in shared memory as the operand of a M.  Head dimensions in between are padded with zeros to
// 64 or 128.  Bound by the float32 units, 4 D (D + 32) FLOP a token and head, and by how two warps
// a scheduler (a block fills an SM's shared memory) wait for each other's chains: 8192 tokens of 32
// heads at D 128 take 889 us, the units' part of it 332 (32 heads on 8 with gradients 2.2 ms); 1500
// tokens of 16 heads, 2 or 3 chunks a block, 99 (43).  With tiles fetched when they were needed, and
// not ahead, these took 1269, 3018 and 104 us; 16 warps with 4 x 4 tiles were slower, too (121).
#include "layer.cuh"

namespace cpattn {
namespace linsimt {

constexpr int kThreads = 256;
constexpr int C = kLinSimtChunk;

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 r = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(r.x << 16), __uint_as_float(r.x & 0xFFFF0000u),
                     __uint_as_float(r.y << 16), __uint_as_float(r.y & 0xFFFF0000u));
}
__device__ __forceinline__ void store4(float* p, float4 x) { *reinterpret_cast<float4*>(p) = x; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 x) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16(x.x, x.y), pack_bf16(x.z, x.w));
}

template <int DP>
struct Smem {
  static constexpr int kLd = DP + 4;   // row stride: eight rows meet eight bank groups
  static constexpr int kPLd = C + 4;
  static constexpr int kTile = C * kLd;
  static constexpr int kP = 4 * kTile;  // (four tiles)
  static constexpr int kM = kP + C * kPLd;
  static constexpr int kPow = kM + DP * kLd;
  static constexpr int kFloats = kPow + C + 2;
};

// Rows of n tokens from pos0 on, zeros behind them and behind D.  float32 comes by asynchronous
// copies, in flight until wait_tiles; bf16 is widened on its way.
template <typename E, int DP>
__device__ __forceinline__ void load_tile(const Linear& p, const void* t, int64_t head, int pos0, int n,
                                          float* dst) {
  constexpr int LD = Smem<DP>::kLd, V = DP / 4, kStep = kThreads / V;
  const int r0 = threadIdx.x / V, c = 4 * (threadIdx.x - r0 * V);
  const E* src = static_cast<const E*>(t) + head * p.T * p.D;
  if constexpr (sizeof(E) == 4) {
#pragma unroll
    for (int r = r0; r < C; r += kStep) {
      const bool there = r < n && c < p.D;
      const float* from = there ? src + (int64_t)p.m.slot(pos0 + r) * p.D + c : src;
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst + r * LD + c)), "l"(from),
                   "r"(there ? 16 : 0)
                   : "memory");
    }
  } else {
    float4 x[C / kStep];
#pragma unroll
    for (int i = 0; i < C / kStep; ++i) {
      const int r = r0 + i * kStep;
      x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < n && c < p.D) x[i] = load4(src + (int64_t)p.m.slot(pos0 + r) * p.D + c);
    }
#pragma unroll
    for (int i = 0; i < C / kStep; ++i) *reinterpret_cast<float4*>(dst + (r0 + i * kStep) * LD + c) = x[i];
  }
}
__device__ __forceinline__ void commit_tile() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// all but the last N groups have come
template <int N>
__device__ __forceinline__ void wait_tiles() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename E, int DP, bool SUM>
__global__ void __launch_bounds__(kThreads, 1) sweep_kernel(const __grid_constant__ Linear p) {
  using L = Smem<DP>;
  constexpr int LD = L::kLd, PL = L::kPLd, R = DP / 64;  // R: 4-wide tiles of DP a thread
  extern __shared__ __align__(16) float sm[];
  // tiles of a, b and c, and of the next chunk's a (SUM: b, c and the next b and c)
  float *sa = sm, *sb = sm + L::kTile, *sc = sm + 2 * L::kTile, *sx = sm + 3 * L::kTile;
  float *const sp = sm + L::kP, *const sM = sm + L::kM, *const pw = sm + L::kPow;
  const int runs = SUM ? p.segs - 1 : p.segs;  // the last run's own sum is nobody's start
  const int bh = blockIdx.x / runs, run = blockIdx.x - bh * runs;
  const LinSweep& w = SUM ? p.sum[blockIdx.y] : p.sweep[blockIdx.y];
  const int n_tok = lin_tokens(p, bh);
  const float ld = lin_decay(p, bh);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int b = bh / p.Hq, h = bh - b * p.Hq, late = w.back;
  const int64_t ha = (int64_t)b * (p.Hq / w.rep_a) + h / w.rep_a;
  const int64_t hb = (int64_t)b * (p.Hq / w.rep_b) + h / w.rep_b;
  const int64_t hc = (int64_t)b * (p.Hq / w.rep_c) + h / w.rep_c;
  for (int i = threadIdx.x; i <= C + 1; i += kThreads) pw[i] = lin_pow(ld, i);

  const int m1 = min((run + 1) * p.cps, p.nch);
  auto pos_of = [&](int m) { return lin_first<C, false>(p, lin_chunk(p.nch, w.back, m)); };
  // (0: a row's padding, in sweeps from the front, or past the run)
  auto size_of = [&](int m) { return m < m1 ? lin_size<C, false>(p, n_tok, lin_chunk(p.nch, w.back, m)) : 0; };
  int m = run * p.cps, n = size_of(m);
  if (n > 0) {
    if (!SUM) load_tile<E, DP>(p, w.a, ha, pos_of(m), n, sa);
    commit_tile();
    load_tile<E, DP>(p, w.b, hb, pos_of(m), n, sb);
    if (SUM) load_tile<E, DP>(p, w.c, hc, pos_of(m), n, sc);
    commit_tile();
  }

  // M of this thread: rows 4 ty + 64 i + x, columns 4 tx + 64 j + 2 y and the next
  float2 M[R][4][R][2] = {};
  const int64_t DD = (int64_t)p.D * p.D;
  if (!SUM) {
    // M = f M + g (a state, as it lies or transposed), a vector of four numbers at a time
    auto fold = [&](float f, float g, const float* src) {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const int r = 4 * ty + 64 * i, c = 4 * tx + 64 * j;
          if (r >= p.D || c >= p.D) continue;
          float v[4][4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float4 u = *reinterpret_cast<const float4*>(
                src + (w.trans ? (int64_t)(c + x) * p.D + r : (int64_t)(r + x) * p.D + c));
            v[x][0] = u.x, v[x][1] = u.y, v[x][2] = u.z, v[x][3] = u.w;
          }
#pragma unroll
          for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              float2& m = M[i][x][j][y];
              m.x = fmaf(f, m.x, g * (w.trans ? v[2 * y][x] : v[x][2 * y]));
              m.y = fmaf(f, m.y, g * (w.trans ? v[2 * y + 1][x] : v[x][2 * y + 1]));
            }
        }
    };
    if (w.init) fold(0.f, w.init_mul, w.init + bh * DD);
    for (int s = 0; s < run; ++s)
      fold(lin_pow(ld, lin_run_tokens<C, false>(p, n_tok, w.back, s)), 1.f, w.sums + ((int64_t)bh * p.segs + s) * DD);
  }

  // A chunk's tiles come ahead of it: a while the chunk before runs, b (in the place of that one's
  // a) during its last product, c during the scores.
  for (int next; n > 0; ++m, n = next) {
    const int pos0 = pos_of(m);
    next = size_of(m + 1);
    __syncthreads();    // the last chunk's tiles have been read
    if (!SUM) {
      load_tile<E, DP>(p, w.c, hc, pos0, n, sc);
      commit_tile();
      if (next > 0) load_tile<E, DP>(p, w.a, ha, pos_of(m + 1), next, sx);
      commit_tile();
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int j = 0; j < R; ++j)
            *reinterpret_cast<float4*>(sM + (4 * ty + 64 * i + x) * LD + 4 * tx + 64 * j) =
                make_float4(M[i][x][j][0].x, M[i][x][j][0].y, M[i][x][j][1].x, M[i][x][j][1].y);
      wait_tiles<2>();
    } else {
      if (next > 0) {
        load_tile<E, DP>(p, w.b, hb, pos_of(m + 1), next, sa);
        load_tile<E, DP>(p, w.c, hc, pos_of(m + 1), next, sx);
      }
      commit_tile();
      wait_tiles<1>();
    }
    __syncthreads();
    if (!SUM) {
      float2 s2[4][4] = {};  // rows ty + 16 i, columns tx + 16 j; even and odd channels apart
#pragma unroll 2
      for (int d = 0; d < DP; d += 4) {
        float4 a[4], v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = *reinterpret_cast<const float4*>(sa + (ty + 16 * i) * LD + d);
          v[i] = *reinterpret_cast<const float4*>(sb + (tx + 16 * i) * LD + d);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            s2[i][j] = fma2(make_float2(a[i].x, a[i].y), make_float2(v[j].x, v[j].y), s2[i][j]);
            s2[i][j] = fma2(make_float2(a[i].z, a[i].w), make_float2(v[j].z, v[j].w), s2[i][j]);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int row = ty + 16 * i, col = tx + 16 * j;
          const int e = w.back ? col - row : row - col;
          sp[row * PL + col] = e >= 0 ? (s2[i][j].x + s2[i][j].y) * pw[e] : 0.f;
        }
      wait_tiles<1>();  // c
      __syncthreads();
      float2 o[4][R][2] = {}, t[4][R][2] = {};  // rows ty + 16 i, columns 4 tx + 64 j + 2 y
      // x[row][k] m[k][columns] over k, four of them a step: their rows of x come as one vector
      auto product = [&](float2(&acc)[4][R][2], const float* x, int ldx, const float* m, int K) {
#pragma unroll 2
        for (int k = 0; k < K; k += 4) {
          float4 xr[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) xr[i] = *reinterpret_cast<const float4*>(x + (ty + 16 * i) * ldx + k);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            float4 v[R];
#pragma unroll
            for (int j = 0; j < R; ++j) v[j] = *reinterpret_cast<const float4*>(m + (k + kk) * LD + 4 * tx + 64 * j);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float f = kk == 0 ? xr[i].x : kk == 1 ? xr[i].y : kk == 2 ? xr[i].z : xr[i].w;
              const float2 f2 = make_float2(f, f);
#pragma unroll
              for (int j = 0; j < R; ++j) {
                acc[i][j][0] = fma2(f2, make_float2(v[j].x, v[j].y), acc[i][j][0]);
                acc[i][j][1] = fma2(f2, make_float2(v[j].z, v[j].w), acc[i][j][1]);
              }
            }
          }
        }
      };
      product(o, sp, PL, sc, C);
      product(t, sa, LD, sM, DP);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = ty + 16 * i;
        if (row >= n) continue;
        const float ow = pw[(w.back ? n - 1 - row : row) + 1 - late];
        const int64_t at = ((int64_t)bh * p.T + p.m.slot(pos0 + row)) * p.D;
#pragma unroll
        for (int j = 0; j < R; ++j) {
          const int c = 4 * tx + 64 * j;
          if (c >= p.D) continue;
          const float4 y = make_float4(w.mul * fmaf(ow, t[i][j][0].x, o[i][j][0].x), w.mul * fmaf(ow, t[i][j][0].y, o[i][j][0].y),
                                       w.mul * fmaf(ow, t[i][j][1].x, o[i][j][1].x), w.mul * fmaf(ow, t[i][j][1].y, o[i][j][1].y));
          if (w.out_f32) store4(static_cast<float*>(w.out) + at + c, y);
          else store4(static_cast<E*>(w.out) + at + c, y);
        }
      }
      __syncthreads();  // a has been read
      if (next > 0) load_tile<E, DP>(p, w.b, hb, pos_of(m + 1), next, sa);
      commit_tile();
    }
    // U = the chunk's own sum, from zero: the rounding errors of M grow with its chunks, not its tokens
    float2 U[R][4][R][2] = {};
#pragma unroll 2
    for (int k = 0; k < n; ++k) {
      const float uw = pw[(w.back ? k : n - 1 - k) + late];
      float2 v[R][2];
      float u[R][4];
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const float4 x = *reinterpret_cast<const float4*>(sc + k * LD + 4 * tx + 64 * j);
        v[j][0] = make_float2(x.x, x.y), v[j][1] = make_float2(x.z, x.w);
        const float4 y = *reinterpret_cast<const float4*>(sb + k * LD + 4 * ty + 64 * j);
        u[j][0] = uw * y.x, u[j][1] = uw * y.y, u[j][2] = uw * y.z, u[j][3] = uw * y.w;
      }
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float2 f2 = make_float2(u[i][x], u[i][x]);
#pragma unroll
          for (int j = 0; j < R; ++j)
#pragma unroll
            for (int y = 0; y < 2; ++y) U[i][x][j][y] = fma2(f2, v[j][y], U[i][x][j][y]);
        }
    }
    const float2 rn = make_float2(pw[n], pw[n]);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int j = 0; j < R; ++j)
#pragma unroll
          for (int y = 0; y < 2; ++y) M[i][x][j][y] = fma2(rn, M[i][x][j][y], U[i][x][j][y]);
    // the next chunk's tiles: a in sx, b in sa, c (SUM: in sx) yet to come
    float* const old = sb;
    sb = sa;
    if (SUM) {
      sa = old;
      float* const o = sc;
      sc = sx;
      sx = o;
    } else {
      sa = sx;
      sx = sc;
      sc = old;
    }
  }

  float* dst = SUM ? w.sums + ((int64_t)bh * p.segs + run) * DD
                   : run == p.segs - 1 && w.fin ? w.fin + bh * DD : nullptr;
  if (!dst) return;
  const float mul = SUM ? 1.f : w.fin_mul;
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int j = 0; j < R; ++j) {
        const int r = 4 * ty + 64 * i + x, c = 4 * tx + 64 * j;
        if (r < p.D && c < p.D)
          store4(dst + (int64_t)r * p.D + c,
                 make_float4(M[i][x][j][0].x * mul, M[i][x][j][0].y * mul, M[i][x][j][1].x * mul, M[i][x][j][1].y * mul));
      }
}

template <typename E, int DP>
static cudaError_t launch(const Linear& p, cudaStream_t st, const char* sums, const char* sweeps) {
  constexpr int kBytes = Smem<DP>::kFloats * 4;
  static ReadyDevices ready;
  cudaError_t e = ready.once([] {
    const cudaError_t r = cudaFuncSetAttribute(sweep_kernel<E, DP, true>,
                                               cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
    return r != cudaSuccess ? r
                            : cudaFuncSetAttribute(sweep_kernel<E, DP, false>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes);
  });
  if (e != cudaSuccess) return e;
  const unsigned bh = (unsigned)(p.B * p.Hq);
  if (p.segs > 1) {
    timing_begin(sums, st);
    sweep_kernel<E, DP, true><<<dim3(bh * (p.segs - 1), p.n_sums), kThreads, kBytes, st>>>(p);
    e = cudaGetLastError();
    timing_end(st);
    if (e != cudaSuccess) return e;
  }
  timing_begin(sweeps, st);
  sweep_kernel<E, DP, false><<<dim3(bh * p.segs, p.n_sweeps), kThreads, kBytes, st>>>(p);
  e = cudaGetLastError();
  timing_end(st);
  return e;
}

// blockIdx.y: dv or dk.
template <typename E>
__global__ void __launch_bounds__(256) group_kernel(int64_t n4, int n_rep, int64_t row4, const float4* part_v,
                                                    const float4* part_k, E* dv, E* dk) {
  griddep_wait();  // (started while the sweeps' last blocks finish)
  const float4* part = blockIdx.y ? part_k : part_v;
  E* out = blockIdx.y ? dk : dv;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n4; i += (int64_t)gridDim.x * 256) {
    const int64_t g = i / row4;
    const float4* src = part + g * (n_rep - 1) * row4 + i;
    float4 s = __ldcs(src);
#pragma unroll 4
    for (int r = 1; r < n_rep; ++r) {
      const float4 x = __ldcs(src + r * row4);
      s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
    }
    store4(out + 4 * i, s);
  }
}

}  // namespace linsimt

cudaError_t launch_linear_simt(const Linear& p, cudaStream_t st, bool backward) {
  const char* sums = backward ? "linear_bwd_sums" : "linear_fwd_sums";
  const char* sweeps = backward ? "linear_bwd" : "linear_fwd";
  if (p.bf16)
    return p.D <= 64 ? linsimt::launch<__nv_bfloat16, 64>(p, st, sums, sweeps)
                     : linsimt::launch<__nv_bfloat16, 128>(p, st, sums, sweeps);
  return p.D <= 64 ? linsimt::launch<float, 64>(p, st, sums, sweeps)
                   : linsimt::launch<float, 128>(p, st, sums, sweeps);
}

cudaError_t launch_linear_group(int64_t groups, int n_rep, int64_t row_elems, const float* part_v,
                                const float* part_k, void* dv, void* dk, int bf16, cudaStream_t st) {
  const int64_t n4 = groups * row_elems / 4;
  const int64_t want = (n4 + 255) / 256, most = 16 * kSms;
  const dim3 grid((unsigned)(want < most ? want : most), 2);
  const float4 *pv = reinterpret_cast<const float4*>(part_v), *pk = reinterpret_cast<const float4*>(part_k);
  timing_begin("linear_group", st);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const int64_t row4 = row_elems / 4;
  const cudaError_t e =
      bf16 ? cudaLaunchKernelEx(&cfg, linsimt::group_kernel<__nv_bfloat16>, n4, n_rep, row4, pv, pk,
                                static_cast<__nv_bfloat16*>(dv), static_cast<__nv_bfloat16*>(dk))
           : cudaLaunchKernelEx(&cfg, linsimt::group_kernel<float>, n4, n_rep, row4, pv, pk, static_cast<float*>(dv),
                                static_cast<float*>(dk));
  timing_end(st);
  return e;
}

}  // namespace cpattn
