// Linear attention, one token of each request over its state:
//     S' = r S + k v^T,   o = scale q^T S'.
// All there is to do is to read and write the states, 8 D^2 bytes a head: each thread takes
// four columns (values' channels) of some of the rows (keys' channels), and o, the sum over
// the rows, is joined over a warp's lanes and then over the warps in shared memory.
//
// 128 requests of 32 heads at D 128: 82 us, 6.6 TB/s, 97 % of a copy's rate; one request 3.0 us.
//
// A block takes all columns of a head's state when requests and heads fill the GPU, else 32
// of them: columns do not meet in o, so the cut costs nothing but q and k read again.
#include "layer.cuh"

namespace cpattn {
namespace linstep {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// LC lanes over 4 LC columns; a warp takes 32 / LC rows at a time.
template <typename E, int LC>
__global__ void __launch_bounds__(kThreads) step_kernel(const LinStep p) {
  constexpr int kCols = 4 * LC, kRows = 32 / LC, kStep = kRows * kWarps;
  constexpr int kDepth = 128 / kStep;  // rows a thread at D 128
  __shared__ float qs[128], ks[128], vs[kCols];
  __shared__ __align__(16) float part[kWarps][kCols];
  const int b = blockIdx.x / p.Hq, h = blockIdx.x - b * p.Hq, g = h / (p.Hq / p.Hkv);
  const int slot = p.slots ? p.slots[b] : b;
  if (slot < 0 || slot >= p.n_states) return;
  const int col0 = blockIdx.y * kCols;
  const E* q = static_cast<const E*>(p.q) + b * p.q_ts + h * p.q_hs;
  const E* k = static_cast<const E*>(p.k) + b * p.k_ts + g * p.k_hs;
  const E* v = static_cast<const E*>(p.v) + b * p.v_ts + g * p.v_hs;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int lc = lane % LC, row0 = warp * kRows + lane / LC, col = col0 + 4 * lc;
  const bool live = col < p.D;
  const int64_t base = ((int64_t)slot * p.Hq + h) * p.D * p.D + col;
  // the state's loads go out first: nothing else takes long
  float4 s[kDepth];
#pragma unroll
  for (int i = 0; i < kDepth; ++i) {
    const int r = row0 + i * kStep;
    s[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live && r < p.D) s[i] = __ldcs(reinterpret_cast<const float4*>(p.in + base + (int64_t)r * p.D));
  }
  for (int i = threadIdx.x; i < p.D; i += kThreads) {
    qs[i] = to_f(q[i]);
    ks[i] = to_f(k[i]);
  }
  if (threadIdx.x < kCols && col0 + threadIdx.x < p.D) vs[threadIdx.x] = to_f(v[col0 + threadIdx.x]);
  const float r1 = expf(fminf(p.log_decay[h], 0.f));
  __syncthreads();
  float4 vv = make_float4(0.f, 0.f, 0.f, 0.f), o = vv;
  if (live) vv = make_float4(vs[4 * lc], vs[4 * lc + 1], vs[4 * lc + 2], vs[4 * lc + 3]);
#pragma unroll
  for (int i = 0; i < kDepth; ++i) {
    const int r = row0 + i * kStep;
    if (live && r < p.D) {
      const float kr = ks[r], qr = qs[r];
      float4 x = s[i];
      x.x = fmaf(kr, vv.x, r1 * x.x);
      x.y = fmaf(kr, vv.y, r1 * x.y);
      x.z = fmaf(kr, vv.z, r1 * x.z);
      x.w = fmaf(kr, vv.w, r1 * x.w);
      __stcs(reinterpret_cast<float4*>(p.out + base + (int64_t)r * p.D), x);
      o.x = fmaf(qr, x.x, o.x);
      o.y = fmaf(qr, x.y, o.y);
      o.z = fmaf(qr, x.z, o.z);
      o.w = fmaf(qr, x.w, o.w);
    }
  }
#pragma unroll
  for (int d = LC; d < 32; d <<= 1) {
    o.x += __shfl_xor_sync(0xffffffffu, o.x, d);
    o.y += __shfl_xor_sync(0xffffffffu, o.y, d);
    o.z += __shfl_xor_sync(0xffffffffu, o.z, d);
    o.w += __shfl_xor_sync(0xffffffffu, o.w, d);
  }
  if (lane < LC) *reinterpret_cast<float4*>(&part[warp][4 * lc]) = o;
  __syncthreads();
  if (threadIdx.x < kCols && col0 + threadIdx.x < p.D) {
    float x = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) x += part[w][threadIdx.x];
    put(static_cast<E*>(p.o) + ((int64_t)b * p.Hq + h) * p.D + col0 + threadIdx.x, x * p.scale);
  }
}

template <typename E>
static void launch(const LinStep& p, cudaStream_t st) {
  const unsigned heads = (unsigned)((int64_t)p.n * p.Hq);
  if (heads >= 8u * kSms || p.D <= 32)
    step_kernel<E, 32><<<dim3(heads, 1), kThreads, 0, st>>>(p);
  else
    step_kernel<E, 8><<<dim3(heads, (p.D + 31) / 32), kThreads, 0, st>>>(p);
}

}  // namespace linstep

cudaError_t launch_linear_step(const LinStep& p, cudaStream_t st) {
  timing_begin("linear_step", st);
  if (p.bf16) linstep::launch<__nv_bfloat16>(p, st);
  else linstep::launch<float>(p, st);
  const cudaError_t e = cudaGetLastError();
  timing_end(st);
  return e;
}

}  // namespace cpattn
