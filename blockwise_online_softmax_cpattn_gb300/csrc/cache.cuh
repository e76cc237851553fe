// The 4-bit key/value cache: geometry, launchers (internal to libcpattn) and the
// device side of its format.
//
// A group of G channels of one token and K/V head is 4-bit codes c and two bf16
// numbers a, z; a channel stands for round_bf16(a * (1 + c / 16) + z).  The form is
// chosen for the reader: 1 + c / 16 in bf16 is the bit pattern 0x3F80 | c << 3, so a
// pair of codes becomes a pair of bf16 values by one shift, one three-input logic
// operation and one packed bf16 FMA -- against a subtraction more for the usual
// code-times-scale-plus-zero.  Tensor-core operands come out exact: the cache's
// values ARE bf16 numbers, as k and v are everywhere else in the library.
#pragma once

#include "kernels.h"

namespace cpattn {

constexpr int kCacheTile = 16;            // tokens per tile (the K dimension of one MMA)
constexpr int kStatusRange = 6;           // device range word: a value the cache cannot hold
constexpr float kCacheHuge = 0x1p120f;    // stored values are held within +- this
constexpr float kCacheTiny = 0x1p-100f;   // a group whose a is below this has a = 0

// n / d for 0 <= n < 2^31 by a multiplication (Granlund and Montgomery's division by invariant
// integers): with s = ceil(log2 d) and
// m = floor(2^32 (2^s - d) / d) + 1, n / d = (hi(m n) + n) >> s.
struct Divider {
  uint32_t d, m, s;
  static Divider of(uint32_t d) {
    uint32_t s = 0;
    while ((1u << s) < d) ++s;
    return {d, (uint32_t)((((uint64_t)1 << s) - d << 32) / d + 1), s};
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(m, n) + n) >> s; }
};

struct Cache {
  int Hq, Hkv, D, G, page, n_pages;
  int bf16;        // q, k, v: 1 bf16, 0 f32
  int o_f32;       // o: 1 f32, 0 as q
  int causal;
  int debug_fault; // cpattn_cache_desc
  float scale;
  // a K half and a V half: codes of 16 rows, their (a, z)
  __host__ __device__ int tile_bytes() const { return 2 * kCacheTile * (D / 2 + 4 * (D / G)); }
  // of one page and K/V head
  __host__ __device__ int64_t block_bytes() const {
    return (int64_t)(page / kCacheTile) * tile_bytes();
  }
  __host__ __device__ int64_t slots() const { return (int64_t)n_pages * page; }
};

// Row of token t (of its tile) in the V half: 2t + e of every eight is in row t + 4e,
// so the eight lanes of an MMA operand that read tokens t and the eight that read
// t + 1 each find theirs in four neighbouring rows.
__host__ __device__ __forceinline__ int cache_v_row(int t) {
  return (t & 8) | ((t >> 1) & 3) | ((t & 1) << 2);
}

// The four pairs of values of one word of 8 codes: pair p = channels (2p, 2p + 1).
// K words are rotated left by 3, which puts pair 0 where it is needed; the others take
// one (funnel) shift each.  V words are plain.
__device__ __forceinline__ uint32_t bf16x2_fma(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// `ones` is kOnes in a register the compiler cannot see through: with two immediates
// the and-or would become two instructions.
constexpr uint32_t kOnes = 0x3F803F80u;
__device__ __forceinline__ uint32_t code_to_bf16(uint32_t x, uint32_t ones) {  // codes at bits 3..6, 19..22
  return (x & 0x00780078u) | ones;
}
template <bool K>
__device__ __forceinline__ void codes_to_bf16(uint32_t w, uint32_t ones, uint32_t (&u)[4]) {
  if constexpr (K) {
    u[0] = code_to_bf16(w, ones);
    u[1] = code_to_bf16(w >> 4, ones);
    u[2] = code_to_bf16(w >> 8, ones);
    u[3] = code_to_bf16(__funnelshift_r(w, w, 12), ones);
  } else {
    u[0] = code_to_bf16(w << 3, ones);
    u[1] = code_to_bf16(w >> 1, ones);
    u[2] = code_to_bf16(w >> 5, ones);
    u[3] = code_to_bf16(w >> 9, ones);
  }
}
// (a, a) and (z, z) of an (a, z) word
__device__ __forceinline__ uint32_t az_a2(uint32_t az) { return __byte_perm(az, az, 0x1010); }
__device__ __forceinline__ uint32_t az_z2(uint32_t az) { return __byte_perm(az, az, 0x3232); }

// min / max that pass a NaN on
__device__ __forceinline__ float min_nan(float a, float b) {
  float d;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

__device__ __forceinline__ float min3_nan(float a, float b, float c) {
  float d;
  asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// ---- cache_plan.cu ---------------------------------------------------------
struct PlanArgs {
  int n_req, max_pages, page, n_pages, n_slots;
  const int *len_old, *len_new;
  int *table, *free_list;
  const int* n_free;
  int *n_free_out, *len_out, *q_start, *slots;
  int* ws;
};
size_t cache_plan_workspace(int n_req);
cudaError_t launch_cache_plan(const PlanArgs& a, cudaStream_t st);

// ---- cache_rows.cu ---------------------------------------------------------
struct RowStrides {
  int64_t token, head;  // elements
};
cudaError_t launch_cache_append(const Cache& c, int n, const void* k, RowStrides ks, const void* v,
                                RowStrides vs, const int* slots, void* cache, int* range,
                                cudaStream_t st);
cudaError_t launch_cache_read(const Cache& c, int n, const int* slots, const void* cache, void* k,
                              RowStrides ks, void* v, RowStrides vs, cudaStream_t st);

// ---- cache_attn.cu ---------------------------------------------------------
struct CacheAttnArgs {
  int n_req, max_pages, n_tokens, max_q;
  const void* q;
  RowStrides qs;
  const int *q_start, *kv_len, *table;
  const uint8_t* cache;
  void* o;
  float* lse;
  void* ws;
  int* status;
};
size_t cache_attn_workspace(const Cache& c);
cudaError_t launch_cache_attn(const Cache& c, const CacheAttnArgs& a, cudaStream_t st);

}  // namespace cpattn
