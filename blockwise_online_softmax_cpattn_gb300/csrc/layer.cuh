// What the calls around and beside softmax attention share: norm and rotation (rotate.cu) and
// linear attention (linear_tc.cu, linear_simt.cu, linear_step.cu); validation in api_layer.cu.
#pragma once

#include <atomic>

#include "kernels.h"

namespace cpattn {

// SMs of a GB300: what work is cut for.  Workspaces depend on the cut, so it is a constant and
// not a question to the device.
constexpr int kSms = 152;

// What a kernel needs set before its first launch on a device: a call on every launch costs the host
// a microsecond.
struct ReadyDevices {
  std::atomic<uint64_t> set[2] = {};
  template <typename F>
  cudaError_t once(F prepare) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (dev < 128 && (set[dev >> 6].load() & bit)) return cudaSuccess;
    if ((e = prepare()) == cudaSuccess && dev < 128) set[dev >> 6].fetch_or(bit);
    return e;
  }
};

// ---- rotate.cu ---------------------------------------------------------------
// A [B][H][T][D] tensor by strides in elements; channels are contiguous.
struct RowView {
  void* p;
  int64_t sb, sh, st;
};

struct Rotate {
  int B, Hq, Hkv, T, D, rot;
  SeqMap m;
  int bf16, near, norm, natural_in;
  float eps;
  // queries, keys, values.  Forward: in = the projection's side, out = the attention's.
  // Backward: in = the upstream gradient (attention's side), x = the forward's input, out =
  // its gradient (projection's side)
  RowView in[3], x[3], out[3];
  const void* w[2];
  const double* inv_freq;
  const int* positions;
  float* sums;   // backward: a row of 2 D numbers a block
  // set by the launch: pairs a lane, lanes a row, groups of slots, parts of the heads
  int P, lanes, groups, splits;
  float inv_d;
};
// Blocks of the backward kernel at most, each with a row of sums: two an SM.
constexpr int kBwdBlocks = 2 * kSms;
size_t rotate_bwd_workspace(int D, int norm);
cudaError_t launch_rotate_fwd(Rotate p, cudaStream_t st);
cudaError_t launch_rotate_bwd(Rotate p, float* dq_weight, float* dk_weight, cudaStream_t st);

// ---- linear attention ---------------------------------------------------------
// Forward and backward are one sum, three times over: with r the decay of a head,
//     out_i = mul * ( sum over j at or before i of r^(i-j) (a_i . b_j) c_j  +  what went before )
//   o  : a = q,  b = k,  c = v    from the front
//   dq : a = dO, b = v,  c = k    from the front
//   dv : a = k,  b = q,  c = dO   from the back (i and j change places)
//   dk : a = v,  b = dO, c = q    from the back
// "What went before" a chunk of tokens is one D x D matrix, M = sum r^.. b_j c_j^T.  A sweep
// goes through its chunks with M in float32: in a chunk of n tokens, the i-th of the sweep's
// direction (from 0) gets r^(i+1-late) a_i M, and M becomes r^n M + sum r^(n-1-j+late) b_j c_j^T.
// late is 1 from the back: the state's gradient behind the last token reaches that token itself
// undecayed, while the state before the first token has decayed once when the first token sees it.
//
// A sequence is cut into `segs` runs of `cps` chunks for the GPU's width.  With more than one, a
// first launch leaves every run's own sum (M from zero) in the workspace, and a run of the
// second starts from the sums of the runs before it, folded in order.
struct LinSweep {
  const void *a, *b, *c;
  int rep_a, rep_b, rep_c;  // query heads per head of the tensor
  int back;                 // from the back, late
  // M before the first run: init [B'][Hq][D][D] or null, times init_mul; as it lies there
  // (rows b's channel) or transposed
  const float* init;
  float init_mul;
  int trans;
  // the runs' own sums, [B' Hq][segs][D][D], read transposed or not like init
  float* sums;
  float mul;
  void* out;
  int out_f32;
  float* fin;  // M behind the last run, times fin_mul, or null
  float fin_mul;
  int exact;   // M is handed out in the end
};

constexpr int kMaxSweeps = 3;

struct Linear {
  int B, Hq, Hkv, T, D, bf16;
  int B_user;      // batch rows of one a2a slice: the slice gives the heads' decays
  SeqMap m;
  const float* log_decay;
  const int* lengths;
  int segs, cps, nch;   // runs, chunks a run, chunks of a sequence
  // A chunk's positions are consecutive slots: where the token order has stretches (zigzag) off the
  // chunks' grid, chunks begin anew with each of them, `per` chunks for its `seg` tokens.  Else one
  // stretch, of the whole sequence.
  int seg, per;
  int n_sums, n_sweeps; // sweeps of the first (sums) and second launch
  LinSweep sum[2], sweep[kMaxSweeps];
  int* status;
  int debug_fault;
};

// A head's log decay, and r^n.
__device__ __forceinline__ float lin_decay(const Linear& p, int bh) {
  const int b = bh / p.Hq, h = bh - b * p.Hq;
  return fminf(p.log_decay[(b / p.B_user) * p.Hq + h], 0.f);  // (of a NaN: 0)
}
// (the product's rounding, up to 2^-24 of the exponent, is made good)
__device__ __forceinline__ float lin_pow(float ld, int n) {
  if (n == 0) return 1.f;
  const float x = ld * n, e = expf(x);
  return x < -80.f ? e : fmaf(e, fmaf(ld, (float)n, -x), e);
}

__device__ __forceinline__ int lin_tokens(const Linear& p, int bh) {
  if (!p.lengths) return p.T;
  const int n = p.lengths[bh / p.Hq];
  return n < 0 ? 0 : n > p.T ? p.T : n;
}

// Chunk number of a sweep's m-th chunk.
__device__ __forceinline__ int lin_chunk(int nch, int back, int m) { return back ? nch - 1 - m : m; }
__device__ __forceinline__ int lin_clamp(int n, int most) { return n < 0 ? 0 : n > most ? most : n; }
// First position of chunk c (of the one behind the last: T), and its tokens in a row of n_tok.
// PIECES: the token order has more stretches than one.
template <int C, bool PIECES>
__device__ __forceinline__ int lin_first(const Linear& p, int c) {
  if (!PIECES) return min(c * C, p.T);
  const int q = c < p.per ? 0 : c / p.per;
  return c == p.nch ? p.T : q * p.seg + (c - q * p.per) * C;
}
template <int C, bool PIECES>
__device__ __forceinline__ int lin_size(const Linear& p, int n_tok, int c) {
  if (!PIECES) return lin_clamp(n_tok - c * C, C);
  const int q = c < p.per ? 0 : c / p.per, at = (c - q * p.per) * C;
  return lin_clamp(n_tok - q * p.seg - at, min(C, p.seg - at));
}
// Chunks that a row of n_tok tokens has.
template <int C, bool PIECES>
__device__ __forceinline__ int lin_chunks(const Linear& p, int n_tok) {
  if (!PIECES) return (n_tok + C - 1) / C;
  const int q = n_tok / p.seg;
  return q * p.per + (n_tok - q * p.seg + C - 1) / C;
}
// Tokens of run s of a sweep over n_tok tokens (from the back: whole rows).
template <int C, bool PIECES>
__device__ __forceinline__ int lin_run_tokens(const Linear& p, int n_tok, int back, int s) {
  const int m0 = s * p.cps, m1 = min(m0 + p.cps, p.nch);
  if (back) return lin_first<C, PIECES>(p, p.nch - m0) - lin_first<C, PIECES>(p, p.nch - m1);
  return min(lin_first<C, PIECES>(p, m1), n_tok) - min(lin_first<C, PIECES>(p, m0), n_tok);
}

// ---- linear_tc.cu (bf16, D 64 or 128) / linear_simt.cu (all else) -------------
constexpr int kLinTcChunk = 128;
constexpr int kLinSimtChunk = 64;
bool linear_tc_supported(const Ring& R);
cudaError_t launch_linear_tc(const Linear& p, cudaStream_t st, bool backward);
cudaError_t launch_linear_simt(const Linear& p, cudaStream_t st, bool backward);
// dv[b][g][t][:] = sum over the group's n_rep query heads of part_v[b][g n_rep + r][t][:]; dk alike.
cudaError_t launch_linear_group(int64_t groups, int n_rep, int64_t row_elems, const float* part_v,
                                const float* part_k, void* dv, void* dk, int bf16, cudaStream_t st);

// ---- linear_step.cu -----------------------------------------------------------
struct LinStep {
  int n, n_states, Hq, Hkv, D, bf16;
  float scale;
  const void *q, *k, *v;
  int64_t q_ts, q_hs, k_ts, k_hs, v_ts, v_hs;
  const float* log_decay;
  const int* slots;
  const float* in;
  float* out;
  void* o;
};
cudaError_t launch_linear_step(const LinStep& p, cudaStream_t st);

}  // namespace cpattn
