// The C ABI of what stands around and beside softmax attention: norm and rotation, linear
// attention.  Argument validation, workspaces and dispatch.
#include <limits.h>
#include <math.h>

#include <initializer_list>

#include "api_internal.h"
#include "layer.cuh"

namespace cpattn {

static bool aligned(const void* p, unsigned n) { return p && ((uintptr_t)p % n == 0); }
static bool null_or_aligned(const void* p, unsigned n) { return !p || ((uintptr_t)p % n == 0); }

// Does one of the outputs begin where an input or another output does?
static bool meet(std::initializer_list<const void*> outs, std::initializer_list<const void*> ins) {
  for (auto o = outs.begin(); o != outs.end(); ++o) {
    if (!*o) continue;
    for (const void* i : ins)
      if (*o == i) return true;
    for (auto u = outs.begin(); u != o; ++u)
      if (*o == *u) return true;
  }
  return false;
}

// ---------------------------------------------------------------------------
// norm and rotation
// ---------------------------------------------------------------------------
static cpattn_status validate_rotate(const cpattn_rotate_desc* d, Rotate* p) {
  if (!d) return CPATTN_ERR_INVALID_ARG;
  if (d->B <= 0 || d->H_q <= 0 || d->H_kv <= 0 || d->T <= 0 || d->D <= 0 || d->cp <= 0)
    return CPATTN_ERR_INVALID_ARG;
  if (d->layout != CPATTN_CONTIGUOUS && d->layout != CPATTN_ZIGZAG) return CPATTN_ERR_INVALID_ARG;
  if (d->dtype != CPATTN_F32 && d->dtype != CPATTN_BF16) return CPATTN_ERR_INVALID_ARG;
  if (d->pairing != CPATTN_HALVES && d->pairing != CPATTN_NEIGHBOURS) return CPATTN_ERR_INVALID_ARG;
  if ((d->norm != 0 && d->norm != 1) || (d->natural_in != 0 && d->natural_in != 1))
    return CPATTN_ERR_INVALID_ARG;
  if (!(d->eps >= 0.f) || !isfinite(d->eps)) return CPATTN_ERR_INVALID_ARG;
  if (d->rot < 0 || d->rot > d->D) return CPATTN_ERR_INVALID_ARG;
  if (d->T % d->cp || (d->layout == CPATTN_ZIGZAG && (d->cp > (1 << 29) || d->T % (2 * d->cp))))
    return CPATTN_ERR_INVALID_ARG;
  if (d->D % 8 || d->D > 128 || d->rot % 8) return CPATTN_ERR_UNSUPPORTED;
  // heads and (at a slot a block) blocks are counted in 32 bits
  if (d->H_q > 32767 || d->H_kv > 32767 || d->T > (1 << 30) || (int64_t)d->B * d->T > INT_MAX / 2)
    return CPATTN_ERR_UNSUPPORTED;
  if (p) {
    *p = Rotate{};
    p->B = d->B;
    p->Hq = d->H_q;
    p->Hkv = d->H_kv;
    p->T = d->T;
    p->D = d->D;
    p->rot = d->rot;
    p->m = SeqMap::make(d->T, d->cp, d->layout == CPATTN_ZIGZAG);
    p->bf16 = d->dtype == CPATTN_BF16;
    p->near = d->pairing == CPATTN_NEIGHBOURS;
    p->norm = d->norm;
    p->natural_in = d->natural_in;
    p->eps = d->eps;
  }
  return CPATTN_OK;
}

// A tensor and its strides (null: contiguous); every row on a 16-byte boundary.  A stride of a
// dimension of extent 1 may be anything; an output's may not be 0, its rows differ.
static bool view(const Rotate& p, const void* t, const int64_t* strides, int heads, bool out, RowView* v) {
  v->p = const_cast<void*>(t);
  if (!strides) {
    v->st = p.D;
    v->sh = (int64_t)p.T * p.D;
    v->sb = v->sh * heads;
  } else {
    v->sb = p.B > 1 ? strides[0] : 0;
    v->sh = heads > 1 ? strides[1] : 0;
    v->st = p.T > 1 ? strides[2] : 0;
    const int64_t vec = p.bf16 ? 8 : 4;
    if (v->sb % vec || v->sh % vec || v->st % vec || v->sb < 0 || v->sh < 0 || v->st < 0) return false;
    if (out && ((p.B > 1 && v->sb < p.D) || (heads > 1 && v->sh < p.D) || (p.T > 1 && v->st < p.D)))
      return false;
  }
  return aligned16(t);
}

// Does an output begin where another one or an input does?  In place, over the same rows of its
// own input, only where every row stays where it is (not of x: the backward pass's other input).
static bool rotate_meet(const Rotate& p) {
  const bool stays = !p.natural_in || !p.m.zz || p.m.cp == 1;
  for (int o = 0; o < 3; ++o) {
    const RowView& y = p.out[o];
    if (!y.p) continue;
    const int heads = o == 0 ? p.Hq : p.Hkv;
    for (int i = 0; i < 3; ++i) {
      const RowView& a = p.in[i];
      const bool same = a.p == y.p && (p.B == 1 || a.sb == y.sb) && (heads == 1 || a.sh == y.sh) &&
                        (p.T == 1 || a.st == y.st);
      if (a.p == y.p && !(i == o && same && stays)) return true;
      if (p.x[i].p == y.p || (i < o && p.out[i].p == y.p)) return true;
    }
  }
  return false;
}

// ---------------------------------------------------------------------------
// linear attention
// ---------------------------------------------------------------------------
// The ring's descriptor, and what linear attention takes of it.
static cpattn_status validate_linear(const cpattn_desc* d, Ring* R) {
  const cpattn_status s = validate_ring(d, R);
  if (s != CPATTN_OK) return s;
  if (d->D % 8) return CPATTN_ERR_UNSUPPORTED;
  // heads times the runs of a sequence (64 at most) are the blocks of one launch
  if ((int64_t)R->B * R->Hq > INT_MAX / 64) return CPATTN_ERR_UNSUPPORTED;
  return CPATTN_OK;
}

// Runs a sequence is cut into, for `sweeps` sweeps and `sums` sums of its heads.  One run needs
// no sums; more fill the GPU when heads are few, but every run but the last reads its keys and
// values twice and starts from its predecessors' states.  In units of a chunk's time on one SM
// (on the tensor cores some 3 us, in float32 some 20): a chunk of a sweep 1, of a sum 0.3 (0.6), a
// block's start 1 (0.15), folding a predecessor's state 0.25 (0.1), the second launch 2 (0.5).  Of
// 22 problems of 2 to 128 heads and 300 to 32768 tokens, backward passes among them, every cut's
// time was within 2 % of the best one's of up to 20 others.
static void cut_runs(const Ring& R, bool tc, int sweeps, int sums, Linear* p) {
  const int C = tc ? kLinTcChunk : kLinSimtChunk;
  // (off the tensor cores a chunk's slots are looked up one by one)
  const int half = R.zz ? R.T / R.cp / 2 : R.T;
  p->seg = tc && half % C ? half : R.T;
  p->per = (p->seg + C - 1) / C;
  p->nch = p->per * (R.T / p->seg);
  const double sum = tc ? 0.3 : 0.6, start = tc ? 1 : 0.15, fold = tc ? 0.25 : 0.1, launch = tc ? 2 : 0.5;
  const double heads = (double)R.B * R.Hq;
  double best = 0;
  for (int segs = 1; segs <= 64 && segs <= p->nch; ++segs) {
    const int cps = (p->nch + segs - 1) / segs;
    if ((p->nch + cps - 1) / cps != segs) continue;  // the same cut as a smaller number of runs
    double t = ceil(heads * sweeps * segs / kSms) * (cps + start + fold * (segs - 1) / 2);
    if (segs > 1) t += ceil(heads * sums * (segs - 1) / kSms) * (sum * cps + start) + launch;
    if (segs == 1 || t < best) {
      best = t;
      p->segs = segs;
      p->cps = cps;
    }
  }
}

static size_t up256(size_t n) { return (n + 255) / 256 * 256; }

// Workspace of a pass: the runs' sums, a copy of state_in (forward, where state_out takes its
// place), the heads' own dk and dv (backward, shared key heads).
struct LinearWs {
  size_t sums, state, part, total;
};
static LinearWs linear_ws(const Ring& R, const Linear& p, bool backward) {
  const size_t states = (size_t)R.B * R.Hq * R.D * R.D * sizeof(float);
  LinearWs w;
  w.sums = p.segs > 1 ? up256(states * p.segs) : 0;
  w.state = !backward && p.segs > 1 ? up256(states) : 0;
  w.part = backward && R.Hq != R.Hkv ? up256((size_t)R.B * R.Hq * R.T * R.D * sizeof(float)) : 0;
  w.total = backward ? 2 * w.sums + 2 * w.part : w.sums + w.state;
  if (w.total < 16) w.total = 16;
  return w;
}

static bool on_tensor_cores(const Ring& R) { return R.bf16 && linear_tc_supported(R); }

static void plan_linear(const cpattn_desc* d, const Ring& R, bool backward, bool tc, Linear* p) {
  *p = Linear{};
  p->B = R.B;
  p->Hq = R.Hq;
  p->Hkv = R.Hkv;
  p->T = R.T;
  p->D = R.D;
  p->bf16 = R.bf16;
  p->B_user = d->B;
  p->m = SeqMap::make(R.T, R.cp, R.zz);
  p->n_sweeps = backward ? 3 : 1;
  p->n_sums = backward ? 2 : 1;
  p->debug_fault = R.debug_fault;
  cut_runs(R, tc, p->n_sweeps, p->n_sums, p);
}

}  // namespace cpattn

using namespace cpattn;

extern "C" {

cpattn_status cpattn_rotate_fwd(const cpattn_rotate_desc* desc, const void* q,
                                const int64_t* q_strides, const void* k, const int64_t* k_strides,
                                const void* v, const int64_t* v_strides, const void* q_weight,
                                const void* k_weight, const double* inv_freq,
                                const int32_t* positions, void* q_out,
                                const int64_t* q_out_strides, void* k_out,
                                const int64_t* k_out_strides, void* v_out,
                                const int64_t* v_out_strides, void* stream) {
  Rotate p;
  cpattn_status s = validate_rotate(desc, &p);
  if (s != CPATTN_OK) return s;
  if (!view(p, q, q_strides, p.Hq, false, &p.in[0]) || !view(p, k, k_strides, p.Hkv, false, &p.in[1]) ||
      !view(p, q_out, q_out_strides, p.Hq, true, &p.out[0]) ||
      !view(p, k_out, k_out_strides, p.Hkv, true, &p.out[1]) || (v != nullptr) != (v_out != nullptr))
    return CPATTN_ERR_INVALID_ARG;
  if (v && (!view(p, v, v_strides, p.Hkv, false, &p.in[2]) || !view(p, v_out, v_out_strides, p.Hkv, true, &p.out[2])))
    return CPATTN_ERR_INVALID_ARG;
  if (!null_or_aligned(q_weight, 16) || !null_or_aligned(k_weight, 16) || !null_or_aligned(positions, 4) ||
      !null_or_aligned(inv_freq, 8) || (p.rot > 0 && !inv_freq))
    return CPATTN_ERR_INVALID_ARG;
  if (rotate_meet(p) || meet({q_out, k_out, v_out}, {q_weight, k_weight, inv_freq, positions})) return CPATTN_ERR_INVALID_ARG;
  p.w[0] = q_weight;
  p.w[1] = k_weight;
  p.inv_freq = inv_freq;
  p.positions = positions;
  cudaGetLastError();
  return from_cuda(launch_rotate_fwd(p, (cudaStream_t)stream));
}

size_t cpattn_rotate_bwd_workspace(const cpattn_rotate_desc* desc) {
  if (validate_rotate(desc, nullptr) != CPATTN_OK) return 0;
  return rotate_bwd_workspace(desc->D, desc->norm);
}

cpattn_status cpattn_rotate_bwd(const cpattn_rotate_desc* desc, const void* q,
                                const int64_t* q_strides, const void* k, const int64_t* k_strides,
                                const void* q_weight, const void* k_weight,
                                const double* inv_freq, const int32_t* positions,
                                const void* dq_out, const int64_t* dq_out_strides,
                                const void* dk_out, const int64_t* dk_out_strides,
                                const void* dv_out, const int64_t* dv_out_strides, void* dq,
                                const int64_t* dq_strides, void* dk, const int64_t* dk_strides,
                                void* dv, const int64_t* dv_strides, float* dq_weight,
                                float* dk_weight, void* workspace, size_t ws_bytes, void* stream) {
  Rotate p;
  cpattn_status s = validate_rotate(desc, &p);
  if (s != CPATTN_OK) return s;
  if (p.norm && (!view(p, q, q_strides, p.Hq, false, &p.x[0]) || !view(p, k, k_strides, p.Hkv, false, &p.x[1])))
    return CPATTN_ERR_INVALID_ARG;
  if (!view(p, dq_out, dq_out_strides, p.Hq, false, &p.in[0]) ||
      !view(p, dk_out, dk_out_strides, p.Hkv, false, &p.in[1]) ||
      !view(p, dq, dq_strides, p.Hq, true, &p.out[0]) || !view(p, dk, dk_strides, p.Hkv, true, &p.out[1]) ||
      (dv_out != nullptr) != (dv != nullptr))
    return CPATTN_ERR_INVALID_ARG;
  if (dv && (!view(p, dv_out, dv_out_strides, p.Hkv, false, &p.in[2]) ||
             !view(p, dv, dv_strides, p.Hkv, true, &p.out[2])))
    return CPATTN_ERR_INVALID_ARG;
  if (!null_or_aligned(q_weight, 16) || !null_or_aligned(k_weight, 16) || !null_or_aligned(positions, 4) ||
      !null_or_aligned(inv_freq, 8) || (p.rot > 0 && !inv_freq) || !null_or_aligned(dq_weight, 4) ||
      !null_or_aligned(dk_weight, 4) || (!p.norm && (dq_weight || dk_weight)))
    return CPATTN_ERR_INVALID_ARG;
  if (!aligned16(workspace) || ws_bytes < rotate_bwd_workspace(p.D, p.norm)) return CPATTN_ERR_INVALID_ARG;
  if (rotate_meet(p) || meet({dq, dk, dv, dq_weight, dk_weight, workspace}, {q_weight, k_weight, inv_freq, positions}) ||
      meet({dq_weight, dk_weight, workspace}, {q, k, dq_out, dk_out, dv_out}))
    return CPATTN_ERR_INVALID_ARG;
  p.w[0] = q_weight;
  p.w[1] = k_weight;
  p.inv_freq = inv_freq;
  p.positions = positions;
  p.sums = static_cast<float*>(workspace);
  cudaGetLastError();
  return from_cuda(launch_rotate_bwd(p, dq_weight, dk_weight, (cudaStream_t)stream));
}

size_t cpattn_linear_workspace(const cpattn_desc* desc) {
  Ring R;
  if (validate_linear(desc, &R) != CPATTN_OK) return 0;
  Linear p;
  plan_linear(desc, R, false, on_tensor_cores(R), &p);
  return linear_ws(R, p, false).total;
}

cpattn_status cpattn_linear_fwd(const cpattn_desc* desc, const void* q, const void* k,
                                const void* v, const float* log_decay, const int32_t* lengths,
                                const float* state_in, void* o, float* state_out, void* workspace,
                                size_t ws_bytes, void* stream) {
  Ring R;
  cpattn_status s = validate_linear(desc, &R);
  if (s != CPATTN_OK) return s;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned(log_decay, 4) ||
      !null_or_aligned(lengths, 4) || !null_or_aligned(state_in, 16) || !null_or_aligned(state_out, 16) ||
      !aligned16(workspace) || meet({o, state_out, workspace}, {q, k, v, log_decay, lengths}) ||
      meet({o, workspace}, {state_in}))
    return CPATTN_ERR_INVALID_ARG;
  const bool tc = on_tensor_cores(R);
  Linear p;
  plan_linear(desc, R, false, tc, &p);
  const LinearWs w = linear_ws(R, p, false);
  if (ws_bytes < w.total) return CPATTN_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  cudaGetLastError();
  char* ws = static_cast<char*>(workspace);
  p.log_decay = log_decay;
  p.lengths = lengths;
  p.status = status_ptr();
  if (state_in && state_in == state_out && p.segs > 1) {
    // other runs may still read what the last one replaces
    float* copy = reinterpret_cast<float*>(ws + w.sums);
    const size_t n = (size_t)R.B * R.Hq * R.D * R.D * sizeof(float);
    if (cudaMemcpyAsync(copy, state_in, n, cudaMemcpyDeviceToDevice, st) != cudaSuccess) return CPATTN_ERR_CUDA;
    state_in = copy;
  }
  const int rep = R.Hq / R.Hkv;
  LinSweep& f = p.sweep[0];
  f.a = q, f.b = k, f.c = v;
  f.rep_a = 1, f.rep_b = f.rep_c = rep;
  f.init = state_in, f.init_mul = 1.f;
  f.sums = reinterpret_cast<float*>(ws);
  f.mul = R.scale;
  f.out = o;
  f.fin = state_out, f.fin_mul = 1.f;
  f.exact = state_out != nullptr;
  p.sum[0] = f;
  return from_cuda(tc ? launch_linear_tc(p, st, false) : launch_linear_simt(p, st, false));
}

size_t cpattn_linear_bwd_workspace(const cpattn_desc* desc) {
  Ring R;
  if (validate_linear(desc, &R) != CPATTN_OK) return 0;
  Linear p;
  plan_linear(desc, R, true, on_tensor_cores(R), &p);
  return linear_ws(R, p, true).total;
}

cpattn_status cpattn_linear_bwd(const cpattn_desc* desc, const void* q, const void* k,
                                const void* v, const float* log_decay, const float* state_in,
                                const void* dO, const float* dstate_out, void* dq, void* dk,
                                void* dv, float* dstate_in, void* workspace, size_t ws_bytes,
                                void* stream) {
  Ring R;
  cpattn_status s = validate_linear(desc, &R);
  if (s != CPATTN_OK) return s;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(dO) || !aligned16(dq) ||
      !aligned16(dk) || !aligned16(dv) || !aligned(log_decay, 4) || !null_or_aligned(state_in, 16) ||
      !null_or_aligned(dstate_out, 16) || !null_or_aligned(dstate_in, 16) || !aligned16(workspace))
    return CPATTN_ERR_INVALID_ARG;
  if (meet({dq, dk, dv, dstate_in, workspace}, {q, k, v, log_decay, dO, state_in, dstate_out}))
    return CPATTN_ERR_INVALID_ARG;
  // the state's gradient is carried divided by the scale
  if (dstate_out && R.scale < 0x1p-64f) return CPATTN_ERR_UNSUPPORTED;
  const bool tc = on_tensor_cores(R);
  Linear p;
  plan_linear(desc, R, true, tc, &p);
  const LinearWs w = linear_ws(R, p, true);
  if (ws_bytes < w.total) return CPATTN_ERR_INVALID_ARG;
  cudaStream_t st = (cudaStream_t)stream;
  cudaGetLastError();
  char* ws = static_cast<char*>(workspace);
  p.log_decay = log_decay;
  p.status = status_ptr();
  const int rep = R.Hq / R.Hkv;
  float* sums_s = reinterpret_cast<float*>(ws);            // sums of k v^T from the front
  float* sums_r = reinterpret_cast<float*>(ws + w.sums);   // sums of q dO^T from the back
  float* part_v = reinterpret_cast<float*>(ws + 2 * w.sums);
  float* part_k = reinterpret_cast<float*>(ws + 2 * w.sums + w.part);
  LinSweep& fq = p.sweep[0];
  fq.a = dO, fq.b = v, fq.c = k;
  fq.rep_a = 1, fq.rep_b = fq.rep_c = rep;
  fq.init = state_in, fq.init_mul = 1.f;
  fq.trans = 1;
  fq.sums = sums_s;
  fq.mul = R.scale;
  fq.out = dq;
  // From the back M carries the state's gradient divided by the scale, which the outputs get.
  LinSweep& fv = p.sweep[1];
  fv.a = k, fv.b = q, fv.c = dO;
  fv.rep_a = rep, fv.rep_b = fv.rep_c = 1;
  fv.back = 1;
  fv.init = dstate_out, fv.init_mul = 1.f / R.scale;
  fv.sums = sums_r;
  fv.mul = R.scale;
  fv.out = rep > 1 ? part_v : dv;
  fv.out_f32 = rep > 1;
  fv.fin = dstate_in, fv.fin_mul = R.scale;
  fv.exact = dstate_in != nullptr;
  LinSweep& fk = p.sweep[2];
  fk = fv;
  fk.a = v, fk.b = dO, fk.c = q;
  fk.trans = 1;
  fk.out = rep > 1 ? part_k : dk;
  fk.fin = nullptr;
  fk.exact = 0;
  p.sum[0].b = k, p.sum[0].c = v;
  p.sum[0].rep_a = p.sum[0].rep_b = p.sum[0].rep_c = rep;
  p.sum[0].sums = sums_s;
  p.sum[1] = fv;
  cudaError_t e = tc ? launch_linear_tc(p, st, true) : launch_linear_simt(p, st, true);
  if (e != cudaSuccess || rep == 1) return from_cuda(e);
  const int64_t groups = (int64_t)R.B * R.Hkv, row = (int64_t)R.T * R.D;
  return from_cuda(launch_linear_group(groups, rep, row, part_v, part_k, dv, dk, R.bf16, st));
}

cpattn_status cpattn_linear_step(const cpattn_desc* desc, int n_states, const void* q,
                                 int64_t q_token_stride, int64_t q_head_stride, const void* k,
                                 int64_t k_token_stride, int64_t k_head_stride, const void* v,
                                 int64_t v_token_stride, int64_t v_head_stride,
                                 const float* log_decay, const int32_t* slots,
                                 const float* state_in, float* state_out, void* o, void* stream) {
  Ring R;
  cpattn_status s = validate_linear(desc, &R);
  if (s != CPATTN_OK) return s;
  if (desc->T != 1 || desc->cp != 1 || desc->a2a != 1 || n_states < 0) return CPATTN_ERR_INVALID_ARG;
  const int64_t vec = R.bf16 ? 8 : 4;
  auto rows = [&](const void* t, int64_t ts, int64_t hs, int heads) {
    return aligned16(t) && (R.B == 1 || (ts >= 0 && ts % vec == 0)) && (heads == 1 || (hs >= 0 && hs % vec == 0));
  };
  if (!rows(q, q_token_stride, q_head_stride, R.Hq) || !rows(k, k_token_stride, k_head_stride, R.Hkv) ||
      !rows(v, v_token_stride, v_head_stride, R.Hkv) || !aligned(log_decay, 4) || !null_or_aligned(slots, 4) ||
      !aligned16(state_in) || !aligned16(state_out) || !aligned16(o) || meet({o, state_out}, {q, k, v, log_decay, slots}) ||
      o == state_in)
    return CPATTN_ERR_INVALID_ARG;
  LinStep p;
  p.n = R.B;
  p.n_states = n_states;
  p.Hq = R.Hq;
  p.Hkv = R.Hkv;
  p.D = R.D;
  p.bf16 = R.bf16;
  p.scale = R.scale;
  p.q = q, p.k = k, p.v = v;
  p.q_ts = q_token_stride, p.q_hs = q_head_stride;
  p.k_ts = k_token_stride, p.k_hs = k_head_stride;
  p.v_ts = v_token_stride, p.v_hs = v_head_stride;
  p.log_decay = log_decay;
  p.slots = slots;
  p.in = state_in;
  p.out = state_out;
  p.o = o;
  cudaGetLastError();
  return from_cuda(launch_linear_step(p, (cudaStream_t)stream));
}

}  // extern "C"
