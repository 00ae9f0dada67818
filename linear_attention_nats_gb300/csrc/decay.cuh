// decay.cuh - linear attention with a decay for each head, as its kernels see
// it: one scan over a sequence,
//
//   forward in time:  S_t = gamma S_(t-1) + k_t v_t^T,   o_t = scale S_t^T q_t,
//   backward in time: the same from the last token down.
//
// The three gradients are scans of the same kind (u the output's gradient, R
// the state's, running backward from the last state's gradient):
//   dq_t = scale S_t u_t            keys v, values k, queries u, forward
//   dk_t = R_t^T v_t,  dv_t = R_t k_t,  R_t = scale u_t q_t^T + gamma R_(t+1):
//                                   keys u / q, values q / u, queries v / k
// so a training step is three scans in one launch.  A state's rows go with the
// scan's keys, its columns with the values.  R takes the scale with what is
// added to it and is read without, so that the gradients of the states go in
// and out as they are, whatever the scale: with x = 1 and y = scale, and the
// other way round in these two scans,
//
// A chunk of n tokens, i its i-th in the scan's order, takes
//   o_i = scale sum_(j <= i) gamma^(i - j) (q_i k_j) v_j + y gamma^(i + 1 - e) S^T q_i
//   S  <- gamma^n S + x sum_j gamma^(n - 1 - j + e) k_j v_j^T
// with e = 0 forward; e = 1 backward, where the state that is carried is the
// gradient of the chunk's first state (one decay further), so that no factor
// is ever divided by gamma.  All exponents are >= 0: no decay, however fast,
// overflows, and gamma = 0 (a log decay of -inf) leaves each token itself.
#pragma once

#include <stdint.h>

#include "../../include/nats.h"
#include "common.cuh"

namespace nats {
namespace decay {

constexpr int kSMs = 152;
constexpr int kWidth = 64;    // state columns of one CTA
constexpr int kMaxOps = 3;    // scans of one launch
constexpr int kMaxSegs = 64;  // parts of a sequence

// A [B, H, L, d] operand.
struct Tokens {
  void* p;
  long long b, h, t;  // elements between sequences, heads, tokens
};

struct Op {
  Tokens q, k, v, o;
  const float* s_in;  // [B, H, d, d] or NULL (zero)
  float* s_out;       // or NULL
  long long s_r, s_c; // elements between a state's rows, columns
  int scaled;         // the state takes the scale with what is added to it, and is read without
  float* part;        // [B H, segs, d, d]: the state ahead of each segment (columns outermost), with segs > 1
  int part_t;         // part belongs to another scan, whose rows are this one's columns
  int back;
};

struct Args {
  Op op[kMaxOps];
  const float* g;       // [H] log decay
  const int32_t* lens;  // [B] or NULL
  int nops;
  int B, H, L;
  float scale;
  int segs, seg;        // segments of a sequence, tokens of each (in the scan's order, counted from token 0 in both)
  int first_op, last_op;  // the scans of this launch
  int vec;              // operands may be read and written four entries at a time (decay_attn.cu)
  int expire;           // the chunk whose values one warp takes for overdue (nats_debug_decay_wait); -1: none
};

// gamma^m; 1 for m = 0 whatever gamma is.
__device__ __forceinline__ float power(float g, int m) { return m == 0 ? 1.f : expf(g * (float)m); }

__device__ __forceinline__ int length(const Args& a, int b) {
  if (!a.lens) return a.L;
  const int n = a.lens[b];
  return n < 0 ? 0 : n < a.L ? n : a.L;
}

// gamma^n S + add, for the state that goes from chunk to chunk.  gamma^n of a
// slow decay is close to 1, and its rounding, the same in every chunk, would
// add up over a long sequence: expm1(g n) holds its distance from 1.  A fast
// decay's distance from 1 would round away what is left.
struct Carry {
  float m;
  bool slow;
  __device__ __forceinline__ Carry(float g, int n) {
    const float x = n == 0 ? 0.f : g * (float)n;
    slow = x > -0.5f;
    m = slow ? expm1f(x) : expf(x);
  }
  __device__ __forceinline__ float operator()(float S, float add) const {
    return fmaf(S, m, slow ? S : 0.f) + add;
  }
};

// ------------------------------------------------------------- host side
nats_status check_dims(const nats_decay_dims* m);
inline Tokens tokens(const void* p, const nats_strides* st) { return {const_cast<void*>(p), st->b, st->h, st->t}; }
// Whether every row starts at a multiple of `bytes`.
inline bool rows_at(const Tokens& x, const nats_decay_dims* m, int bytes) {
  const int n = bytes / (m->dtype == NATS_BF16 ? 2 : 4);
  return ((uintptr_t)x.p & (uintptr_t)(bytes - 1)) == 0 && (m->B == 1 || x.b % n == 0) && (m->H == 1 || x.h % n == 0) &&
         (m->L == 1 || x.t % n == 0);
}

// The bf16 scans on the tensor cores (decay_attn_tc.cu).
cudaError_t launch_tc(const Args& a, int d, bool states_only, cudaStream_t st);
// Whether a bounded wait of theirs has expired on this device since the last question (synchronises st).
cudaError_t expired_waits(int* out, cudaStream_t st);

}  // namespace decay
}  // namespace nats
