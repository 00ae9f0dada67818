// decay_step.cu - linear attention with a decay for each head, one new token
// of each sequence on its kept state (nats_decay_attn_step):
//   S <- e^g S + v k^T,  o = scale S q        (S [dv, dk] fp32, in place)
// Bound by HBM: a state is read and written once, 8 d^2 bytes a head.
// Measured on one GB300: 96 x 16 heads of d = 128, 35.4 us (5.7 TB/s; copy rate
// 6.7); 16 heads 4.7 us, the launch.
#include <cmath>

#include "../../include/nats.h"
#include "decay.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace nats {
namespace decay {
namespace {

constexpr int kInFlight = 8;  // 16-byte pieces of the state that a lane has in flight

struct StepArgs {
  Tokens q, k, v, o;
  const float* g;
  float* S;
  int H;
  float scale;
  int vec;  // q and k may be read four entries at a time
};

template <class T>
__device__ __forceinline__ float4 row4(const T* p, bool vec) {
  if (vec) {
    if constexpr (sizeof(T) == 4) {
      return *(const float4*)p;
    } else {
      const uint2 u = *(const uint2*)p;
      return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                         __uint_as_float(u.y & 0xffff0000u));
    }
  }
  return make_float4(to_f32(p[0]), to_f32(p[1]), to_f32(p[2]), to_f32(p[3]));
}

// A state's row of d entries lies across d / 4 lanes; a warp takes
// kInFlight * 128 / d rows, all of them in flight before the first is used.
template <class T, int D>
__global__ void __launch_bounds__(256) step_kernel(const StepArgs a) {
  begin();
  constexpr int kLanes = D / 4, kSide = 32 / kLanes, kRows = kInFlight * kSide;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (blockDim.x >> 5) * kRows;  // rows of a CTA
  const long long bh = blockIdx.x / (D / per);
  const int r0 = (blockIdx.x % (D / per)) * per + warp * kRows + lane / kLanes;
  const int c = (lane % kLanes) * 4;
  const int b = (int)(bh / a.H), h = (int)(bh % a.H);
  float* S = a.S + bh * D * D + (long long)r0 * D + c;
  float4 s[kInFlight];
#pragma unroll
  for (int i = 0; i < kInFlight; ++i) s[i] = *(const float4*)(S + i * kSide * D);
  const float4 q = row4((const T*)a.q.p + b * a.q.b + h * a.q.h + c, a.vec & 1);
  const float4 k = row4((const T*)a.k.p + b * a.k.b + h * a.k.h + c, a.vec & 1);
  const T* v = (const T*)a.v.p + b * a.v.b + h * a.v.h + r0;
  float w[kInFlight];
#pragma unroll
  for (int i = 0; i < kInFlight; ++i) w[i] = to_f32(v[i * kSide]);
  const Carry carry(a.g[h], 1);
  float o[kInFlight];
#pragma unroll
  for (int i = 0; i < kInFlight; ++i) {
    s[i].x = carry(s[i].x, w[i] * k.x), s[i].y = carry(s[i].y, w[i] * k.y);
    s[i].z = carry(s[i].z, w[i] * k.z), s[i].w = carry(s[i].w, w[i] * k.w);
    *(float4*)(S + i * kSide * D) = s[i];
    o[i] = fmaf(s[i].x, q.x, fmaf(s[i].y, q.y, fmaf(s[i].z, q.z, s[i].w * q.w)));
  }
#pragma unroll
  for (int x = kLanes / 2; x > 0; x >>= 1)
#pragma unroll
    for (int i = 0; i < kInFlight; ++i) o[i] += __shfl_xor_sync(0xffffffffu, o[i], x);
  // lane i of each row's lanes writes the i-th of its rows
  T* out = (T*)a.o.p + b * a.o.b + h * a.o.h + r0;
#pragma unroll
  for (int i = 0; i < kInFlight; ++i)
    if (lane % kLanes == i) out[i * kSide] = from_f32<T>(a.scale * o[i]);
}

template <class T, int D>
cudaError_t launch(const StepArgs& a, long long heads, cudaStream_t st) {
  constexpr int kRows = kInFlight * 32 / (D / 4);
  // few heads: two warps to a CTA, so that more SMs have a part
  int warps = D / kRows < 8 ? D / kRows : 8;
  if (heads * D / (warps * kRows) < kSMs) warps = 2;
  return after(step_kernel<T, D>, (unsigned)(heads * (D / (warps * kRows))), dim3(32 * warps), 0, st, 0, a);
}

}  // namespace
}  // namespace decay
}  // namespace nats

using namespace nats;
using namespace nats::decay;

extern "C" nats_status nats_decay_attn_step(const nats_decay_dims* dims, const void* q, const nats_strides* q_st,
                                            const void* k, const nats_strides* k_st, const void* v,
                                            const nats_strides* v_st, const float* log_decay, float* state, void* out,
                                            const nats_strides* out_st, nats_stream_t stream) {
  const nats_status s = check_dims(dims);
  if (s != NATS_OK) return s;
  if (dims->L != 1) return NATS_ERR_SHAPE;
  if (dims->B == 0 || dims->H == 0) return NATS_OK;
  if (!q || !q_st || !k || !k_st || !v || !v_st || !log_decay || !state || !out || !out_st) return NATS_ERR_NULL;
  const int es = dims->dtype == NATS_BF16 ? 2 : 4;
  for (const void* p : {q, k, v, (const void*)out})
    if ((uintptr_t)p & (uintptr_t)(es - 1)) return NATS_ERR_ALIGN;
  if (((uintptr_t)log_decay & 3u) || ((uintptr_t)state & 15u)) return NATS_ERR_ALIGN;
  StepArgs a = {tokens(q, q_st), tokens(k, k_st), tokens(v, v_st), tokens(out, out_st), log_decay, state, dims->H,
                dims->scale > 0.f ? dims->scale : 1.0f / std::sqrt((float)dims->d),
                rows_at(tokens(q, q_st), dims, 4 * es) && rows_at(tokens(k, k_st), dims, 4 * es)};
  const long long heads = (long long)dims->B * dims->H;
  cudaStream_t st = (cudaStream_t)stream;
  cudaError_t e;
  if (dims->dtype == NATS_BF16)
    e = dims->d == 64 ? launch<__nv_bfloat16, 64>(a, heads, st) : launch<__nv_bfloat16, 128>(a, heads, st);
  else
    e = dims->d == 64 ? launch<float, 64>(a, heads, st) : launch<float, 128>(a, heads, st);
  return (nats_status)record_cuda_error(e);
}
