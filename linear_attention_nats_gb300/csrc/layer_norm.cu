// layer_norm.cu - layer norm of rows of D entries (nats_layer_norm) and its
// gradient (nats_layer_norm_bwd):
//   z = (x - mean(x)) r,  r = 1 / sqrt(mean((x - mean(x))^2) + eps),  y = w z + b
//   with u the gradient of y and t = w u:
//   dx = r (t - mean(t) - z mean(t z)),  dw = sum over rows of u z,  db = sum of u
// Bound by HBM: a row is held in the registers of a group of G threads, so it
// is read once and its statistics take two passes over registers (the mean,
// then the squared distances from it: no cancellation for rows far from zero).
// The gradient forms mean and r again from x, which it reads anyway, so the
// forward has nothing to keep.
#include <cmath>

#include "../../include/nats.h"
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace nats {
namespace {

constexpr int kSMs = 152;
constexpr int kMaxD = 16384;
constexpr int kBwdCtas = 4 * kSMs;  // rows of partial sums that the workspace holds

struct Rows {
  char* p;
  long long b, h, t;  // bytes between the outer, middle and inner rows
};
struct NormArgs {
  Rows x, y, u;  // bwd: y is dx, u the gradient of the output
  const float *w, *bias;
  float* part;  // [CTAs, 2, D]
  int rows, H, L, D;
  float eps, inv_d;
};

__device__ __forceinline__ char* row_at(const Rows& r, const NormArgs& a, int i) {
  const int t = i % a.L, bh = i / a.L;
  return r.p + (bh / a.H) * r.b + (bh % a.H) * r.h + t * r.t;
}

// VEC entries of a row, read or written at once.
template <class T, int VEC>
struct Piece;
template <>
struct Piece<float, 4> {
  float4 r;
  __device__ __forceinline__ void zero() { r = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) { r = *(const float4*)p; }
  __device__ __forceinline__ float operator[](int e) const { return e == 0 ? r.x : e == 1 ? r.y : e == 2 ? r.z : r.w; }
  static __device__ __forceinline__ void store(float* p, const float (&v)[4]) {
    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Piece<__nv_bfloat16, 8> {
  uint4 r;
  __device__ __forceinline__ void zero() { r = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *(const uint4*)p; }
  __device__ __forceinline__ float operator[](int e) const {
    const uint32_t x = e < 2 ? r.x : e < 4 ? r.y : e < 6 ? r.z : r.w;
    return __uint_as_float(e & 1 ? x & 0xffff0000u : x << 16);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[8]) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      u[i] = *(const uint32_t*)&h;
    }
    *(uint4*)p = make_uint4(u[0], u[1], u[2], u[3]);
  }
};
template <class T>
struct Piece<T, 1> {
  T r;
  __device__ __forceinline__ void zero() { r = from_f32<T>(0.f); }
  __device__ __forceinline__ void load(const T* p) { r = *p; }
  __device__ __forceinline__ float operator[](int) const { return to_f32(r); }
  static __device__ __forceinline__ void store(T* p, const float (&v)[1]) { *p = from_f32<T>(v[0]); }
};

// Sums of N numbers over the G threads of a row, left in all of them; a group
// is part of a warp or a whole CTA.  `flip` changes from call to call, so that
// one barrier a sum is enough.
template <int G, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], float* sm, int& flip) {
#pragma unroll
  for (int x = (G < 32 ? G : 32) / 2; x > 0; x >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], x);
  if constexpr (G > 32) {
    constexpr int W = G / 32;
    float* s = sm + flip * 2 * W;
    flip ^= 1;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
      for (int i = 0; i < N; ++i) s[i * W + (threadIdx.x >> 5)] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = s[i * W];
#pragma unroll
      for (int j = 1; j < W; ++j) t += s[i * W + j];
      v[i] = t;
    }
  }
}

// Thread j of a group holds pieces j, j + G, .. of its row, NV of them.
template <class T, int VEC, int G, int NV>
__global__ void __launch_bounds__(G < 128 ? 128 : G) norm_kernel(const NormArgs a) {
  begin();
  constexpr int kBlock = G < 128 ? 128 : G, kGroups = kBlock / G;
  __shared__ float sm[G > 32 ? 4 * (G / 32) : 1];
  int flip = 0;
  const int j = threadIdx.x % G;
  const long long at = (long long)blockIdx.x * kGroups + threadIdx.x / G;
  const bool live = at < a.rows;
  const int row = live ? (int)at : a.rows - 1;
  const T* x = (const T*)row_at(a.x, a, row);
  Piece<T, VEC> in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + j) * VEC;
    if (c < a.D) in[i].load(x + c);
    else in[i].zero();
  }
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[0] += in[i][e];
  group_sum<G>(s, sm, flip);
  const float mean = s[0] * a.inv_d;
  s[0] = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    if ((i * G + j) * VEC < a.D)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float d = in[i][e] - mean;
        s[0] = fmaf(d, d, s[0]);
      }
  group_sum<G>(s, sm, flip);
  const float r = 1.f / sqrtf(fmaf(s[0], a.inv_d, a.eps));
  if (!live) return;
  T* y = (T*)row_at(a.y, a, row);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + j) * VEC;
    if (c >= a.D) continue;
    float v[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      v[e] = (in[i][e] - mean) * r;
      const float w = a.w ? a.w[c + e] : 1.f, bias = a.bias ? a.bias[c + e] : 0.f;
      v[e] = fmaf(v[e], w, bias);
    }
    Piece<T, VEC>::store(y + c, v);
  }
}

// The gradient: a CTA takes rows blockIdx.x kGroups + group, a grid further on
// each time, the next row's pieces in flight while one is worked on; every
// thread sums its own columns' parts of dw and db in registers, the groups of
// a CTA are added in order, and norm_dw_kernel adds the CTAs'.
template <class T, int VEC, int G, int NV>
__global__ void __launch_bounds__(G < 128 ? 128 : G) norm_bwd_kernel(const NormArgs a) {
  begin();
  constexpr int kBlock = G < 128 ? 128 : G, kGroups = kBlock / G;
  __shared__ float sm[G > 32 ? 4 * (G / 32) : 1];
  int flip = 0;
  const int j = threadIdx.x % G;
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const int c = (i * G + j) * VEC + e;
      w[i][e] = a.w && c < a.D ? a.w[c] : 1.f;
      dw[i][e] = db[i][e] = 0.f;
    }
  Piece<T, VEC> nx[NV], nu[NV];
  const auto fetch = [&](long long at) {
    const int row = at < a.rows ? (int)at : a.rows - 1;
    const T *x = (const T*)row_at(a.x, a, row), *u = (const T*)row_at(a.u, a, row);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * G + j) * VEC;
      if (c < a.D) {
        nx[i].load(x + c), nu[i].load(u + c);
      } else {
        nx[i].zero(), nu[i].zero();
      }
    }
  };
  const long long step = (long long)gridDim.x * kGroups;
  const long long first = (long long)blockIdx.x * kGroups;
  if (first < a.rows) fetch(first + threadIdx.x / G);
  // (all groups of a CTA go round alike: those behind the last row work on it again, and drop the result)
  for (long long base = first; base < a.rows; base += step) {
    const long long at = base + threadIdx.x / G;
    const bool live = at < a.rows;
    Piece<T, VEC> in[NV], gu[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) in[i] = nx[i], gu[i] = nu[i];
    if (base + step < a.rows) fetch(at + step);
    float s[1] = {0.f};
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[0] += in[i][e];
    group_sum<G>(s, sm, flip);
    const float mean = s[0] * a.inv_d;
    s[0] = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * G + j) * VEC < a.D)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float d = in[i][e] - mean;
          s[0] = fmaf(d, d, s[0]);
        }
    group_sum<G>(s, sm, flip);
    const float r = 1.f / sqrtf(fmaf(s[0], a.inv_d, a.eps));
    float m[2] = {0.f, 0.f};  // sums of t and t z
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float z = (in[i][e] - mean) * r, u = gu[i][e], t = u * w[i][e];
        m[0] += t;
        m[1] = fmaf(t, z, m[1]);
        if (live) dw[i][e] = fmaf(u, z, dw[i][e]), db[i][e] += u;
      }
    group_sum<G>(m, sm, flip);
    m[0] *= a.inv_d, m[1] *= a.inv_d;
    if (!live) continue;
    T* y = (T*)row_at(a.y, a, (int)at);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * G + j) * VEC;
      if (c >= a.D) continue;
      float v[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float z = (in[i][e] - mean) * r;
        v[e] = r * (fmaf(gu[i][e], w[i][e], -m[0]) - z * m[1]);
      }
      Piece<T, VEC>::store(y + c, v);
    }
  }
  if (!a.part) return;
  float* part = a.part + (long long)blockIdx.x * 2 * a.D;
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int c = (i * G + j) * VEC + e;
        if (c < a.D) part[c] = dw[i][e], part[a.D + c] = db[i][e];
      }
  } else {
    __shared__ float acc[2][G * NV * VEC];
    for (int g = 0; g < kGroups; ++g) {
      if ((int)threadIdx.x / G == g)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const int c = (i * G + j) * VEC + e;
            acc[0][c] = g ? acc[0][c] + dw[i][e] : dw[i][e];
            acc[1][c] = g ? acc[1][c] + db[i][e] : db[i][e];
          }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.D; c += kBlock) part[c] = acc[0][c], part[a.D + c] = acc[1][c];
  }
}

// dw and db: 32 columns a CTA, 32 threads a column over the CTAs' sums.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* __restrict__ part, int n, int D, float* dw, float* db) {
  begin();
  __shared__ float sm[32][33];
  const int c = blockIdx.x * 32 + threadIdx.x;  // of [dw | db]
  float s = 0.f;
  if (c < 2 * D)
    for (int i = threadIdx.y; i < n; i += 32) s += part[(long long)i * 2 * D + c];
  sm[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  const float t = warp_sum(sm[threadIdx.x][threadIdx.y]);
  const int o = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && o < 2 * D) {
    float* out = o < D ? dw : db;
    if (out) out[o < D ? o : o - D] = t;
  }
}

// ----------------------------------------------------------------- launches

template <class T, int VEC, int G, int NV>
cudaError_t go(const NormArgs& a, bool bwd, int* ctas, cudaStream_t st) {
  constexpr int kBlock = G < 128 ? 128 : G, kGroups = kBlock / G;
  const long long need = ((long long)a.rows + kGroups - 1) / kGroups;
  if (!bwd) return after(norm_kernel<T, VEC, G, NV>, (unsigned)need, dim3(kBlock), 0, st, 0, a);
  *ctas = (int)(need < kBwdCtas ? need : kBwdCtas);
  return after(norm_bwd_kernel<T, VEC, G, NV>, (unsigned)*ctas, dim3(kBlock), 0, st, 0, a);
}

// Threads and pieces of a row by its length: short rows share a warp, long
// ones take a CTA.
template <class T>
cudaError_t choose(const NormArgs& a, bool vec, bool bwd, int* ctas, cudaStream_t st) {
  constexpr int V = sizeof(T) == 2 ? 8 : 4;
  const int n = vec ? a.D / V : a.D;
#define NATS_NORM(VEC, G, NV) \
  if (n <= (G) * (NV)) return go<T, VEC, G, NV>(a, bwd, ctas, st)
  if (vec) {
    NATS_NORM(V, 8, 1);
    NATS_NORM(V, 16, 1);
    NATS_NORM(V, 32, 1);
    NATS_NORM(V, 32, 2);
    NATS_NORM(V, 128, 1);
    NATS_NORM(V, 256, 1);
    NATS_NORM(V, 512, 1);
    NATS_NORM(V, 512, 2);
    NATS_NORM(V, 512, 4);
    if constexpr (V == 4) NATS_NORM(V, 512, 8);
  } else {
    NATS_NORM(1, 32, 2);
    NATS_NORM(1, 32, 8);
    NATS_NORM(1, 128, 8);
    NATS_NORM(1, 512, 4);
    NATS_NORM(1, 512, 8);
    NATS_NORM(1, 512, 32);
  }
#undef NATS_NORM
  return cudaErrorInvalidValue;
}

nats_status check_norm(const nats_norm_dims* d) {
  if (!d) return NATS_ERR_NULL;
  if (d->dtype != NATS_BF16 && d->dtype != NATS_F32) return NATS_ERR_DTYPE;
  if (d->B < 0 || d->H < 0 || d->L < 0 || d->D < 1) return NATS_ERR_SHAPE;
  if (d->D > kMaxD || (double)d->B * d->H * d->L > 2147483647.0) return NATS_ERR_UNSUPPORTED;
  if (!std::isfinite(d->eps) || d->eps < 0.f) return NATS_ERR_VALUE;
  return NATS_OK;
}

bool elem_ok(const void* p, int es) { return ((uintptr_t)p & (uintptr_t)(es - 1)) == 0; }

Rows rows_of(const void* p, const nats_strides* st, int es) {
  return {(char*)const_cast<void*>(p), st->b * es, st->h * es, st->t * es};
}
bool vec_ok(const Rows& r, const nats_norm_dims* d) {
  return elem_ok(r.p, 16) && (d->B == 1 || r.b % 16 == 0) && (d->H == 1 || r.h % 16 == 0) && (d->L == 1 || r.t % 16 == 0);
}

}  // namespace
}  // namespace nats

using namespace nats;

extern "C" {

nats_status nats_layer_norm(const nats_norm_dims* dims, const void* x, const nats_strides* x_st, const float* w,
                            const float* b, void* out, const nats_strides* out_st, nats_stream_t stream) {
  const nats_status s = check_norm(dims);
  if (s != NATS_OK) return s;
  if (dims->B == 0 || dims->H == 0 || dims->L == 0) return NATS_OK;
  if (!x || !x_st || !out || !out_st) return NATS_ERR_NULL;
  const int es = dims->dtype == NATS_BF16 ? 2 : 4;
  if (!elem_ok(x, es) || !elem_ok(out, es) || !elem_ok(w, 4) || !elem_ok(b, 4)) return NATS_ERR_ALIGN;
  NormArgs a = {};
  a.x = rows_of(x, x_st, es), a.y = rows_of(out, out_st, es);
  a.w = w, a.bias = b;
  a.rows = dims->B * dims->H * dims->L, a.H = dims->H, a.L = dims->L, a.D = dims->D;
  a.eps = dims->eps, a.inv_d = 1.f / dims->D;
  const bool vec = dims->D % (16 / es) == 0 && vec_ok(a.x, dims) && vec_ok(a.y, dims);
  cudaStream_t st = (cudaStream_t)stream;
  return (nats_status)record_cuda_error(es == 2 ? choose<__nv_bfloat16>(a, vec, false, nullptr, st)
                                                : choose<float>(a, vec, false, nullptr, st));
}

size_t nats_layer_norm_bwd_workspace_size(const nats_norm_dims* dims) {
  if (check_norm(dims) != NATS_OK) return 0;
  const long long rows = (long long)dims->B * dims->H * dims->L;
  return sizeof(float) * 2 * dims->D * (size_t)(rows < kBwdCtas ? rows : kBwdCtas);
}

nats_status nats_layer_norm_bwd(const nats_norm_dims* dims, const void* dout, const nats_strides* dout_st, const void* x,
                                const nats_strides* x_st, const float* w, void* dx, const nats_strides* dx_st, float* dw,
                                float* db, void* workspace, size_t workspace_bytes, nats_stream_t stream) {
  const nats_status s = check_norm(dims);
  if (s != NATS_OK) return s;
  const int es = dims->dtype == NATS_BF16 ? 2 : 4;
  const bool empty = dims->B == 0 || dims->H == 0 || dims->L == 0;
  if (!empty && (!dout || !dout_st || !x || !x_st || !dx || !dx_st)) return NATS_ERR_NULL;
  if (!elem_ok(dout, es) || !elem_ok(x, es) || !elem_ok(dx, es) || !elem_ok(w, 4) || !elem_ok(dw, 4) || !elem_ok(db, 4))
    return NATS_ERR_ALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  if (empty) {
    for (float* o : {dw, db})
      if (o) {
        const int r = record_cuda_error(cudaMemsetAsync(o, 0, sizeof(float) * dims->D, st));
        if (r != NATS_OK) return (nats_status)r;
      }
    return NATS_OK;
  }
  const bool sums = dw || db;
  if (sums) {
    if (!workspace) return NATS_ERR_NULL;
    if (!elem_ok(workspace, 16)) return NATS_ERR_ALIGN;
    if (workspace_bytes < nats_layer_norm_bwd_workspace_size(dims)) return NATS_ERR_WORKSPACE;
  }
  NormArgs a = {};
  a.x = rows_of(x, x_st, es), a.y = rows_of(dx, dx_st, es), a.u = rows_of(dout, dout_st, es);
  a.w = w, a.part = sums ? (float*)workspace : nullptr;
  a.rows = dims->B * dims->H * dims->L, a.H = dims->H, a.L = dims->L, a.D = dims->D;
  a.eps = dims->eps, a.inv_d = 1.f / dims->D;
  const bool vec = dims->D % (16 / es) == 0 && vec_ok(a.x, dims) && vec_ok(a.y, dims) && vec_ok(a.u, dims);
  int ctas = 0;
  const int r = record_cuda_error(es == 2 ? choose<__nv_bfloat16>(a, vec, true, &ctas, st)
                                          : choose<float>(a, vec, true, &ctas, st));
  if (r != NATS_OK || !sums) return (nats_status)r;
  const float* part = a.part;
  return (nats_status)record_cuda_error(after(norm_dw_kernel, (unsigned)((2 * dims->D + 31) / 32), dim3(32, 32), 0, st, 0,
                                              part, ctas, (int)dims->D, dw, db));
}

}  // extern "C"
