// layer_norm.cu - layer norm of rows of D entries (nats_layer_norm) and its
// gradient (nats_layer_norm_bwd):
//   z = (x - mean(x)) r,  r = 1 / sqrt(mean((x - mean(x))^2) + eps),  y = w z + b
//   with u the gradient of y and t = w u:
//   dx = r (t - mean(t) - z mean(t z)),  dw = sum over rows of u z,  db = sum of u
// Bound by HBM: a row is held in the registers of a group of G threads, so it
// is read once and its statistics take two passes over registers (a first mean,
// then the distances from it and their squares: no cancellation for rows far from
// zero, and a mean that is off by its own rounding alone).
// The gradient forms mean and r again from x, which it reads anyway, so the
// forward has nothing to keep.
//
// Measured on one GB300 (HBM copy rate 6.7 TB/s): 32,768 rows of 2048, bf16,
// forward 47 us (5.7 TB/s), gradient 81 us (5.0 TB/s) with its weights' sums;
// fp32 79 us (6.8) and 143 us (5.6).  524,288 rows of 64, bf16: 31 and 49 us.
// Odd rows, entry by entry (32,768 of 2047): 129 and 132 us.
#include <atomic>
#include <cmath>
#include <type_traits>

#include "../../include/nats.h"
#include "common.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "tc.cuh"

namespace nats {
namespace {

constexpr int kSMs = 152;
constexpr int kMaxD = 16384;
constexpr int kBwdCtas = 8 * kSMs;  // most CTAs of the gradient: rows of partial sums that the workspace holds

struct Rows {
  char* p;
  long long b, h, t;  // bytes between the outer, middle and inner rows
};
struct NormArgs {
  Rows x, y, u;  // bwd: y is dx, u the gradient of the output
  const float *w, *bias;
  float* part;  // [CTAs, 2, D]
  int rows, H, L, D;
  int flat;  // rows follow one another at one stride
  float eps, inv_d;
};

struct Row {
  int b, h, t;
};
__device__ __forceinline__ Row row_of(const NormArgs& a, int i) {
  if (a.flat) return {0, 0, i};
  const int bh = i / a.L;
  return {bh / a.H, bh % a.H, i - bh * a.L};
}
__device__ __forceinline__ char* row_at(const Rows& r, const Row& i) { return r.p + i.b * r.b + i.h * r.h + i.t * r.t; }

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
template <>
struct Piece<__nv_bfloat16, 2> {
  uint32_t r;
  __device__ __forceinline__ void zero() { r = 0; }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = *(const uint32_t*)p; }
  __device__ __forceinline__ float operator[](int e) const { return __uint_as_float(e ? r & 0xffff0000u : r << 16); }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&v)[2]) {
    *(__nv_bfloat162*)p = __floats2bfloat162_rn(v[0], v[1]);
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
// is part of a warp or whole warps of the CTA.  `sm` is the group's own; `flip`
// changes from call to call, so that one barrier a sum is enough.
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
      for (int i = 0; i < N; ++i) s[i * W + (threadIdx.x % G >> 5)] = v[i];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + (int)threadIdx.x / G), "n"(G) : "memory");
#pragma unroll
    for (int i = 0; i < N; ++i) {
      float t = s[i * W];
#pragma unroll
      for (int j = 1; j < W; ++j) t += s[i * W + j];
      v[i] = t;
    }
  }
}
template <int G>
constexpr int kSums = G > 32 ? 4 * (G / 32) : 1;  // floats of a group's sums

// VEC consecutive weights.
template <int VEC>
__device__ __forceinline__ void weights(const float* p, float (&w)[VEC], float none) {
#pragma unroll
  for (int e = 0; e < VEC; ++e) w[e] = none;
  if (!p) return;
  if constexpr (VEC % 4 == 0) {
#pragma unroll
    for (int e = 0; e < VEC; e += 4) {
      const float4 x = *(const float4*)(p + e);
      w[e] = x.x, w[e + 1] = x.y, w[e + 2] = x.z, w[e + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[e] = p[e];
  }
}

// Entries 2 k and 2 k + 1 of a thread's own, as a pair for the packed fp32
// instructions (one for both).
template <int K, class T, int VEC, int NV>
__device__ __forceinline__ uint64_t pair_of(const Piece<T, VEC> (&in)[NV]) {
  return tc::f2_pack(in[2 * K / VEC][2 * K % VEC], in[(2 * K + 1) / VEC][(2 * K + 1) % VEC]);
}
__device__ __forceinline__ uint64_t both(float x) { return tc::f2_pack(x, x); }
__device__ __forceinline__ float sum_of(uint64_t v) {
  float a, b;
  tc::f2_unpack(v, a, b);
  return a + b;
}
template <int N, class F>
__device__ __forceinline__ void each(F&& f) {
  if constexpr (N > 0) {
    each<N - 1>(f);
    f(std::integral_constant<int, N - 1>{});
  }
}

// The mean of a row from a first one and the mean of the distances from that
// (a sum of D entries far from zero is some of their last places off, as much as
// the entries of a row of one value differ from its mean, whose z is 0: without
// this, up to 0.97 for fp32 values of 1e3 to 1e5), and the variance from their mean
// and their squares'.  It costs 1 % of the forward's time, 3 % of the gradient's
// (32,768 rows of 2048, bf16: 46.1 -> 46.5 us, 78.1 -> 80.6).
__device__ __forceinline__ float2 corrected(float mean, float d, float d2, float inv_d) {
  const float by = d * inv_d;
  return make_float2(mean + by, fmaxf(fmaf(d2, inv_d, -by * by), 0.f));
}

// The mean and 1 / standard deviation of the row whose pieces a group holds
// (zero behind its end).
template <bool FULL, class T, int VEC, int G, int NV>
__device__ __forceinline__ float2 statistics(const Piece<T, VEC> (&in)[NV], const NormArgs& a, int j, float* sm, int& flip) {
  constexpr int kPairs = NV * VEC / 2;
  uint64_t t[2] = {0, 0};
  each<kPairs>([&](auto k) { t[k % 2] = tc::f2_add(t[k % 2], pair_of<k>(in)); });
  float s[1] = {sum_of(tc::f2_add(t[0], t[1]))};
  group_sum<G>(s, sm, flip);
  const float mean = s[0] * a.inv_d;
  const uint64_t less = both(-mean);
  uint64_t l = 0;
  t[0] = t[1] = 0;
  each<kPairs>([&](auto k) {
    uint64_t d = tc::f2_add(pair_of<k>(in), less);
    if constexpr (VEC == 1) {
      float x, y;
      tc::f2_unpack(d, x, y);
      d = tc::f2_pack(2 * k * G + j < a.D ? x : 0.f, (2 * k + 1) * G + j < a.D ? y : 0.f);
    } else if (!FULL && (2 * k / VEC * G + j) * VEC >= a.D) {
      d = 0;
    }
    t[k % 2] = tc::f2_fma(d, d, t[k % 2]);
    l = tc::f2_add(l, d);
  });
  float s2[2] = {sum_of(l), sum_of(tc::f2_add(t[0], t[1]))};
  group_sum<G>(s2, sm, flip);
  const float2 st = corrected(mean, s2[0], s2[1], a.inv_d);
  return make_float2(st.x, 1.f / sqrtf(st.y + a.eps));
}

// Thread j of a group holds pieces j, j + G, .. of its R rows, NV of each; the
// weights are read once for all of them.
template <bool FULL, class T, int VEC, int G, int NV, int R>
__global__ void __launch_bounds__(G < 128 ? 128 : G) norm_kernel(const NormArgs a) {
  begin();
  __shared__ float sums[G < 128 ? 128 / G : 1][kSums<G>];
  int flip = 0;
  const int j = threadIdx.x % G;
  const long long at = ((long long)blockIdx.x * (blockDim.x / G) + threadIdx.x / G) * R;
  Piece<T, VEC> in[R][NV];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const T* x = (const T*)row_at(a.x, row_of(a, at + r < a.rows ? (int)at + r : a.rows - 1));
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * G + j) * VEC;
      if (FULL || c < a.D) in[r][i].load(x + c);
      else in[r][i].zero();
    }
  }
  float2 st[R];
  T* y[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    st[r] = statistics<FULL, T, VEC, G, NV>(in[r], a, j, sums[threadIdx.x / G], flip);
    y[r] = (T*)row_at(a.y, row_of(a, at + r < a.rows ? (int)at + r : a.rows - 1));
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * G + j) * VEC;
    if (!FULL && c >= a.D) continue;
    float v[VEC], w[VEC], b[VEC];
    weights(a.w ? a.w + c : nullptr, w, 1.f);
    weights(a.bias ? a.bias + c : nullptr, b, 0.f);
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) v[e] = fmaf((in[r][i][e] - st[r].x) * st[r].y, w[e], b[e]);
      if (at + r < a.rows) Piece<T, VEC>::store(y[r] + c, v);
    }
  }
}

// Rows of one piece a thread: a group takes R rows, a grid's groups apart,
// their reads and the steps of their sums side by side.
template <class T, int VEC, int G, int R>
__global__ void __launch_bounds__(256) norm_short_kernel(const NormArgs a) {
  begin();
  const int j = threadIdx.x % G, c = j * VEC;
  const int step = gridDim.x * (256 / G), at = blockIdx.x * (256 / G) + threadIdx.x / G;
  Piece<T, VEC> in[R];
  float w[VEC], b[VEC], s[R];
  const bool mine = c < a.D;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    in[i].zero();
    if (mine && (long long)at + (long long)i * step < a.rows) in[i].load((const T*)row_at(a.x, row_of(a, at + i * step)) + c);
  }
  weights(a.w && mine ? a.w + c : nullptr, w, 1.f);
  weights(a.bias && mine ? a.bias + c : nullptr, b, 0.f);
  int flip = 0;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    s[i] = 0.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[i] += in[i][e];
  }
  group_sum<G>(s, nullptr, flip);
  float mean[R], d[2 * R];
#pragma unroll
  for (int i = 0; i < R; ++i) {
    mean[i] = s[i] * a.inv_d, d[2 * i] = d[2 * i + 1] = 0.f;
    if (mine)
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float x = in[i][e] - mean[i];
        d[2 * i] += x, d[2 * i + 1] = fmaf(x, x, d[2 * i + 1]);
      }
  }
  group_sum<G>(d, nullptr, flip);
#pragma unroll
  for (int i = 0; i < R; ++i) {
    if (!mine || (long long)at + (long long)i * step >= a.rows) continue;
    const float2 st = corrected(mean[i], d[2 * i], d[2 * i + 1], a.inv_d);
    const float r = 1.f / sqrtf(st.y + a.eps);
    float v[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) v[e] = fmaf((in[i][e] - st.x) * r, w[e], b[e]);
    Piece<T, VEC>::store((T*)row_at(a.y, row_of(a, at + i * step)) + c, v);
  }
}

template <int G>
constexpr int kBwdBlock = G < 128 ? 128 : G;
// CTAs of an SM that the registers are to allow
template <int VEC, int G, int NV>
constexpr int kBwdFit = kBwdBlock<G> > 512 ? 1 : (NV * VEC > 16 ? 384 : 512) / kBwdBlock<G> < 1 ? 1
                                                : (NV * VEC > 16 ? 384 : 512) / kBwdBlock<G>;

__device__ __forceinline__ void copy16(void* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(dst)), "l"(src)
               : "memory");
}

// The gradient: a group takes row (CTA kGroups + group), then a grid further
// on; every thread sums its own columns' parts of dw and db in registers, the
// groups of a CTA are added in order, and norm_dw_kernel adds the CTAs'.
// Pieces of 16 bytes are copied ahead into shared memory, each by the thread
// that will use it, and read from there in each pass over the row: kAhead rows
// are held without a register, those of the sums leave no room for them.
template <int G, int NV>
constexpr int kAhead = 3 * 2 * NV * kBwdBlock<G> * 16 <= 200 * 1024 ? 3 : 1;  // (one: fp32 rows of more than 8192)
template <bool FULL, class T, int VEC, int G, int NV>
__global__ void __launch_bounds__(kBwdBlock<G>, kBwdFit<VEC, G, NV>) norm_bwd_kernel(const NormArgs a) {
  begin();
  constexpr int kBlock = kBwdBlock<G>, kGroups = kBlock / G;
  constexpr bool kAsync = VEC * sizeof(T) == 16;
  constexpr int kRing = kAhead<G, NV>;
  __shared__ float sums[kGroups][kSums<G>];
  extern __shared__ __align__(16) uint4 ring[];  // [kRing][2 NV][kBlock]
  int flip = 0;
  const int j = threadIdx.x % G;
  constexpr int kPairs = NV * VEC / 2;
  uint64_t w[kPairs], dw[kPairs], db[kPairs];  // of a thread's entries, in pairs
  {
    float x[NV * VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * G + j) * VEC;
      weights(a.w && c < a.D ? a.w + c : nullptr, *(float(*)[VEC])&x[i * VEC], 1.f);
    }
#pragma unroll
    for (int k = 0; k < kPairs; ++k) w[k] = tc::f2_pack(x[2 * k], x[2 * k + 1]), dw[k] = db[k] = 0;
  }
  const long long step = (long long)gridDim.x * kGroups;
  const long long first = (long long)blockIdx.x * kGroups;
  const auto fetch = [&](long long base, int slot) {
    const long long at = base + threadIdx.x / G;
    if (base < a.rows) {
      const Row row = row_of(a, at < a.rows ? (int)at : a.rows - 1);
      const T *x = (const T*)row_at(a.x, row), *u = (const T*)row_at(a.u, row);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * G + j) * VEC;
        if (FULL || c < a.D) {
          copy16(&ring[(slot * 2 * NV + 2 * i) * kBlock + threadIdx.x], x + c);
          copy16(&ring[(slot * 2 * NV + 2 * i + 1) * kBlock + threadIdx.x], u + c);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int slot = 0;
  if constexpr (kAsync) {
#pragma unroll
    for (int s = 0; s < kRing; ++s) fetch(first + s * step, s);
  }
  // (all groups of a CTA go round alike: those behind the last row work on it again, and drop the result)
  for (long long base = first; base < a.rows; base += step) {
    const long long at = base + threadIdx.x / G;
    const bool live = at < a.rows;
    const Row row = row_of(a, live ? (int)at : a.rows - 1);
    Piece<T, VEC> in[NV], gu[NV];
    const uint4* mine = &ring[slot * 2 * NV * kBlock + threadIdx.x];
    if constexpr (kAsync) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
    } else {
      const T *x = (const T*)row_at(a.x, row), *u = (const T*)row_at(a.u, row);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * G + j) * VEC;
        if (c < a.D) {
          in[i].load(x + c), gu[i].load(u + c);
        } else {
          in[i].zero(), gu[i].zero();
        }
      }
    }
    // the row's pieces, again for each pass
    const auto pieces = [&](bool both) {
      if constexpr (kAsync) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (!FULL) in[i].zero(), gu[i].zero();
          if (FULL || (i * G + j) * VEC < a.D) {
            in[i].load((const T*)(mine + 2 * i * kBlock));
            if (both) gu[i].load((const T*)(mine + (2 * i + 1) * kBlock));
          }
        }
      }
    };
    pieces(false);
    const float2 st = statistics<FULL, T, VEC, G, NV>(in, a, j, sums[threadIdx.x / G], flip);
    pieces(true);
    // with d = x - mean, z = r d
    const uint64_t r2 = both(st.y), less = both(-st.x);
    uint64_t t0 = 0, t1 = 0;  // sums of t and t d
    each<kPairs>([&](auto k) {
      const uint64_t d = tc::f2_add(pair_of<k>(in), less), u = pair_of<k>(gu), t = tc::f2_mul(u, w[k]);
      t0 = tc::f2_add(t0, t);
      t1 = tc::f2_fma(t, d, t1);
      if (live) dw[k] = tc::f2_fma(tc::f2_mul(u, r2), d, dw[k]), db[k] = tc::f2_add(db[k], u);
    });
    float m[2] = {sum_of(t0), sum_of(t1)};
    group_sum<G>(m, sums[threadIdx.x / G], flip);
    const uint64_t m0 = both(-m[0] * a.inv_d), m1 = both(-(m[1] * st.y * a.inv_d) * st.y * st.y);
    pieces(true);
    T* y = (T*)row_at(a.y, row);
    float v[NV * VEC];
    each<kPairs>([&](auto k) {
      const uint64_t d = tc::f2_add(pair_of<k>(in), less), t = tc::f2_fma(pair_of<k>(gu), w[k], m0);
      tc::f2_unpack(tc::f2_fma(d, m1, tc::f2_mul(r2, t)), v[2 * k], v[2 * k + 1]);
    });
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * G + j) * VEC;
      if ((FULL || c < a.D) && live) Piece<T, VEC>::store(y + c, *(const float(*)[VEC])&v[i * VEC]);
    }
    if constexpr (kAsync) {
      fetch(base + kRing * step, slot);
      slot = slot + 1 == kRing ? 0 : slot + 1;
    }
  }
  if (!a.part) return;
  float* part = a.part + (long long)blockIdx.x * 2 * a.D;
  float sw[NV * VEC], sb[NV * VEC];
#pragma unroll
  for (int k = 0; k < kPairs; ++k) {
    tc::f2_unpack(dw[k], sw[2 * k], sw[2 * k + 1]);
    tc::f2_unpack(db[k], sb[2 * k], sb[2 * k + 1]);
  }
  if constexpr (kGroups == 1) {
#pragma unroll
    for (int i = 0; i < NV * VEC; ++i) {
      const int c = (i / VEC * G + j) * VEC + i % VEC;
      if (c < a.D) part[c] = sw[i], part[a.D + c] = sb[i];
    }
  } else {
    __shared__ float acc[2][G * NV * VEC];
    for (int g = 0; g < kGroups; ++g) {
      if ((int)threadIdx.x / G == g)
#pragma unroll
        for (int i = 0; i < NV * VEC; ++i) {
          const int c = (i / VEC * G + j) * VEC + i % VEC;
          acc[0][c] = g ? acc[0][c] + sw[i] : sw[i];
          acc[1][c] = g ? acc[1][c] + sb[i] : sb[i];
        }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.D; c += kBlock) part[c] = acc[0][c], part[a.D + c] = acc[1][c];
  }
}

// dw and db: blockDim.x columns a CTA, blockDim.y threads (a power of two) a
// column over the CTAs' sums, added by halves.
__global__ void __launch_bounds__(1024) norm_dw_kernel(const float* __restrict__ part, int n, int D, float* dw, float* db) {
  begin();
  __shared__ float sm[1024];
  const int c = blockIdx.x * blockDim.x + threadIdx.x;  // of [dw | db]
  float s[8] = {};                                      // (eight reads in flight)
  if (c < 2 * D)
    for (int i = threadIdx.y; i < n; i += 8 * blockDim.y)
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int at = i + u * blockDim.y;
        if (at < n) s[u] += part[(long long)at * 2 * D + c];
      }
  float* mine = sm + threadIdx.y * blockDim.x + threadIdx.x;
  *mine = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  for (int h = blockDim.y / 2; h > 0; h >>= 1) {
    __syncthreads();
    if ((int)threadIdx.y < h) *mine += mine[h * blockDim.x];
  }
  if (threadIdx.y > 0 || c >= 2 * D) return;
  float* out = c < D ? dw : db;
  if (out) out[c < D ? c : c - D] = *mine;
}

// ----------------------------------------------------------------- launches

template <bool BWD, bool FULL, class T, int VEC, int G, int NV>
cudaError_t go(const NormArgs& a, int* ctas, cudaStream_t st) {
  if constexpr (!BWD && G <= 32 && NV == 1 && VEC > 1) {
    // (rows enough for four CTAs' worth of groups on every SM; 524,288 rows of 64 one row a group 35 us, four 30,
    // fp32 67 and 42)
    constexpr int R = 4;
    if (a.rows >= 32 * kSMs * (256 / G)) {
      const long long groups = ((long long)a.rows + R - 1) / R;
      return after(norm_short_kernel<T, VEC, G, R>, (unsigned)((groups + 256 / G - 1) / (256 / G)), dim3(256), 0, st, 0, a);
    }
  }
  if constexpr (!BWD) {
    // rows enough for every SM, and of 32 entries a thread or more: two of them to a group (bf16, 32,768 rows of 2048
    // one row 50 us, two 47; 65,536 of 1024 48 and 43)
    constexpr int R = sizeof(T) == 2 && VEC == 8 && NV * VEC >= 32 ? 2 : 1;
    // few rows: a CTA each, so that more SMs have a part
    const bool few = a.rows < 8 * kSMs;
    const int block = G >= 128 ? G : few && G >= 32 ? G : 128;
    const int groups = block / G;
    const long long rows = (long long)groups * (few ? 1 : R);
    return after(few ? norm_kernel<FULL, T, VEC, G, NV, 1> : norm_kernel<FULL, T, VEC, G, NV, R>,
                 (unsigned)((a.rows + rows - 1) / rows), dim3(block), 0, st, 0, a);
  } else {
  constexpr int kBlock = kBwdBlock<G>, kGroups = kBlock / G;
  constexpr int smem = VEC * sizeof(T) == 16 ? kAhead<G, NV> * 2 * NV * kBlock * 16 : 0;
  auto kern = norm_bwd_kernel<FULL, T, VEC, G, NV>;
  cudaError_t e = cudaSuccess;
  if (smem > 0) e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  static std::atomic<int> fits{0};  // the same on every GPU that this library runs on
  int fit = fits.load(std::memory_order_relaxed);
  if (e == cudaSuccess && fit == 0) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, kern, kBlock, smem);
    if (e == cudaSuccess) fits.store(fit, std::memory_order_relaxed);
  }
  if (e != cudaSuccess) return e;
  // as many CTAs as fit, but no more than one an SM where their sums would be more than a quarter of the rows' bytes
  // (as many as fit at 1024 rows of 2048, bf16: 7 MB of sums for 12 MB of rows)
  long long most = kSMs * (fit < kBwdCtas / kSMs ? fit : kBwdCtas / kSMs);
  const long long few = (long long)a.rows * sizeof(T) * 3 / 32;
  if (most > few) most = few > kSMs ? few : kSMs;
  const long long need = ((long long)a.rows + kGroups - 1) / kGroups;
  *ctas = (int)(need < most ? need : most);
  return after(kern, (unsigned)*ctas, dim3(kBlock), smem, st, 0, a);
  }
}

// Threads and pieces of a row by its length: up to 64 entries a thread forward,
// so that the steps of the row's sums are few beside its entries; up to 32 in the
// gradient, which keeps two sums and a weight for each (16 in rows of more than
// 4096 to 8192 entries, on 512 threads, and wherever rows move in pairs or entry by
// entry).
template <bool BWD, class T>
cudaError_t choose(const NormArgs& a, bool vec, bool pairs, int* ctas, cudaStream_t st) {
  constexpr int V = sizeof(T) == 2 ? 8 : 4;
  constexpr int M = 32 / V;
  const int n = vec ? a.D / V : a.D;
#define NATS_NORM(VEC, G, NV) \
  if (n <= (G) * (NV))        \
  return (VEC) > 2 && n == (G) * (NV) ? go<BWD, ((VEC) > 2), T, VEC, G, NV>(a, ctas, st) \
                                      : go<BWD, false, T, VEC, G, NV>(a, ctas, st)
  if (vec) {
    NATS_NORM(V, 8, 1);
    NATS_NORM(V, 16, 1);
    NATS_NORM(V, 32, 1);
    NATS_NORM(V, 32, 2);
    if constexpr (BWD) {
      if constexpr (M / 2 > 2) {
        NATS_NORM(V, 32, M / 2);
      }
      NATS_NORM(V, 32, M);
      NATS_NORM(V, 64, M);
      NATS_NORM(V, 128, M);
      NATS_NORM(V, 512, M / 2);
      NATS_NORM(V, 512, M);
    } else {
      NATS_NORM(V, 32, M);
      NATS_NORM(V, 32, 2 * M);
      NATS_NORM(V, 64, 2 * M);
      NATS_NORM(V, 128, 2 * M);
      NATS_NORM(V, 256, 2 * M);
    }
    return cudaErrorInvalidValue;
  }
  if constexpr (V == 8) {
    if (pairs) {
      const int n = a.D / 2;
      NATS_NORM(2, 32, 4);
      NATS_NORM(2, 32, 8);
      if constexpr (!BWD) NATS_NORM(2, 32, 16);
      NATS_NORM(2, 64, 8);
      NATS_NORM(2, 128, 8);
      NATS_NORM(2, 256, 8);
      NATS_NORM(2, 512, 8);
      NATS_NORM(2, 1024, 8);
      return cudaErrorInvalidValue;
    }
  }
  {
    NATS_NORM(1, 32, 4);
    NATS_NORM(1, 32, 16);
    if constexpr (!BWD) NATS_NORM(1, 32, 32);
    NATS_NORM(1, 64, 16);
    NATS_NORM(1, 128, 16);
    NATS_NORM(1, 256, 16);
    NATS_NORM(1, 512, 16);
    NATS_NORM(1, 1024, 16);
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
bool rows_at(const Rows& r, const nats_norm_dims* d, int n) {
  return elem_ok(r.p, n) && (d->B == 1 || r.b % n == 0) && (d->H == 1 || r.h % n == 0) && (d->L == 1 || r.t % n == 0);
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
  a.rows = dims->B * dims->H * dims->L, a.H = dims->H, a.L = dims->L, a.D = dims->D, a.flat = dims->B == 1 && dims->H == 1;
  a.eps = dims->eps, a.inv_d = 1.f / dims->D;
  const bool vec = dims->D % (16 / es) == 0 && rows_at(a.x, dims, 16) && rows_at(a.y, dims, 16) && elem_ok(w, 16) && elem_ok(b, 16);
  const bool pairs = dims->D % 2 == 0 && rows_at(a.x, dims, 4) && rows_at(a.y, dims, 4);
  cudaStream_t st = (cudaStream_t)stream;
  return (nats_status)record_cuda_error(es == 2 ? choose<false, __nv_bfloat16>(a, vec, pairs, nullptr, st)
                                                : choose<false, float>(a, vec, pairs, nullptr, st));
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
  a.rows = dims->B * dims->H * dims->L, a.H = dims->H, a.L = dims->L, a.D = dims->D, a.flat = dims->B == 1 && dims->H == 1;
  a.eps = dims->eps, a.inv_d = 1.f / dims->D;
  const bool vec = dims->D % (16 / es) == 0 && rows_at(a.x, dims, 16) && rows_at(a.y, dims, 16) && rows_at(a.u, dims, 16) &&
                   elem_ok(w, 16);
  const bool pairs = dims->D % 2 == 0 && rows_at(a.x, dims, 4) && rows_at(a.y, dims, 4) && rows_at(a.u, dims, 4);
  int ctas = 0;
  const int r = record_cuda_error(es == 2 ? choose<true, __nv_bfloat16>(a, vec, pairs, &ctas, st)
                                          : choose<true, float>(a, vec, pairs, &ctas, st));
  if (r != NATS_OK || !sums) return (nats_status)r;
  const float* part = a.part;
  // a short row's columns are few: fewer of them to a CTA, and more threads to each
  const dim3 block = dims->D <= 512 ? dim3(8, 128) : dim3(32, ctas > 64 ? 32 : 8);
  return (nats_status)record_cuda_error(
      after(norm_dw_kernel, (2 * dims->D + block.x - 1) / block.x, block, 0, st, 0, part, ctas, (int)dims->D, dw, db));
}

}  // extern "C"
