// decay_attn.cu - linear attention with a decay for each head: the entry
// points of the prompt form and its gradient (nats_decay_attn,
// nats_decay_attn_bwd), the split of long sequences into segments, and the
// fp32 kernel, which also takes bf16 operands that TMA cannot address.
// decay.cuh has the mathematics, decay_attn_tc.cu the tensor-core kernel.
#include <cmath>

#include "../../include/nats.h"
#include "decay.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace nats {
namespace decay {
namespace {

constexpr int kC = 32;  // tokens of a chunk

template <class T>
__device__ __forceinline__ float4 load4(const T* p, bool vec);
template <>
__device__ __forceinline__ float4 load4<float>(const float* p, bool vec) {
  if (vec) return *(const float4*)p;
  return make_float4(p[0], p[1], p[2], p[3]);
}
template <>
__device__ __forceinline__ float4 load4<__nv_bfloat16>(const __nv_bfloat16* p, bool vec) {
  if (vec) {
    const uint2 u = *(const uint2*)p;
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xffff0000u));
  }
  return make_float4(to_f32(p[0]), to_f32(p[1]), to_f32(p[2]), to_f32(p[3]));
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4], bool vec) {
  if (vec)
    *(float4*)p = make_float4(v[0], v[1], v[2], v[3]);
  else
    for (int e = 0; e < 4; ++e) p[e] = v[e];
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4], bool vec) {
  if (vec) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
    *(uint2*)p = make_uint2(*(const uint32_t*)&a, *(const uint32_t*)&b);
  } else {
    for (int e = 0; e < 4; ++e) p[e] = __float2bfloat16_rn(v[e]);
  }
}

template <int D>
struct Simt {
  static constexpr int kRow = D + 4;  // padded: 8 rows' 16-byte pieces lie in different banks
  static constexpr int kP = kC + 1;
  static constexpr int offQ = 0, offK = offQ + kC * kRow, offV = offK + kC * kRow, offS = offV + kC * kWidth,
                       offP = offS + D * kWidth, offW = offP + kC * kP + 3, kFloats = offW + kC + 1;
};

// One CTA walks the chunks of one segment of one (scan, sequence, head, 64
// state columns); the state is in registers (rows 8 (or 4) to a group of 16
// threads) with a copy in shared memory for its product with the queries.
template <class T, int D, bool STATES>
__global__ void __launch_bounds__(256) scan_simt_kernel(const Args a) {
  begin();
  using M = Simt<D>;
  extern __shared__ __align__(16) float sm[];
  float *Qs = sm + M::offQ, *Ks = sm + M::offK, *Vs = sm + M::offV, *Ss = sm + M::offS, *Ps = sm + M::offP,
        *Ws = sm + M::offW;  // Ws[m] = gamma^m, m = 0 .. kC
  constexpr int kSlices = D / kWidth;
  constexpr int R = D / 16;  // state rows of a thread

  const int segs = STATES ? a.segs - 1 : a.segs;
  long long x = blockIdx.x;
  const int slice = (int)(x % kSlices);
  x /= kSlices;
  int seg = (int)(x % segs);
  x /= segs;
  const int bh = (int)(x % ((long long)a.B * a.H));
  const Op& op = a.op[a.first_op + (int)(x / ((long long)a.B * a.H))];
  const int b = bh / a.H, h = bh % a.H;
  // the states of a segment are asked for by the next one in the scan's order
  if (STATES && op.back) ++seg;
  const int len = length(a, b);
  const int t0 = seg * a.seg, t1 = min(t0 + a.seg, a.L);
  const int n_seg = max(0, min(t1, len) - t0);
  const int tid = threadIdx.x;
  const float g = a.g[h];
  const bool vec = a.vec != 0, back = op.back != 0;
  const T* q = (const T*)op.q.p + b * op.q.b + h * op.q.h;
  const T* k = (const T*)op.k.p + b * op.k.b + h * op.k.h;
  const T* v = (const T*)op.v.p + b * op.v.b + h * op.v.h + slice * kWidth;
  T* o = (T*)op.o.p + b * op.o.b + h * op.o.h + slice * kWidth;

  if (tid <= kC) Ws[tid] = power(g, tid);
  const int r0 = (tid >> 4) * R, c4 = (tid & 15) * 4;
  float S[R][4];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float s = 0.f;
      if (!STATES) {
        const int c = slice * kWidth + c4 + e;
        if (a.segs > 1)
          s = op.part[((long long)bh * a.segs + seg) * D * D + (op.part_t ? (r0 + r) * D + c : c * D + r0 + r)];
        else if (op.s_in)
          s = op.s_in[(long long)bh * D * D + (r0 + r) * op.s_r + c * op.s_c] * op.in_scale;
      }
      S[r][e] = s;
      Ss[(r0 + r) * kWidth + c4 + e] = s;
    }
  const int chunks = (n_seg + kC - 1) / kC;
  for (int cc = 0; cc < chunks; ++cc) {
    const int c = back ? chunks - 1 - cc : cc;
    const int base = t0 + c * kC, n = min(kC, n_seg - c * kC);
    __syncthreads();  // the chunk before has been read, S is in place
    for (int i = tid; i < kC * (D / 4); i += 256) {
      const int t = i / (D / 4), f = (i % (D / 4)) * 4;
      // rows in the scan's order; those behind the end are zero
      const long long src = base + (back ? n - 1 - t : t);
      const float4 z = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!STATES) *(float4*)(Qs + t * M::kRow + f) = t < n ? load4(q + src * op.q.t + f, vec) : z;
      *(float4*)(Ks + t * M::kRow + f) = t < n ? load4(k + src * op.k.t + f, vec) : z;
    }
    for (int i = tid; i < kC * (kWidth / 4); i += 256) {
      const int t = i / (kWidth / 4), f = (i % (kWidth / 4)) * 4;
      const long long src = base + (back ? n - 1 - t : t);
      *(float4*)(Vs + t * kWidth + f) =
          t < n ? load4(v + src * op.v.t + f, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    __syncthreads();
    if (!STATES) {
      {  // P: rows ti, ti + 16, columns tj, tj + 16
        const int ti = tid >> 4, tj = tid & 15;
        float p[2][2] = {};
        for (int f = 0; f < D; f += 4) {
          const float4 q0 = *(const float4*)(Qs + ti * M::kRow + f), q1 = *(const float4*)(Qs + (ti + 16) * M::kRow + f);
          const float4 k0 = *(const float4*)(Ks + tj * M::kRow + f), k1 = *(const float4*)(Ks + (tj + 16) * M::kRow + f);
          const auto dot = [](float s, const float4& x, const float4& y) {
            return fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s))));
          };
          p[0][0] = dot(p[0][0], q0, k0), p[0][1] = dot(p[0][1], q0, k1);
          p[1][0] = dot(p[1][0], q1, k0), p[1][1] = dot(p[1][1], q1, k1);
        }
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int z = 0; z < 2; ++z) {
            const int i = ti + 16 * y, j = tj + 16 * z;
            Ps[i * M::kP + j] = j <= i ? p[y][z] * Ws[i - j] : 0.f;
          }
      }
      __syncthreads();
      // o: rows ti, ti + 16, columns c4 .. c4 + 3
      const int ti = tid >> 4;
      float acc[2][4] = {}, inter[2][4] = {};
      for (int f = 0; f < D; f += 4) {
        const float4 q0 = *(const float4*)(Qs + ti * M::kRow + f), q1 = *(const float4*)(Qs + (ti + 16) * M::kRow + f);
        const float x0[4] = {q0.x, q0.y, q0.z, q0.w}, x1[4] = {q1.x, q1.y, q1.z, q1.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const float4 s = *(const float4*)(Ss + (f + u) * kWidth + c4);
          const float y[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            inter[0][e] = fmaf(x0[u], y[e], inter[0][e]), inter[1][e] = fmaf(x1[u], y[e], inter[1][e]);
        }
      }
      for (int j = 0; j < kC; ++j) {
        const float4 w = *(const float4*)(Vs + j * kWidth + c4);
        const float y[4] = {w.x, w.y, w.z, w.w};
        const float p0 = Ps[ti * M::kP + j], p1 = Ps[(ti + 16) * M::kP + j];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][e] = fmaf(p0, y[e], acc[0][e]), acc[1][e] = fmaf(p1, y[e], acc[1][e]);
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int i = ti + 16 * y;
        if (i >= n) continue;
        const float w = Ws[i + 1 - (back ? 1 : 0)];
        float r[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) r[e] = a.scale * fmaf(w, inter[y][e], acc[y][e]);
        const long long dst = base + (back ? n - 1 - i : i);
        store4(o + dst * op.o.t + c4, r, vec);
      }
      __syncthreads();  // Ss has been read
    }
    float add[R][4] = {};
    for (int j = 0; j < n; ++j) {
      const float w = Ws[n - 1 - j + (back ? 1 : 0)];
      const float4 z = *(const float4*)(Vs + j * kWidth + c4);
      const float y[4] = {z.x * w, z.y * w, z.z * w, z.w * w};
      float x[R];
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        const float4 f = *(const float4*)(Ks + j * M::kRow + r0 + r);
        x[r] = f.x, x[r + 1] = f.y, x[r + 2] = f.z, x[r + 3] = f.w;
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int e = 0; e < 4; ++e) add[r][e] = fmaf(x[r], y[e], add[r][e]);
    }
    const Carry carry(g, n);
#pragma unroll
    for (int r = 0; r < R; ++r) {
#pragma unroll
      for (int e = 0; e < 4; ++e) S[r][e] = carry(S[r][e], add[r][e]);
      if (!STATES) *(float4*)(Ss + (r0 + r) * kWidth + c4) = make_float4(S[r][0], S[r][1], S[r][2], S[r][3]);
    }
  }
  if (STATES) {
    // the segment's own sum, at the segment that takes it
    const int to = back ? seg - 1 : seg + 1;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        op.part[((long long)bh * a.segs + to) * D * D + (slice * kWidth + c4 + e) * D + r0 + r] = S[r][e];
    return;
  }
  // rows behind the sequence's end
  for (int i = tid; i < (t1 - t0 - n_seg) * (kWidth / 4); i += 256) {
    const float z[4] = {};
    store4(o + (t0 + n_seg + i / (kWidth / 4)) * op.o.t + (i % (kWidth / 4)) * 4, z, vec);
  }
  if (op.s_out && seg == (back ? 0 : a.segs - 1)) {
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        op.s_out[(long long)bh * D * D + (r0 + r) * op.s_r + (slice * kWidth + c4 + e) * op.s_c] =
            S[r][e] * op.out_scale;
  }
}

// part of segment s holds the sum of the segment before it (in the scan's
// order) alone; each entry's running state replaces it.
template <int D>
__global__ void __launch_bounds__(256) join_kernel(const Args a) {
  begin();
  constexpr int kBlocks = D * D / 256;
  const int x = blockIdx.x / kBlocks;
  const int bh = x % (a.B * a.H);
  const Op& op = a.op[a.first_op + x / (a.B * a.H)];
  const int at = (blockIdx.x % kBlocks) * 256 + threadIdx.x;
  const int r = at % D, c = at / D;
  const float g = a.g[bh % a.H];
  const int len = length(a, bh / a.H);
  float* part = op.part + (long long)bh * a.segs * D * D + at;
  float S = op.s_in ? op.s_in[(long long)bh * D * D + r * op.s_r + c * op.s_c] * op.in_scale : 0.f;
  const auto seg_at = [&](int i) { return op.back ? a.segs - 1 - i : i; };
  part[(long long)seg_at(0) * D * D] = S;
  for (int i = 1; i < a.segs; i += 8) {
    float own[8];  // (eight reads in flight)
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i + u < a.segs) own[u] = part[(long long)seg_at(i + u) * D * D];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      if (i + u < a.segs) {
        const int before = seg_at(i + u - 1);
        const int n = max(0, min(min(before * a.seg + a.seg, a.L), len) - before * a.seg);
        S = Carry(g, n)(S, own[u]);
        part[(long long)seg_at(i + u) * D * D] = S;
      }
  }
}

// The states of empty sequences pass through.
__global__ void pass_kernel(const float* __restrict__ in, float* __restrict__ out, long long n) {
  begin();
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256)
    out[i] = in ? in[i] : 0.f;
}

template <class T, int D>
cudaError_t launch_simt(const Args& a, bool states, cudaStream_t st) {
  auto kern = states ? scan_simt_kernel<T, D, true> : scan_simt_kernel<T, D, false>;
  const int smem = Simt<D>::kFloats * 4;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long long grid = (long long)(a.last_op - a.first_op) * a.B * a.H * (D / kWidth) * (states ? a.segs - 1 : a.segs);
  return after(kern, (unsigned)grid, dim3(256), smem, st, 0, a);
}

// --------------------------------------------------------------- the split

// How many segments a sequence of `chunks` chunks is cut into, for `units`
// independent walks (scan, sequence, head, 64 state columns).  A CTA walks one
// segment; the states ahead of the segments come from a launch that reads keys
// and values alone, at about half a walk's time, which has to be worth it: the
// cut that takes the fewest rounds of chunks over the SMs is chosen.
int segments(long long units, int chunks, int ctas) {
  int best = 1;
  double least = 1e300;
  for (int s = 1; s <= kMaxSegs && s <= chunks; ++s) {
    const int per = (chunks + s - 1) / s;
    if ((chunks + per - 1) / per != s) continue;  // a cut with an empty last segment
    const double rounds = std::ceil((double)units * s / ctas) * per;
    const double before = s == 1 ? 0.0 : std::ceil((double)units * (s - 1) / ctas) * per * 0.5 + 4.0;
    if (rounds + before < least) least = rounds + before, best = s;
  }
  return best;
}

constexpr int kChunkTc = 128;

struct Cut {
  int segs, seg;
};
Cut cut(const nats_decay_dims* m, int nops, bool tc) {
  const int C = tc ? kChunkTc : kC;
  const int chunks = (m->L + C - 1) / C;
  const long long units = (long long)nops * m->B * m->H * (m->d / kWidth);
  // (fp32: two CTAs to an SM)
  const int segs = segments(units, chunks, tc ? kSMs : 2 * kSMs);
  return {segs, (chunks + segs - 1) / segs * C};
}

size_t part_bytes(const nats_decay_dims* m, int segs) {
  return segs > 1 ? (size_t)m->B * m->H * segs * m->d * m->d * 4 : 0;
}
size_t workspace(const nats_decay_dims* m, int nops) {
  const size_t simt = part_bytes(m, cut(m, nops, false).segs);
  const size_t tc = m->dtype == NATS_BF16 ? part_bytes(m, cut(m, nops, true).segs) : 0;
  return (nops == 1 ? 1 : 2) * (simt > tc ? simt : tc);
}

// ------------------------------------------------------------------ checks

bool elem_ok(const void* p, int es) { return ((uintptr_t)p & (uintptr_t)(es - 1)) == 0; }

// what a tensor map can address
bool mapped(const Tokens& x, const nats_decay_dims* m) {
  const auto ok = [](int extent, long long s) { return extent == 1 || (s > 0 && s < (1LL << 38)); };
  return rows_at(x, m, 16) && ok(m->B, x.b) && ok(m->H, x.h) && ok(m->L, x.t);
}

nats_status run(Args& a, const nats_decay_dims* m, const float* log_decay, const int32_t* lens, void* ws,
                size_t ws_bytes, cudaStream_t st) {
  a.g = log_decay, a.lens = lens, a.B = m->B, a.H = m->H, a.L = m->L;
  a.scale = m->scale > 0.f ? m->scale : 1.0f / std::sqrt((float)m->d);
  const int nops = a.nops;
  bool tc = m->dtype == NATS_BF16, vec = true;
  for (int i = 0; i < nops; ++i)
    for (const Tokens* x : {&a.op[i].q, &a.op[i].k, &a.op[i].v, &a.op[i].o}) {
      if (!elem_ok(x->p, m->dtype == NATS_BF16 ? 2 : 4)) return NATS_ERR_ALIGN;
      vec = vec && rows_at(*x, m, m->dtype == NATS_BF16 ? 8 : 16);
      tc = tc && mapped(*x, m);
    }
  const Cut c = cut(m, nops, tc);
  const size_t one = part_bytes(m, c.segs);
  if (one) {
    if (!ws) return NATS_ERR_NULL;
    if ((uintptr_t)ws & 15u) return NATS_ERR_ALIGN;
    if (ws_bytes < workspace(m, nops)) return NATS_ERR_WORKSPACE;
  }
  a.segs = c.segs, a.seg = c.seg, a.vec = vec;
  // the scans for dk and dv carry the same states, one the other's transpose:
  // the last scan forms them for both
  for (int i = 0; i < nops; ++i) {
    const bool shared = nops == 3 && i == 1;
    a.op[i].part = (float*)((char*)ws + (nops == 3 && i > 0 ? one : 0)), a.op[i].part_t = shared;
  }
  const auto scans = [&](int first, int last, bool states) {
    a.first_op = first, a.last_op = last;
    if (tc) return launch_tc(a, m->d, states, st);
    if (m->dtype == NATS_BF16)
      return m->d == 64 ? launch_simt<__nv_bfloat16, 64>(a, states, st) : launch_simt<__nv_bfloat16, 128>(a, states, st);
    return m->d == 64 ? launch_simt<float, 64>(a, states, st) : launch_simt<float, 128>(a, states, st);
  };
  cudaError_t e = cudaSuccess;
  if (c.segs > 1) {
    // the scans whose states are formed, side by side: the first and the last
    const Args all = a;
    a.op[1] = all.op[nops - 1];
    const int formed = nops == 3 ? 2 : 1;
    e = scans(0, formed, true);
    if (e != cudaSuccess) return (nats_status)record_cuda_error(e);
    const unsigned grid = (unsigned)((long long)formed * m->B * m->H * (m->d * m->d / 256));
    e = after(m->d == 64 ? join_kernel<64> : join_kernel<128>, grid, dim3(256), 0, st, 0, a);
    if (e != cudaSuccess) return (nats_status)record_cuda_error(e);
    a = all;
  }
  return (nats_status)record_cuda_error(scans(0, nops, false));
}

// an empty call: a last state is the first one
nats_status pass(const nats_decay_dims* m, const float* in, float* out, cudaStream_t st) {
  const long long n = (long long)m->B * m->H * m->d * m->d;
  if (!out || n == 0) return NATS_OK;
  const long long blocks = (n + 255) / 256;
  return (nats_status)record_cuda_error(
      after(pass_kernel, (unsigned)(blocks < 8 * kSMs ? blocks : 8 * kSMs), dim3(256), 0, st, 0, in, out, n));
}

}  // namespace

nats_status check_dims(const nats_decay_dims* m) {
  if (!m) return NATS_ERR_NULL;
  if (m->dtype != NATS_BF16 && m->dtype != NATS_F32) return NATS_ERR_DTYPE;
  if (m->B < 0 || m->H < 0 || m->L < 0) return NATS_ERR_SHAPE;
  if (m->d != 64 && m->d != 128) return NATS_ERR_UNSUPPORTED;
  if (!std::isfinite(m->scale) || m->scale < 0.f || (m->scale > 0.f && m->scale < 1.17549435e-38f)) return NATS_ERR_VALUE;
  // CTAs are numbered in 31 bits, with up to 64 segments, 2 column halves and 3 scans
  if ((double)m->B * m->H > 4194304.0 || m->L > (1 << 30)) return NATS_ERR_UNSUPPORTED;
  return NATS_OK;
}

}  // namespace decay
}  // namespace nats

using namespace nats;
using namespace nats::decay;

extern "C" {

size_t nats_decay_attn_workspace_size(const nats_decay_dims* dims) {
  return check_dims(dims) == NATS_OK && dims->L > 0 ? workspace(dims, 1) : 0;
}
size_t nats_decay_attn_bwd_workspace_size(const nats_decay_dims* dims) {
  return check_dims(dims) == NATS_OK && dims->L > 0 ? workspace(dims, 3) : 0;
}

nats_status nats_decay_attn(const nats_decay_dims* dims, const void* q, const nats_strides* q_st, const void* k,
                            const nats_strides* k_st, const void* v, const nats_strides* v_st, const float* log_decay,
                            const int32_t* lens, const float* state_in, void* out, const nats_strides* out_st,
                            float* state_out, void* ws, size_t workspace_bytes, nats_stream_t stream) {
  const nats_status s = check_dims(dims);
  if (s != NATS_OK) return s;
  if (!elem_ok(log_decay, 4) || !elem_ok(lens, 4) || !elem_ok(state_in, 4) || !elem_ok(state_out, 4)) return NATS_ERR_ALIGN;
  cudaStream_t st = (cudaStream_t)stream;
  if (dims->B == 0 || dims->H == 0) return NATS_OK;
  if (dims->L == 0) return state_in == state_out ? NATS_OK : pass(dims, state_in, state_out, st);
  if (!q || !q_st || !k || !k_st || !v || !v_st || !log_decay || !out || !out_st) return NATS_ERR_NULL;
  Args a = {};
  a.nops = 1;
  a.op[0] = {tokens(q, q_st), tokens(k, k_st), tokens(v, v_st), tokens(out, out_st), state_in, state_out,
             1, dims->d, 1.f, 1.f, nullptr, 0, 0};
  return run(a, dims, log_decay, lens, ws, workspace_bytes, st);
}

nats_status nats_decay_attn_bwd(const nats_decay_dims* dims, const void* dout, const nats_strides* dout_st,
                                const void* q, const nats_strides* q_st, const void* k, const nats_strides* k_st,
                                const void* v, const nats_strides* v_st, const float* log_decay, const int32_t* lens,
                                const float* state_in, const float* dstate_out, void* dq, const nats_strides* dq_st,
                                void* dk, const nats_strides* dk_st, void* dv, const nats_strides* dv_st,
                                float* dstate_in, void* ws, size_t workspace_bytes, nats_stream_t stream) {
  const nats_status s = check_dims(dims);
  if (s != NATS_OK) return s;
  for (const void* p : {(const void*)log_decay, (const void*)lens, (const void*)state_in, (const void*)dstate_out,
                        (const void*)dstate_in})
    if (!elem_ok(p, 4)) return NATS_ERR_ALIGN;
  if (dstate_in && dstate_in == dstate_out) return NATS_ERR_VALUE;
  cudaStream_t st = (cudaStream_t)stream;
  if (dims->B == 0 || dims->H == 0) return NATS_OK;
  if (dims->L == 0) return pass(dims, dstate_out, dstate_in, st);
  if (!dout || !dout_st || !q || !q_st || !k || !k_st || !v || !v_st || !log_decay || !dq || !dq_st || !dk || !dk_st ||
      !dv || !dv_st)
    return NATS_ERR_NULL;
  const Tokens tu = tokens(dout, dout_st), tq = tokens(q, q_st), tk = tokens(k, k_st), tv = tokens(v, v_st);
  const float scale = dims->scale > 0.f ? dims->scale : 1.0f / std::sqrt((float)dims->d);
  const long long d = dims->d;
  Args a = {};
  a.nops = 3;
  // the state's gradient is carried without the scale of the outputs
  a.op[0] = {tu, tv, tk, tokens(dq, dq_st), state_in, nullptr, d, 1, 1.f, 1.f, nullptr, 0, 0};
  a.op[1] = {tv, tu, tq, tokens(dk, dk_st), dstate_out, nullptr, d, 1, 1.f / scale, scale, nullptr, 0, 1};
  a.op[2] = {tk, tq, tu, tokens(dv, dv_st), dstate_out, dstate_in, 1, d, 1.f / scale, scale, nullptr, 0, 1};
  return run(a, dims, log_decay, lens, ws, workspace_bytes, st);
}

nats_status nats_decay_attn_check(nats_stream_t stream) {
  int expired = 0;
  const int r = record_cuda_error(expired_waits(&expired, (cudaStream_t)stream));
  return r != NATS_OK ? (nats_status)r : expired ? NATS_ERR_INTERNAL : NATS_OK;
}

}  // extern "C"
