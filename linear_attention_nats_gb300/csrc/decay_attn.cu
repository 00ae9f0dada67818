// decay_attn.cu - linear attention with a decay for each head: the entry
// points of the prompt form and its gradient (nats_decay_attn,
// nats_decay_attn_bwd), the split of long sequences into segments, and the
// fp32 kernel, which also takes bf16 operands that TMA cannot address.
// decay.cuh has the mathematics, decay_attn_tc.cu the bf16 kernel.
//
// Measured on one GB300 (fp32, d = 64): 3 x 12 heads of 1021 tokens with states
// 43 us, of which 15 the segments' states and their join; gradient of 2 x 12
// heads 71 us.  d = 128, 32 x 16 heads of 512 tokens: 683 us, gradient 2018.  bf16
// operands that TMA cannot address, 4 x 16 heads of 8192 tokens, d = 128: 2383 us
// with one key and value head for all, 2620 at odd addresses (117 on the tensor
// cores).  Error 4.6e-7 of the outputs (plain fp32 operations 2.5e-7).
#include <cmath>
#include <type_traits>

#include "../../include/nats.h"
#include "decay.cuh"
#include "kernels.h"
#include "launch.cuh"

namespace nats {
namespace decay {
namespace {

constexpr int kC = 64;  // tokens of a chunk

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

__device__ __forceinline__ void store2(float* p, float x, float y, bool vec) {
  if (vec) *(float2*)p = make_float2(x, y);
  else p[0] = x, p[1] = y;
}
__device__ __forceinline__ void store2(__nv_bfloat16* p, float x, float y, bool vec) {
  if (vec) *(__nv_bfloat162*)p = __floats2bfloat162_rn(x, y);
  else p[0] = __float2bfloat16_rn(x), p[1] = __float2bfloat16_rn(y);
}

// Row pitches: a fragment's 8 rows x 4 entries lie in different banks where it
// is read along rows (kRow, kP), its 4 rows x 8 entries where along columns (kCol).
template <int D>
struct Split {
  static constexpr int kRow = D + 4, kP = kC + 4, kCol = kWidth + 8;
  static constexpr int offQ = 0, offK = offQ + kC * kRow, offV = offK + kC * kRow, offS = offV + kC * kCol,
                       offP = offS + D * kCol, offW = offP + kC * kP, kFloats = offW + kC + 4;
  static constexpr int kCtas = D == 64 ? 2 : 1;  // of an SM
};

// x as the sum of two tf32 numbers (10 bits of the fraction, the other 13 zero):
// the first is x rounded, and what is left of it, at most 2^12 units in x's last
// place, is cut off to 11 bits: one unit at most, 2^-23 of x.  (A rounding there
// would leave a unit too.  By cvt.rna, at a fraction of the rate of integer
// operations, 3 x 12 heads of 1021 tokens, d = 64, took 50 us where 43 were
// measured with these and without the products of rows behind the end or with a
// state of zero.)
__device__ __forceinline__ void split(float x, uint32_t& hi, uint32_t& lo) {
  hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
  lo = __float_as_uint(x - __uint_as_float(hi)) & 0xffffe000u;
}
__device__ __forceinline__ void mma8(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile(
      "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// acc += A B for a warp's 16 rows and 32 columns, k8 steps of 8.  a_at(k, row)
// and b_at(k, column) read an entry; a lane's rows are lane / 4 and that + 8, its
// columns of a tile of 8 lane / 4 as B's and 2 (lane % 4), + 1 as the sum's.
// Each factor goes in as two tf32 numbers, the product of the two second ones
// (at most 2^-11 of their factors: 2^-22) left out; the small products have a sum
// of their own.
template <class A, class B>
__device__ __forceinline__ void add_product(float (&acc)[4][4], int k8, const A& a_at, const B& b_at) {
  const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
  float small[4][4] = {};
#pragma unroll 2
  for (int s = 0; s < k8; ++s) {
    const int k = 8 * s + t;
    uint32_t ah[4], al[4];
    split(a_at(k, g), ah[0], al[0]);
    split(a_at(k, g + 8), ah[1], al[1]);
    split(a_at(k + 4, g), ah[2], al[2]);
    split(a_at(k + 4, g + 8), ah[3], al[3]);
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
      uint32_t bh[2], bl[2];
      split(b_at(k, 8 * nt + g), bh[0], bl[0]);
      split(b_at(k + 4, 8 * nt + g), bh[1], bl[1]);
      mma8(acc[nt], ah, bh);
      mma8(small[nt], ah, bl);
      mma8(small[nt], al, bh);
    }
  }
#pragma unroll
  for (int nt = 0; nt < 4; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[nt][e] += small[nt][e];
}

// One CTA walks the chunks of one segment of one (scan, sequence, head, 64
// state columns).  Every product is 64 x 64 (the state d x 64) on the tf32
// instructions in split precision, 16 rows and 32 columns to a warp, operands
// in shared memory; the state is in registers, with a copy there for its product
// with the queries.  (As fp32 FMAs, four rows and four columns to a thread, the
// reads from shared memory took twice the time of the FMAs: 3 x 12 heads of 1021
// tokens, d = 64, 83 us.)
template <class T, int D, bool STATES>
__global__ void __launch_bounds__(256, Split<D>::kCtas) scan_split_kernel(const Args a) {
  begin();
  using M = Split<D>;
  extern __shared__ __align__(16) float sm[];
  float *Qs = sm + M::offQ, *Ks = sm + M::offK, *Vs = sm + M::offV, *Ss = sm + M::offS, *Ps = sm + M::offP,
        *Ws = sm + M::offW;  // Ws[m] = gamma^m, m = 0 .. kC
  constexpr int kSlices = D / kWidth;
  constexpr int G = D / 64;  // tiles of the state's rows, 64 rows apart

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
  // the scale goes in with the values, or out with the outputs
  const float in_scale = op.scaled ? a.scale : 1.f, out_scale = op.scaled ? 1.f : a.scale;
  const T* q = (const T*)op.q.p + b * op.q.b + h * op.q.h;
  const T* k = (const T*)op.k.p + b * op.k.b + h * op.k.h;
  const T* v = (const T*)op.v.p + b * op.v.b + h * op.v.h + slice * kWidth;
  T* o = (T*)op.o.p + b * op.o.b + h * op.o.h + slice * kWidth;

  if (tid <= kC) Ws[tid] = power(g, tid);
  // the warp's rows and columns of every product; entry e of this lane in its tile nt of 8 columns is at
  // (at_row(e), at_col(nt, e))
  const int warp = tid >> 5, lane = tid & 31, wr = (warp >> 1) * 16, wc = (warp & 1) * 32;
  const auto at_row = [&](int e) { return wr + (lane >> 2) + (e >> 1) * 8; };
  const auto at_col = [&](int nt, int e) { return wc + 8 * nt + 2 * (lane & 3) + (e & 1); };
  float S[G][4][4];
#pragma unroll
  for (int gr = 0; gr < G; ++gr)
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = 64 * gr + at_row(e), c = slice * kWidth + at_col(nt, e);
        float s = 0.f;
        if (!STATES) {
          if (a.segs > 1)
            s = op.part[((long long)bh * a.segs + seg) * D * D + (op.part_t ? row * D + c : c * D + row)];
          else if (op.s_in)
            s = op.s_in[(long long)bh * D * D + row * op.s_r + c * op.s_c];
        }
        S[gr][nt][e] = s;
      }
  const int chunks = (n_seg + kC - 1) / kC;
  for (int cc = 0; cc < chunks; ++cc) {
    const int c = back ? chunks - 1 - cc : cc;
    const int base = t0 + c * kC, n = min(kC, n_seg - c * kC);
    __syncthreads();  // the chunk before has been read, S is in place
    // (all of a thread's reads of a tile are in flight at once)
    const auto load = [&](const T* from, long long stride, float* to, int pitch, auto width, float by) {
      constexpr int kW = decltype(width)::value / 4, kN = kC * kW / 256;
      float4 x[kN];
#pragma unroll
      for (int u = 0; u < kN; ++u) {
        const int i = tid + 256 * u, t = i / kW, f = (i % kW) * 4;
        // rows in the scan's order; those behind the end are zero
        x[u] = t < n ? load4(from + (base + (back ? n - 1 - t : t)) * stride + f, vec) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < kN; ++u) {
        const int i = tid + 256 * u;
        *(float4*)(to + i / kW * pitch + (i % kW) * 4) = make_float4(x[u].x * by, x[u].y * by, x[u].z * by, x[u].w * by);
      }
    };
    load(k, op.k.t, Ks, M::kRow, std::integral_constant<int, D>{}, 1.f);
    load(v, op.v.t, Vs, M::kCol, std::integral_constant<int, kWidth>{}, in_scale);
    if (!STATES) load(q, op.q.t, Qs, M::kRow, std::integral_constant<int, D>{}, 1.f);
    if (!STATES && cc == 0) {  // (the first state's reads run beside the first chunk's)
#pragma unroll
      for (int gr = 0; gr < G; ++gr)
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) Ss[(64 * gr + at_row(e)) * M::kCol + at_col(nt, e)] = S[gr][nt][e];
    }
    __syncthreads();
    if (!STATES) {
      const float *Qw = Qs + wr * M::kRow, *Kw = Ks + wc * M::kRow, *Pw = Ps + wr * M::kP;
      // (not a warp whose rows are all behind the end, or whose columns are all ahead of its rows)
      if (wr < n && wr + 15 >= wc) {
        float p[4][4] = {};
        add_product(p, D / 8, [&](int f, int r) { return Qw[r * M::kRow + f]; },
                    [&](int f, int j) { return Kw[j * M::kRow + f]; });
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int m = at_row(e) - at_col(nt, e);
            Ps[at_row(e) * M::kP + at_col(nt, e)] = m >= 0 ? p[nt][e] * Ws[m] : 0.f;
          }
      }
      __syncthreads();
      float acc[4][4] = {};
      if (wr < n && (cc > 0 || a.segs > 1 || op.s_in)) {  // (a first state of zero adds nothing)
        add_product(acc, D / 8, [&](int f, int r) { return Qw[r * M::kRow + f]; },
                    [&](int f, int c) { return Ss[f * M::kCol + wc + c]; });
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][e] *= Ws[at_row(e) + 1 - (back ? 1 : 0)];
      }
      // (columns behind the warp's last row are zero)
      add_product(acc, wr < n ? (wr + 16) / 8 : 0, [&](int j, int r) { return Pw[r * M::kP + j]; },
                  [&](int j, int c) { return Vs[j * M::kCol + wc + c]; });
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const int i = at_row(e);
        if (i >= n) continue;
        T* to = o + (base + (back ? n - 1 - i : i)) * op.o.t;
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
          store2(to + at_col(nt, 0), out_scale * acc[nt][e], out_scale * acc[nt][e + 1], vec);
      }
      __syncthreads();  // Ss has been read
    }
    const Carry carry(g, n);
#pragma unroll
    for (int gr = 0; gr < G; ++gr) {
      float add[4][4] = {};
      // (tokens behind the end are zero; their weights are any)
      add_product(add, (n + 7) / 8, [&](int j, int r) { return Ks[j * M::kRow + 64 * gr + wr + r]; },
                  [&](int j, int c) { return Vs[j * M::kCol + wc + c] * Ws[max(0, n - 1 - j + (back ? 1 : 0))]; });
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          S[gr][nt][e] = carry(S[gr][nt][e], add[nt][e]);
          if (!STATES) Ss[(64 * gr + at_row(e)) * M::kCol + at_col(nt, e)] = S[gr][nt][e];
        }
    }
  }
  if (STATES) {
    // the segment's own sum, at the segment that takes it
    float* to = op.part + ((long long)bh * a.segs + (back ? seg - 1 : seg + 1)) * D * D;
#pragma unroll
    for (int gr = 0; gr < G; ++gr)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          to[(slice * kWidth + at_col(nt, e)) * D + 64 * gr + at_row(e)] = S[gr][nt][e];
    return;
  }
  // rows behind the sequence's end
  for (int i = tid; i < (t1 - t0 - n_seg) * (kWidth / 4); i += 256) {
    const float z[4] = {};
    store4(o + (t0 + n_seg + i / (kWidth / 4)) * op.o.t + (i % (kWidth / 4)) * 4, z, vec);
  }
  if (op.s_out && seg == (back ? 0 : a.segs - 1)) {
#pragma unroll
    for (int gr = 0; gr < G; ++gr)
#pragma unroll
      for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          op.s_out[(long long)bh * D * D + (64 * gr + at_row(e)) * op.s_r + (slice * kWidth + at_col(nt, e)) * op.s_c] =
              S[gr][nt][e];
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
  float S = op.s_in ? op.s_in[(long long)bh * D * D + r * op.s_r + c * op.s_c] : 0.f;
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
cudaError_t launch_split(const Args& a, bool states, cudaStream_t st) {
  auto kern = states ? scan_split_kernel<T, D, true> : scan_split_kernel<T, D, false>;
  const int smem = Split<D>::kFloats * 4;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const long long grid = (long long)(a.last_op - a.first_op) * a.B * a.H * (D / kWidth) * (states ? a.segs - 1 : a.segs);
  return after(kern, (unsigned)grid, dim3(256), smem, st, 0, a);
}

// --------------------------------------------------------------- the split

// What a cut costs, in times of one chunk of a walk: a CTA's start, in the
// launch that forms the segments' own states too; a chunk there, which is keys
// and values alone; the two launches ahead of the scan's.
struct Cost {
  double start, states_start, states, launches;
};
// Fitted to the times of 1 to 64 segments (powers of two and some between) for
// 28 shapes of the bf16 and 16 of the fp32 kernel: 1 to 160 heads of 1000 to
// 131,072 tokens, both head sizes, forward and gradient.  The cut chosen takes
// 1.004 and 1.01 times the best one's time on average, 1.08 and 1.03 at most.
// (Without the starts, and with all scans counted where two are formed: 1.39 and
// 1.06; bf16, 40 heads of 4096 tokens, d = 128: 32 segments 223 us, whole 61; 64
// heads of 8192, d = 64: 64 segments 299, two 88, whole 96; gradient of 8 heads of
// 32,768, d = 128: 64 segments 392, nine 235, whole 441.)
constexpr Cost kCostTc = {1.5, 2.0, 0.8, 4.0}, kCostSplit = {0.3, 0.0, 0.5, 0.5};

// How many segments a sequence of `chunks` chunks is cut into, for `units`
// independent walks (scan, sequence, head, 64 state columns), the states ahead
// of the segments formed for `formed` of them.  A CTA walks one segment; the cut
// that takes the least time in rounds over the SMs is chosen.
int segments(long long units, long long formed, int chunks, int ctas, const Cost& k) {
  int best = 1;
  double least = 1e300;
  for (int s = 1; s <= kMaxSegs && s <= chunks; ++s) {
    const int per = (chunks + s - 1) / s;
    if ((chunks + per - 1) / per != s) continue;  // a cut with an empty last segment
    double time = std::ceil((double)units * s / ctas) * (k.start + per);
    if (s > 1) time += std::ceil((double)formed * (s - 1) / ctas) * (k.states_start + k.states * per) + k.launches;
    if (time < least) least = time, best = s;
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
  const long long walks = (long long)m->B * m->H * (m->d / kWidth);
  const int segs = segments(walks * nops, walks * (nops == 3 ? 2 : 1), chunks,
                            tc ? kSMs : kSMs * (m->d == 64 ? Split<64>::kCtas : Split<128>::kCtas), tc ? kCostTc : kCostSplit);
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

// nats_debug_decay_wait: of the next call on this host thread
thread_local int g_expire = -1;

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
  a.expire = g_expire;
  g_expire = -1;
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
      return m->d == 64 ? launch_split<__nv_bfloat16, 64>(a, states, st) : launch_split<__nv_bfloat16, 128>(a, states, st);
    return m->d == 64 ? launch_split<float, 64>(a, states, st) : launch_split<float, 128>(a, states, st);
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
             1, dims->d, 0, nullptr, 0, 0};
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
  const long long d = dims->d;
  Args a = {};
  a.nops = 3;
  a.op[0] = {tu, tv, tk, tokens(dq, dq_st), state_in, nullptr, d, 1, 0, nullptr, 0, 0};
  a.op[1] = {tv, tu, tq, tokens(dk, dk_st), dstate_out, nullptr, d, 1, 1, nullptr, 0, 1};
  a.op[2] = {tk, tq, tu, tokens(dv, dv_st), dstate_out, dstate_in, 1, d, 1, nullptr, 0, 1};
  return run(a, dims, log_decay, lens, ws, workspace_bytes, st);
}

nats_status nats_decay_attn_check(nats_stream_t stream) {
  int expired = 0;
  const int r = record_cuda_error(expired_waits(&expired, (cudaStream_t)stream));
  return r != NATS_OK ? (nats_status)r : expired ? NATS_ERR_INTERNAL : NATS_OK;
}

void nats_debug_decay_wait(int32_t chunk) { g_expire = chunk < 0 ? -1 : chunk; }

}  // extern "C"
