// paged_decode.cu - attention of one new token of each sequence over a paged
// key / value cache (nats_paged_decode):
//   out = sum_j p_j v_j,  p = softmax_j(scale q . k_j),  j < lens[b]
// for every query head, the Hq / Hk heads of a group reading one key head.
//
// Bound by HBM: every key and value row is read once, in one pass with the
// running maximum and sum of the softmax.  The rows are cut into 64-slot
// tiles, the tiles of all (sequence, key head) pairs are numbered in one
// line, and a fixed grid of CTAs takes equal runs of that line, whatever the
// lengths are; they are read on the device, so a captured call follows them.
// A run that covers a pair's tiles from first to last writes its output; the
// others leave (max, sum, weighted values) in the workspace, two slots a CTA
// (a run begins at most one pair that it does not finish and ends at most one
// that it did not begin), and decode_join_kernel adds them up in order.
#include <cmath>

#include "kernels.h"
#include "paged.cuh"

namespace nats {
namespace {

constexpr int kTile = 64;
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kSMs = 152;
constexpr int kMaxCtas = kSMs * 4;
constexpr int kMaxHeads = 16;  // query heads of a unit, at most
constexpr float kLog2e = 1.44269504088896340736f;

struct DecodeArgs {
  PagedView pg;
  const void *k, *v;  // pools
  const void* q;
  long long q_b, q_h;
  void* out;
  float* lse;
  int Hq, G, GT, ngroups;  // heads of a group, of a unit, units of a group
  float scale2;            // scale log2 e
  long long* prefix;       // [B + 1] tiles before each sequence
  float* lse_ws;           // [B, Hq]
  float* part_ml;          // [2 ctas, GT, 2]
  float* part_o;           // [2 ctas, GT, D]
  float* scores;           // [B, Hk, cap, G] or NULL
  float* weight;
};

__device__ __forceinline__ int tiles_of(int n) { return (n + kTile - 1) / kTile; }

// CTAs that share T tiles: none has an empty run.
__device__ __forceinline__ int ctas_used(long long T, int grid) { return (int)min(T, (long long)grid); }

// This CTA's run [s, e) of the tile line, and the sequence b0 (with `pre`
// tiles before it) in which it starts.  Every thread calls it; CTA 0 also
// writes the prefix sums and reports lengths out of range.
struct Run {
  long long s, e, pre;
  int b0;
};
__device__ __forceinline__ Run my_run(const PagedView& pg, int U, long long* prefix) {
  __shared__ long long red[kWarps + 1], found[2];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long mine = 0;
  for (int b = tid; b < pg.B; b += kThreads) mine += tiles_of(pg.length(b));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, o);
  if (lane == 0) red[warp] = mine;
  if (tid == 0) found[0] = found[1] = 0;
  __syncthreads();
  long long total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += red[w];
  Run r;
  const long long T = total * U;
  const int n = ctas_used(T, gridDim.x), i = min((int)blockIdx.x, n);
  r.s = n ? T * i / n : 0;
  r.e = i < n ? T * (i + 1) / n : r.s;
  const bool first = blockIdx.x == 0 && prefix;
  long long run = 0;
  for (int b1 = 0; b1 < pg.B && (first || run * U <= r.s); b1 += kThreads) {
    const int b = b1 + tid;
    long long x = 0;
    if (b < pg.B) {
      x = tiles_of(pg.length(b));
      if (first) {
        const int raw = pg.lens[b];
        if (raw < 0 || raw > pg.cap()) *pg.err = 1;
      }
    }
    const long long own = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) red[warp] = x;
    __syncthreads();
    long long chunk = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) x += red[w];
      chunk += red[w];
    }
    const long long before = run + x - own;
    if (b < pg.B) {
      if (first) prefix[b] = before;
      if (before * U <= r.s && r.s < (before + own) * U) found[0] = b, found[1] = before;
    }
    run += chunk;
  }
  if (first && tid == 0) prefix[pg.B] = total;
  __syncthreads();
  r.b0 = (int)found[0];
  r.pre = found[1];
  return r;
}

template <typename T>
__device__ __forceinline__ void load8(const T* p, float* o);
template <>
__device__ __forceinline__ void load8(const float* p, float* o) {
  const float4 a = *(const float4*)p, b = *(const float4*)(p + 4);
  o[0] = a.x, o[1] = a.y, o[2] = a.z, o[3] = a.w;
  o[4] = b.x, o[5] = b.y, o[6] = b.z, o[7] = b.w;
}

// e^(m - M) factors in base 2, with 0 for an empty part
__device__ __forceinline__ float part_scale(float m, float M) { return m == -INFINITY ? 0.f : exp2f(m - M); }

// A unit's result from the CTA's warps (shared memory) to the output or to
// partial slot `slot` (-1: the output).
template <typename T, int D, int GT>
__device__ __forceinline__ void finish_unit(const DecodeArgs& a, const float* so, const float* sml, int b, int h0,
                                            int heads, long long slot) {
  // so [kWarps][GT][D], sml [kWarps][GT][2]
  for (int i = threadIdx.x; i < GT * D; i += kThreads) {
    const int g = i / D, e = i % D;
    if (g >= heads) break;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sml[(w * GT + g) * 2]);
    float l = 0.f, o = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = part_scale(sml[(w * GT + g) * 2], M);
      l += f * sml[(w * GT + g) * 2 + 1];
      o += f * so[(w * GT + g) * D + e];
    }
    if (slot < 0) {
      ((T*)a.out)[((long long)b * a.Hq + h0 + g) * D + e] = from_f32<T>(l == 0.f ? 0.f : o / l);
      if (e == 0) {
        const float v = l == 0.f ? -INFINITY : M + log2f(l);
        a.lse_ws[(long long)b * a.Hq + h0 + g] = v;
        if (a.lse) a.lse[(long long)b * a.Hq + h0 + g] = v;
      }
    } else {
      a.part_o[(slot * GT + g) * D + e] = o;
      if (e == 0) {
        a.part_ml[(slot * GT + g) * 2] = M;
        a.part_ml[(slot * GT + g) * 2 + 1] = l;
      }
    }
  }
}

// Eight entries of a row a lane, D / 8 lanes a row, fp32 arithmetic.
template <typename T, int D, int GT>
__global__ void __launch_bounds__(kThreads) decode_simt_kernel(DecodeArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  __shared__ float so[kWarps * GT * D], sml[kWarps * GT * 2];
  const int U = a.pg.Hk * a.ngroups;
  const Run run = my_run(a.pg, U, a.prefix);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane % LPR, sub = lane / LPR;
  long long cur = run.s, pre = run.pre;
  int b = run.b0;
  while (cur < run.e) {
    const int n = a.pg.length(b), nt = tiles_of(n);
    if (cur >= (pre + nt) * U) {
      pre += nt;
      ++b;
      continue;
    }
    const long long local = cur - pre * U;
    const int u = (int)(local / nt), t0 = (int)(local % nt);
    const int t1 = (int)min((long long)nt, t0 + (run.e - cur));
    const int hk = u / a.ngroups, g0 = (u % a.ngroups) * GT;
    const int heads = min(GT, a.G - g0), h0 = hk * a.G + g0;
    float q[GT][8], o[GT][8], mx[GT], sum[GT];
#pragma unroll
    for (int g = 0; g < GT; ++g) {
      mx[g] = -INFINITY, sum[g] = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) q[g][i] = o[g][i] = 0.f;
      if (g < heads) {
        load8((const T*)a.q + b * a.q_b + (h0 + g) * a.q_h + 8 * l, q[g]);
#pragma unroll
        for (int i = 0; i < 8; ++i) q[g][i] *= a.scale2;
      }
    }
    for (int t = t0; t < t1; ++t) {
      const int j0 = t * kTile + warp * 16;
      if (j0 >= n) break;
      const int pg = a.pg.page_of(b, j0 / a.pg.page);
      if (pg < 0 && lane == 0) *a.pg.err = 1;
      const long long row0 = pg < 0 ? 0 : a.pg.row(pg, hk, j0 % a.pg.page);
#pragma unroll 4
      for (int st = 0; st < 16; st += RPW) {
        const int j = j0 + st + sub;
        const bool on = j < n && pg >= 0;
        float k[8], v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) k[i] = v[i] = 0.f;
        if (on) {
          load8((const T*)a.k + (row0 + st + sub) * D + 8 * l, k);
          load8((const T*)a.v + (row0 + st + sub) * D + 8 * l, v);
        }
#pragma unroll
        for (int g = 0; g < GT; ++g) {
          float s = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) s = fmaf(q[g][i], k[i], s);
#pragma unroll
          for (int x = LPR / 2; x > 0; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
          if (!on) s = -INFINITY;
          if (a.scores && l == 0 && j < n && g < heads)
            a.scores[(((long long)b * a.pg.Hk + hk) * a.pg.cap() + j) * a.G + g0 + g] = s;
          const float mn = fmaxf(mx[g], s);
          const float f = part_scale(mx[g], mn), p = s == -INFINITY ? 0.f : exp2f(s - mn);
          mx[g] = mn;
          sum[g] = sum[g] * f + p;
#pragma unroll
          for (int i = 0; i < 8; ++i) o[g][i] = fmaf(o[g][i], f, p * v[i]);
        }
      }
    }
    // the rows of a warp, then its warps
#pragma unroll
    for (int g = 0; g < GT; ++g) {
      float M = mx[g];
#pragma unroll
      for (int x = 16; x >= LPR; x >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, x));
      const float f = part_scale(mx[g], M);
      sum[g] *= f;
#pragma unroll
      for (int x = 16; x >= LPR; x >>= 1) sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], x);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float y = o[g][i] * f;
#pragma unroll
        for (int x = 16; x >= LPR; x >>= 1) y += __shfl_xor_sync(0xffffffffu, y, x);
        if (sub == 0) so[(warp * GT + g) * D + 8 * l + i] = y;
      }
      if (lane == 0) sml[(warp * GT + g) * 2] = M, sml[(warp * GT + g) * 2 + 1] = sum[g];
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == nt;
    finish_unit<T, D, GT>(a, so, sml, b, h0, heads, whole ? -1 : 2LL * blockIdx.x + (cur == run.s ? 0 : 1));
    __syncthreads();
    cur += t1 - t0;
  }
}

// ------------------------------------------------ bf16: tensor-core products

// Sixteen bytes of a page, read once: past L1.
__device__ __forceinline__ uint4 ldg_once(const void* p) {
  uint4 u;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
      : "l"(p));
  return u;
}

// c += A B, A 16 x 16 and B 16 x 8 bf16, fp32 accumulators
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// the transpose of an 8 x 8 matrix of 16-bit entries held two a lane
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *(const uint32_t*)&v;
}

// how far a score may rise above the running maximum (in powers of two)
// before the sums are rescaled: 2^8 leaves fp32 its full precision
constexpr float kSlack = 8.f;

// A unit of up to 8 NH heads.  Each warp takes 16 slots of every tile, on its
// own: both products run with the slots or the entries on the rows of the
// 16 x 8 x 16 instruction and the heads on its 8 columns,
//   S^T [16 slots x 8 heads] += K [16 x 16 entries] Q^T,
//   O^T [16 entries x 8 heads] += V^T [16 x 16 slots] P^T,
// so few heads waste little, and which entry (slot) carries which index of a
// sum is free, so that every operand is a plain 16-byte load of a row:
//   K: lane 4g + c holds entries 32 x + 8 c .. + 7 of slots g and g + 8 for
//      each 32-entry block x, the same entries that it holds of head g's q;
//   V: it holds entries 8 g .. + 7 (and 64 + 8 g .. + 7) of slots 2c, 2c + 1,
//      2c + 8, 2c + 9, and pairs of slots are packed with byte permutes.
// No shared memory in the loop.  P moves from S^T's to P^T's layout by an
// 8 x 8 transpose; it is carried as two bf16, high and low part, so that the
// rounding of p (2^-8 each) does not double the output's own.
// A tile's K registers are refilled for the next tile as soon as the scores
// are done, V's when the values are: about 8 KB in flight a warp.
template <int D, int NH>
__global__ void __launch_bounds__(kThreads, NH == 1 ? 3 : 2) decode_mma_kernel(DecodeArgs a) {
  constexpr int KB = D / 32;        // 32-entry blocks of a key row
  constexpr int VS = D / 64;        // 8-entry segments of a value row a lane holds
  constexpr int MT = D / 16;        // 16-entry tiles of O^T
  constexpr int GT = 8 * NH;
  __shared__ float so[kWarps * GT * D], sml[kWarps * GT * 2];
  const int U = a.pg.Hk * a.ngroups;
  const Run run = my_run(a.pg, U, a.prefix);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const __nv_bfloat16 *kp = (const __nv_bfloat16*)a.k, *vp = (const __nv_bfloat16*)a.v;
  long long cur = run.s, pre = run.pre;
  int b = run.b0;
  while (cur < run.e) {
    const int n = a.pg.length(b), nt = tiles_of(n);
    if (cur >= (pre + nt) * U) {
      pre += nt;
      ++b;
      continue;
    }
    const long long local = cur - pre * U;
    const int u = (int)(local / nt), t0 = (int)(local % nt);
    const int t1 = (int)min((long long)nt, t0 + (run.e - cur));
    const int hk = u / a.ngroups, g0 = (u % a.ngroups) * GT;
    const int heads = min(GT, a.G - g0), h0 = hk * a.G + g0;
    uint4 q[NH][KB];
    float o[NH][MT][4], mx[NH][2], sum[NH][2];
#pragma unroll
    for (int x = 0; x < NH; ++x) {
#pragma unroll
      for (int y = 0; y < KB; ++y) {
        q[x][y] = make_uint4(0, 0, 0, 0);
        if (8 * x + g < heads)
          q[x][y] = *(const uint4*)((const __nv_bfloat16*)a.q + b * a.q_b + (h0 + 8 * x + g) * a.q_h + 32 * y + 8 * c);
      }
#pragma unroll
      for (int y = 0; y < MT; ++y)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[x][y][i] = 0.f;
      mx[x][0] = mx[x][1] = -INFINITY;
      sum[x][0] = sum[x][1] = 0.f;
    }
    uint4 k[2][KB], v[4][VS];
    // row of this warp's first slot in tile t, or -1: past the end or without a page
    auto first_row = [&](int t) -> long long {
      const int j0 = t * kTile + warp * 16;
      if (t >= t1 || j0 >= n) return -1;
      const int pg = a.pg.page_of(b, j0 / a.pg.page);
      if (pg < 0) {
        if (lane == 0) *a.pg.err = 1;
        return -1;
      }
      return a.pg.row(pg, hk, j0 % a.pg.page);
    };
    auto load_k = [&](long long row) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int y = 0; y < KB; ++y)
          k[i][y] = row < 0 ? make_uint4(0, 0, 0, 0) : ldg_once(kp + (row + g + 8 * i) * D + 32 * y + 8 * c);
    };
    // values of slots behind the sequence are zero: 0 x NaN would not be
    auto load_v = [&](long long row, int left) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 2 * c + (i & 1) + 8 * (i >> 1);
#pragma unroll
        for (int y = 0; y < VS; ++y)
          v[i][y] = row < 0 || r >= left ? make_uint4(0, 0, 0, 0) : ldg_once(vp + (row + r) * D + 64 * y + 8 * g);
      }
    };
    long long row = first_row(t0), next = first_row(t0 + 1);
    load_k(row);
    load_v(row, n - t0 * kTile - warp * 16);
    for (int t = t0; t < t1; ++t) {
      const int j0 = t * kTile + warp * 16;
      const long long after = first_row(t + 2);
      float s[NH][4];
#pragma unroll
      for (int x = 0; x < NH; ++x) {
        s[x][0] = s[x][1] = s[x][2] = s[x][3] = 0.f;
#pragma unroll
        for (int y = 0; y < KB; ++y) {
          mma16816(s[x], k[0][y].x, k[1][y].x, k[0][y].y, k[1][y].y, q[x][y].x, q[x][y].y);
          mma16816(s[x], k[0][y].z, k[1][y].z, k[0][y].w, k[1][y].w, q[x][y].z, q[x][y].w);
        }
      }
      load_k(next);
      const bool lo = row >= 0 && j0 + g < n, hi = row >= 0 && j0 + g + 8 < n;
      uint32_t ph[NH][2], pl[NH][2];
      bool rises = false;
#pragma unroll
      for (int x = 0; x < NH; ++x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[x][i] = (i < 2 ? lo : hi) ? s[x][i] * a.scale2 : -INFINITY;
        if (a.scores) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = j0 + g + 8 * (i >> 1), h = 8 * x + 2 * c + (i & 1);
            if (j < n && h < heads)
              a.scores[(((long long)b * a.pg.Hk + hk) * a.pg.cap() + j) * a.G + g0 + h] = s[x][i];
          }
        }
        rises |= fmaxf(s[x][0], s[x][2]) > mx[x][0] + kSlack || fmaxf(s[x][1], s[x][3]) > mx[x][1] + kSlack;
      }
      if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
        for (int x = 0; x < NH; ++x)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float m = fmaxf(s[x][i], s[x][i + 2]);
#pragma unroll
            for (int z = 4; z < 32; z <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, z));
            m = fmaxf(m, mx[x][i]);
            const float f = part_scale(mx[x][i], m);
            mx[x][i] = m;
            sum[x][i] *= f;
#pragma unroll
            for (int y = 0; y < MT; ++y) o[x][y][i] *= f, o[x][y][i + 2] *= f;
          }
      }
#pragma unroll
      for (int x = 0; x < NH; ++x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          // (a head without a slot yet has no maximum to subtract: its scores are all -inf)
          s[x][i] = s[x][i] == -INFINITY ? 0.f : exp2f(s[x][i] - mx[x][i & 1]);
          sum[x][i & 1] += s[x][i];
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w = pack_bf16(s[x][2 * i], s[x][2 * i + 1]);
          const float l0 = s[x][2 * i] - __uint_as_float(w << 16), l1 = s[x][2 * i + 1] - __uint_as_float(w & 0xffff0000u);
          ph[x][i] = transpose8(w);
          pl[x][i] = transpose8(pack_bf16(l0, l1));
        }
      }
#pragma unroll
      for (int y = 0; y < MT; ++y) {
        // rows g and g + 8 of tile y: entries 8g + y and 64 + 8g + y (D = 64: 8g + y and 8g + 4 + y)
        const int ya = y, sa = 0, yb = D == 128 ? y : y + 4, sb = D == 128 ? VS - 1 : 0;
        auto pair = [&](int s0, int e, int sg) {
          const uint32_t* r0 = (const uint32_t*)&v[s0][sg];
          const uint32_t* r1 = (const uint32_t*)&v[s0 + 1][sg];
          return __byte_perm(r0[e / 2], r1[e / 2], e % 2 ? 0x7632 : 0x5410);
        };
        const uint32_t a0 = pair(0, ya, sa), a1 = pair(0, yb, sb), a2 = pair(2, ya, sa), a3 = pair(2, yb, sb);
#pragma unroll
        for (int x = 0; x < NH; ++x) {
          mma16816(o[x][y], a0, a1, a2, a3, ph[x][0], ph[x][1]);
          mma16816(o[x][y], a0, a1, a2, a3, pl[x][0], pl[x][1]);
        }
      }
      load_v(next, n - j0 - kTile);
      row = next;
      next = after;
    }
#pragma unroll
    for (int x = 0; x < NH; ++x) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int z = 4; z < 32; z <<= 1) sum[x][i] += __shfl_xor_sync(0xffffffffu, sum[x][i], z);
        const int h = 8 * x + 2 * c + i;
        if (g == 0) sml[(warp * GT + h) * 2] = mx[x][i], sml[(warp * GT + h) * 2 + 1] = sum[x][i];
#pragma unroll
        for (int y = 0; y < MT; ++y) {
          float* at = so + (warp * GT + h) * D + 8 * g + y;
          at[0] = o[x][y][i];
          at[D == 128 ? 64 : 4] = o[x][y][i + 2];
        }
      }
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == nt;
    finish_unit<__nv_bfloat16, D, GT>(a, so, sml, b, h0, heads, whole ? -1 : 2LL * blockIdx.x + (cur == run.s ? 0 : 1));
    __syncthreads();
    cur += t1 - t0;
  }
}

// The CTA whose run holds tile x of the line (the run of CTA i of n is
// [i T / n, (i + 1) T / n)).
__device__ __forceinline__ int cta_of(long long x, long long T, int n) { return (int)(((x + 1) * n - 1) / T); }

// A warp per (sequence, query head): joins the partials of a unit that lies
// in more than one run, and writes the rows of empty sequences.
template <typename T, int D>
__global__ void __launch_bounds__(kThreads) decode_join_kernel(DecodeArgs a, int ctas) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const long long i = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= (long long)a.pg.B * a.Hq) return;
  const int b = (int)(i / a.Hq), h = (int)(i % a.Hq);
  const long long pre = a.prefix[b], nt = a.prefix[b + 1] - pre, total = a.prefix[a.pg.B];
  const int U = a.pg.Hk * a.ngroups;
  float o[E], M = -INFINITY, l = 0.f;
#pragma unroll
  for (int x = 0; x < E; ++x) o[x] = 0.f;
  if (nt > 0) {
    const int hk = h / a.G, g = (h % a.G) % a.GT, u = hk * a.ngroups + (h % a.G) / a.GT;
    const long long x0 = pre * U + u * nt, T_ = total * U;
    ctas = ctas_used(T_, ctas);
    const int c0 = cta_of(x0, T_, ctas), c1 = cta_of(x0 + nt - 1, T_, ctas);
    if (c0 == c1) return;  // written by its CTA
    // a CTA whose run begins in the unit (or before it with the unit as its first) used slot 0
    const long long first = 2LL * c0 + (T_ * c0 / ctas == x0 ? 0 : 1);
    for (int c = c0; c <= c1; ++c) {
      const long long slot = c == c0 ? first : 2LL * c;
      M = fmaxf(M, a.part_ml[(slot * a.GT + g) * 2]);
    }
    for (int c = c0; c <= c1; ++c) {
      const long long slot = c == c0 ? first : 2LL * c;
      const float f = part_scale(a.part_ml[(slot * a.GT + g) * 2], M);
      l += f * a.part_ml[(slot * a.GT + g) * 2 + 1];
#pragma unroll
      for (int x = 0; x < E; ++x) o[x] += f * a.part_o[(slot * a.GT + g) * D + lane * E + x];
    }
  }
#pragma unroll
  for (int x = 0; x < E; ++x) ((T*)a.out)[i * D + lane * E + x] = from_f32<T>(l == 0.f ? 0.f : o[x] / l);
  if (lane == 0) {
    const float v = l == 0.f ? -INFINITY : M + log2f(l);
    a.lse_ws[i] = v;
    if (a.lse) a.lse[i] = v;
  }
}

// weight[slot] += sum over the group's heads of 2^(score - lse): every slot
// has one thread, so nothing is summed in an order that varies.
__global__ void __launch_bounds__(kThreads) decode_weight_kernel(DecodeArgs a) {
  const int U = a.pg.Hk;
  const Run run = my_run(a.pg, U, nullptr);
  long long cur = run.s, pre = run.pre;
  int b = run.b0;
  while (cur < run.e) {
    const int n = a.pg.length(b), nt = tiles_of(n);
    if (cur >= (pre + nt) * U) {
      pre += nt;
      ++b;
      continue;
    }
    const long long local = cur - pre * U;
    const int hk = (int)(local / nt), t0 = (int)(local % nt);
    const int t1 = (int)min((long long)nt, t0 + (run.e - cur));
    const float* lse = a.lse_ws + (long long)b * a.Hq + hk * a.G;
    for (int j = t0 * kTile + threadIdx.x; j < min(n, t1 * kTile); j += kThreads) {
      const int pg = a.pg.page_of(b, j / a.pg.page);
      if (pg < 0) continue;
      const float* s = a.scores + (((long long)b * a.pg.Hk + hk) * a.pg.cap() + j) * a.G;
      float w = 0.f;
      for (int g = 0; g < a.G; ++g) w += s[g] == -INFINITY ? 0.f : exp2f(s[g] - lse[g]);
      float* at = a.weight + a.pg.row(pg, hk, j % a.pg.page);
      *at += w;
    }
    cur += t1 - t0;
  }
}

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

size_t layout(const nats_paged_cache* c, int Hq, bool accumulate, char* base, DecodeArgs* a) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = base ? base + off : nullptr;
    off += align_up(bytes);
    return p;
  };
  DecodeArgs d = {};
  d.prefix = (long long*)take(8 * ((size_t)c->B + 1));
  d.lse_ws = (float*)take(4 * (size_t)c->B * Hq);
  d.part_ml = (float*)take(4 * 2 * (size_t)kMaxCtas * kMaxHeads * 2);
  d.part_o = (float*)take(4 * 2 * (size_t)kMaxCtas * kMaxHeads * c->d);
  d.scores = accumulate ? (float*)take(4 * (size_t)c->B * Hq * c->max_pages * c->page) : nullptr;
  if (a) *a = d;
  return off;
}

nats_status check_decode(const nats_paged_cache* c, int32_t Hq, int32_t accumulate) {
  const nats_status s = check_cache(c);
  if (s != NATS_OK) return s;
  if (Hq < 0 || Hq % c->Hk != 0) return NATS_ERR_SHAPE;
  if ((long long)c->B * Hq > (1LL << 31) - 1) return NATS_ERR_UNSUPPORTED;
  if (accumulate && (double)c->B * Hq * c->max_pages * c->page > 1099511627776.0) return NATS_ERR_UNSUPPORTED;
  return NATS_OK;
}

// fp32: units of up to four heads on the lanes.  bf16: eight heads a unit on
// the tensor cores, sixteen where a group has more than eight (two products'
// worth of registers, but the rows are read once).
template <int D>
cudaError_t launch(DecodeArgs& a, int dtype, cudaStream_t st) {
  int ctas;
  if (dtype == NATS_BF16) {
    a.GT = a.G <= 8 ? 8 : 16;
    a.ngroups = (a.G + a.GT - 1) / a.GT;
    ctas = kSMs * (a.GT == 8 ? 3 : 2);
    if (a.GT == 8)
      decode_mma_kernel<D, 1><<<ctas, kThreads, 0, st>>>(a);
    else
      decode_mma_kernel<D, 2><<<ctas, kThreads, 0, st>>>(a);
  } else {
    ctas = kSMs * 3;
    a.GT = a.G == 1 ? 1 : a.G == 2 ? 2 : 4;
    a.ngroups = (a.G + a.GT - 1) / a.GT;
    if (a.GT == 1)
      decode_simt_kernel<float, D, 1><<<ctas, kThreads, 0, st>>>(a);
    else if (a.GT == 2)
      decode_simt_kernel<float, D, 2><<<ctas, kThreads, 0, st>>>(a);
    else
      decode_simt_kernel<float, D, 4><<<ctas, kThreads, 0, st>>>(a);
  }
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const long long rows = (long long)a.pg.B * a.Hq;
  const unsigned grid = (unsigned)((rows + kWarps - 1) / kWarps);
  if (dtype == NATS_BF16)
    decode_join_kernel<__nv_bfloat16, D><<<grid, kThreads, 0, st>>>(a, ctas);
  else
    decode_join_kernel<float, D><<<grid, kThreads, 0, st>>>(a, ctas);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.scores) return e;
  decode_weight_kernel<<<kSMs * 8, kThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace
}  // namespace nats

using namespace nats;

extern "C" {

size_t nats_paged_decode_workspace_size(const nats_paged_cache* cache, int32_t Hq, int32_t accumulate) {
  if (check_decode(cache, Hq, accumulate) != NATS_OK) return 0;
  return layout(cache, Hq, accumulate != 0, nullptr, nullptr);
}

nats_status nats_paged_decode(const nats_paged_cache* cache, int32_t Hq, float scale, const void* q,
                              int64_t q_stride_b, int64_t q_stride_h, void* out, float* lse, int32_t accumulate,
                              void* workspace, size_t workspace_bytes, nats_stream_t stream) {
  nats_status s = check_decode(cache, Hq, accumulate);
  if (s != NATS_OK) return s;
  if (!std::isfinite(scale) || scale < 0.f) return NATS_ERR_VALUE;
  if (cache->B == 0 || Hq == 0) return NATS_OK;
  s = check_cache_pointers(cache);
  if (s != NATS_OK) return s;
  if (!q || !out || !workspace || (accumulate && cache->n_pages > 0 && !cache->weight)) return NATS_ERR_NULL;
  const int es = cache->dtype == NATS_BF16 ? 2 : 4;
  if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15u) return NATS_ERR_ALIGN;
  if ((q_stride_b * es) % 16 != 0 || (q_stride_h * es) % 16 != 0 || ((uintptr_t)lse & 3u)) return NATS_ERR_ALIGN;
  DecodeArgs a;
  if (workspace_bytes < layout(cache, Hq, accumulate != 0, (char*)workspace, &a)) return NATS_ERR_WORKSPACE;
  a.pg = view_of(cache), a.k = cache->k_pages, a.v = cache->v_pages, a.weight = cache->weight;
  a.q = q, a.q_b = q_stride_b, a.q_h = q_stride_h, a.out = out, a.lse = lse;
  a.Hq = Hq, a.G = Hq / cache->Hk;
  a.scale2 = (scale > 0.f ? scale : 1.0f / std::sqrt((float)cache->d)) * kLog2e;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = cache->d == 128 ? launch<128>(a, cache->dtype, st) : launch<64>(a, cache->dtype, st);
  return (nats_status)record_cuda_error(e);
}

}  // extern "C"
