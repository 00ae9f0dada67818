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
// that it did not begin), and decode_finish_kernel adds them up in order.
//
// Measured on one GB300 (HBM copy rate 6.8 TB/s): 32 contexts of 3000 to 8192
// slots, 32 query and 8 key heads of 128, bf16: 112 us, 6.2 TB/s, the tensor
// pipe 18 % busy; 4 contexts of up to 131,072 with weights 289 us, 5.7 TB/s (and
// 134 MB of scores between the kernels); fp32 the same way, 5.8 TB/s at 8 x
// 16384; 517 slots of one sequence 9.1 us, the latencies of the two kernels one
// after the other.
#include <cmath>

#include "kernels.h"
#include "launch.cuh"
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
  long long* prefix;       // [B + 2] tiles before each sequence, all, and the CTAs that share them
  float2* ml_ws;           // [B, Hq] maximum and 1 / sum of the units of one CTA
  float* part_ml;          // [2 ctas, GT, 2] maximum and sum
  float* part_o;           // [2 ctas, GT, D]
  float* scores;           // [B, Hk, cap, G], or pooled [n_pages, Hk, page, G], or NULL: q . k, not yet scaled
  bool pooled;
  float* weight;
};

// The scores of a unit of sequence b and key head hk: from scores_of on, those of
// slot j, in row `row` of the pool, G times scores_row further.
__device__ __forceinline__ float* scores_of(const DecodeArgs& a, int b, int hk) {
  return a.scores + (a.pooled ? 0 : ((long long)b * a.pg.Hk + hk) * a.pg.cap() * a.G);
}
__device__ __forceinline__ long long scores_row(const DecodeArgs& a, int j, int row) { return a.pooled ? row : j; }

__device__ __forceinline__ int tiles_of(int n) { return (int)((uint32_t)(n + kTile - 1) / kTile); }

// a / b and a % b, 32-bit where a allows
__device__ __forceinline__ long long div_rem(long long a, int b, int* rest) {
  if ((unsigned long long)a >> 32) {
    *rest = (int)(a % b);
    return a / b;
  }
  const uint32_t q = (uint32_t)a / (uint32_t)b;
  *rest = (int)((uint32_t)a - q * (uint32_t)b);
  return q;
}
// a * b / c for 0 <= a, b and 0 < c
__device__ __forceinline__ long long mul_div(long long a, int b, long long c) {
  const long long ab = a * b;
  return (ab | c) >> 32 ? ab / c : (long long)((uint32_t)ab / (uint32_t)c);
}

// CTAs that share T tiles: none has an empty run.
__device__ __forceinline__ int ctas_used(long long T, int grid) { return (int)min(T, (long long)grid); }
// Of the decode kernel: runs of at least four tiles where units would otherwise
// fall into more than 32 parts each, whose joining then costs more than the
// shorter runs save (1 x 8192 slots, 2 key heads: 18 us without, 12.6 with).
__device__ __forceinline__ int decode_ctas(long long T, long long units, int grid) {
  return ctas_used(min(T, max(32 * units, T / 4)), grid);
}

// This CTA's run [s, e) of the tile line, and the sequence b0 (with `pre`
// tiles before it) in which it starts.  Every thread calls it; CTA 0 also
// writes the prefix sums and reports lengths out of range.
struct Run {
  long long s, e, pre;
  int b0;
};
__device__ __forceinline__ Run my_run(const PagedView& pg, int U, long long* prefix) {
  __shared__ long long red[kWarps], found[2];
  __shared__ int red_seqs[kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool first = blockIdx.x == 0;
  long long total = 0, units = 0, run = 0;
  Run r = {0, 0, 0, 0};
  int n = 0;
  // a first pass for the sums, a second one for the place; the chunk of the
  // first pass is kept, so that a batch of up to kThreads sequences is read once
  long long mine = 0;
  int seqs = 0, kept = 0;
  for (int b = tid; b < pg.B; b += kThreads) {
    kept = tiles_of(pg.length(b));
    mine += kept, seqs += kept > 0;
  }
  for (int b1 = 0; b1 == 0 || (b1 < pg.B && (first || run * U <= r.s)); b1 += kThreads) {
    const int b = b1 + tid;
    int own = 0;
    if (b < pg.B) {
      own = pg.B <= kThreads ? kept : tiles_of(pg.length(b));
      if (first) {
        const int raw = pg.lens[b];
        if (raw < 0 || raw > pg.cap()) *pg.err = 1;
      }
    }
    // (up to 2^24 tiles a sequence: 32 of them fit 32 bits)
    uint32_t x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    long long all = x;
    if (b1 == 0) {
      if (pg.B > kThreads) {
        all = mine;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
      }
      seqs = __reduce_add_sync(0xffffffffu, seqs);
      if (lane == 31) red[warp] = all, red_seqs[warp] = seqs;
      if (tid == 0) found[0] = found[1] = 0;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) total += red[w], units += red_seqs[w];
      const long long T = total * U;
      n = decode_ctas(T, units * U, gridDim.x);
      const int i = min((int)blockIdx.x, n);
      r.s = n ? mul_div(T, i, n) : 0;
      r.e = i < n ? mul_div(T, i + 1, n) : r.s;
    }
    if (pg.B > kThreads) {  // (else red holds the warps' sums of this chunk already)
      __syncthreads();
      if (lane == 31) red[warp] = x;
      __syncthreads();
    }
    long long before = run + x - own, chunk = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += red[w];
      chunk += red[w];
    }
    if (b < pg.B) {
      if (first) prefix[b] = before;
      if (before * U <= r.s && r.s < (before + own) * U) found[0] = b, found[1] = before;
    }
    run += chunk;
  }
  if (first && tid == 0) prefix[pg.B] = total, prefix[pg.B + 1] = n;
  __syncthreads();
  r.b0 = (int)found[0];
  r.pre = found[1];
  return r;
}

// 2^x, the hardware's approximation (2 ulp; results below 2^-126 are 0)
__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void store4(float* p, float a, float b, float c, float d) {
  *(float4*)p = make_float4(a, b, c, d);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, float a, float b, float c, float d) {
  const __nv_bfloat162 x = __floats2bfloat162_rn(a, b), y = __floats2bfloat162_rn(c, d);
  *(uint2*)p = make_uint2(*(const uint32_t*)&x, *(const uint32_t*)&y);
}
// The maximum of no scores: below any real one, and finite, so that a score of
// -inf less it is still -inf and two of it subtract to 0 (their sums are 0).
constexpr float kNoMax = -1e38f;
// the factor that brings sums taken at maximum m to maximum M >= m
__device__ __forceinline__ float part_scale(float m, float M) { return pow2(m - M); }
__device__ __forceinline__ float lse_of(float M, float l) { return l == 0.f ? -INFINITY : M + log2f(l); }
// 2^(scaled score - maximum m) of the raw score s.  The scaled score is not
// rounded before the maximum is subtracted; the maximum is a rounded one, but the
// same for a sum and all that is divided by it, so that its rounding cancels.
__device__ __forceinline__ float weight_of(float s, float scale2, float m) { return pow2(fmaf(s, scale2, -m)); }

// Where entry e of a row stands in shared memory: rows padded to D + 4, and
// within a row such that the lanes that hold neighbouring entry tiles (X::place)
// write to different banks.
template <int D>
constexpr int kPitch = D + 4;

// A unit's result from W warps (shared memory: so [W][GT][pitch], sml [W][GT][2])
// to the output or to partial slot `slot` (-1: the output), four entries a
// thread of 32 W.
template <class X, int GT, int W>
__device__ __forceinline__ void finish_unit(const DecodeArgs& a, const float* so, const float* sml, int b, int h0,
                                            int heads, long long slot, int tid) {
  using T = typename X::T;
  constexpr int D = X::kD;
  for (int i = tid; i < heads * (D / 4); i += 32 * W) {
    const int g = i / (D / 4), e = 4 * (i % (D / 4));
    float f[W], M = kNoMax, l = 0.f, o[4] = {};
#pragma unroll
    for (int w = 0; w < W; ++w) f[w] = sml[(w * GT + g) * 2], M = fmaxf(M, f[w]);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      f[w] = part_scale(f[w], M);
      l += f[w] * sml[(w * GT + g) * 2 + 1];
#pragma unroll
      for (int x = 0; x < 4; ++x) o[x] += f[w] * so[(w * GT + g) * kPitch<D> + X::place(e + x)];
    }
    if (slot < 0) {
      const float r = l == 0.f ? 0.f : 1.f / l;
      T* out = (T*)a.out + ((long long)b * a.Hq + h0 + g) * D + e;
      store4(out, o[0] * r, o[1] * r, o[2] * r, o[3] * r);
      if (e == 0) {
        a.ml_ws[(long long)b * a.Hq + h0 + g] = make_float2(M, r);
        if (a.lse) a.lse[(long long)b * a.Hq + h0 + g] = lse_of(M, l);
      }
    } else {
      *(float4*)(a.part_o + (slot * GT + g) * D + e) = make_float4(o[0], o[1], o[2], o[3]);
      if (e == 0) *(float2*)(a.part_ml + (slot * GT + g) * 2) = make_float2(M, l);
    }
  }
}

// ------------------------------------------------------ the two products
//
// Each warp takes 16 slots of every tile, on its own, and the up to 8 NH heads
// of a unit.  Both products run on the tensor cores with the slots or the
// entries on the 16 rows of an instruction and the heads on its 8 columns,
//   S^T [16 slots x 8 heads] += K Q^T,   O^T [16 entries x 8 heads] += V^T P^T,
// so few heads waste little, and which entry (slot) carries which index of a
// sum is free, so that every operand is a plain 16-byte load of a row and the
// loop needs no shared memory.  Lane 4 g + c holds slots g and g + 8 of S^T
// for heads 2 c, 2 c + 1, in
//   s[0], s[1] (slot g), s[2], s[3] (slot g + 8).

// Sixteen bytes of a page, read once: past L1.
__device__ __forceinline__ uint4 ldg_once(const void* p) {
  uint4 u;
  asm("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
      : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
      : "l"(p));
  return u;
}

// bf16 rows, D entries.  K: the lane holds entries 32 y + 8 c .. + 7 of its two
// slots for each block y, the same entries that it holds of head g's q.  V: it
// holds entries 8 g .. + 7 (and 64 + 8 g .. + 7) of slots 2c, 2c + 1, 2c + 8,
// 2c + 9; pairs of slots are packed with byte permutes.  P moves from S^T's
// layout to P^T's by an 8 x 8 transpose and is carried as three bf16 parts, all
// of its fp32.  The instruction cuts its sums off where fp32 additions round, so
// a run of kRun steps' sums at most stands in its accumulators; they are then
// added to the unit's in shared memory, each lane its own.  4 x 131072 slots, 4
// heads a group: 0.06 % of the outputs are not the rounded exact value, with two
// parts and one run 0.32 % (as fast); fresh accumulators for every step the same
// 0.06 %, 312 us where this took 290.  Groups of 12, 16 x 16384 slots, 8 key heads
// of 128: 123 us, 117 with two parts.
template <int D>
struct Bf16 {
  using T = __nv_bfloat16;
  static constexpr int kD = D;
  static constexpr int KB = D / 32, VS = D / 64, MT = D / 16;
  static constexpr int kParts = 3;  // of a weight
  static constexpr int kRun = 16;   // steps that share the instruction's accumulators
  struct Q { uint4 r[KB]; };
  struct K { uint4 r[2][KB]; };
  struct V { uint4 r[4][VS]; };

  // c += A B, A 16 x 16 and B 16 x 8 bf16, fp32 accumulators
  static __device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
  // the transpose of an 8 x 8 matrix of 16-bit entries held two a lane
  static __device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
  }
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *(const uint32_t*)&v;
  }

  static __device__ __forceinline__ void load_q(Q& q, const T* p, bool on, int c) {
#pragma unroll
    for (int y = 0; y < KB; ++y) q.r[y] = on ? *(const uint4*)(p + 32 * y + 8 * c) : make_uint4(0, 0, 0, 0);
  }
  // where the lane's 16 bytes lie: entries from its first of the 16 slots' first
  // row (k_base, v_base), and from there
  static __device__ __forceinline__ int k_base(int g, int c) { return g * D + 8 * c; }
  static constexpr __device__ int k_off(int i, int y) { return 8 * i * D + 32 * y; }
  static __device__ __forceinline__ int v_slot(int i, int c) { return 2 * c + (i & 1) + 8 * (i >> 1); }
  static __device__ __forceinline__ int v_base(int g, int c) { return 2 * c * D + 8 * g; }
  static constexpr __device__ int v_off(int i, int y) { return ((i & 1) + 8 * (i >> 1)) * D + 64 * y; }
  template <int NH>
  static __device__ __forceinline__ void scores(float (&s)[NH][4], const K& k, const Q (&q)[NH]) {
#pragma unroll
    for (int y = 0; y < KB; ++y) {
      const uint4 k0 = k.r[0][y], k1 = k.r[1][y];
#pragma unroll
      for (int x = 0; x < NH; ++x) {
        mma(s[x], k0.x, k1.x, k0.y, k1.y, q[x].r[y].x, q[x].r[y].y);
        mma(s[x], k0.z, k1.z, k0.w, k1.w, q[x].r[y].z, q[x].r[y].w);
      }
    }
  }
  template <int NH>
  static __device__ __forceinline__ void values(float (&o)[NH][MT][4], const V& v, const float (&p)[NH][4], int, int) {
    uint32_t ph[kParts][NH][2];
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float a = p[x][2 * i], b = p[x][2 * i + 1];
#pragma unroll
        for (int z = 0; z < kParts; ++z) {
          const uint32_t w = pack(a, b);
          ph[z][x][i] = transpose8(w);
          a -= __uint_as_float(w << 16), b -= __uint_as_float(w & 0xffff0000u);
        }
      }
#pragma unroll
    for (int y = 0; y < MT; ++y) {
      // rows g and g + 8 of tile y: entries 8g + y and 64 + 8g + y (D = 64: 8g + y and 8g + 4 + y)
      const int yb = D == 128 ? y : y + 4, sb = VS - 1;
      auto pair = [&](int s0, int e, int sg) {
        const uint32_t *r0 = (const uint32_t*)&v.r[s0][sg], *r1 = (const uint32_t*)&v.r[s0 + 1][sg];
        return __byte_perm(r0[e / 2], r1[e / 2], e % 2 ? 0x7632 : 0x5410);
      };
      const uint32_t a0 = pair(0, y, 0), a1 = pair(0, yb, sb), a2 = pair(2, y, 0), a3 = pair(2, yb, sb);
#pragma unroll
      for (int x = 0; x < NH; ++x) {
#pragma unroll
        for (int z = kParts - 1; z >= 0; --z) mma(o[x][y], a0, a1, a2, a3, ph[z][x][0], ph[z][x][1]);
      }
    }
  }
  // the entry of row g (row g + 8) of tile y
  static __device__ __forceinline__ int entry(int y, int g, int upper) {
    return 8 * g + y + (upper ? (D == 128 ? 64 : 4) : 0);
  }
  // entry 8 g + y of each 64 at 8 y + g
  static __device__ __forceinline__ int place(int e) { return (e & 64) + 8 * (e & 7) + ((e >> 3) & 7); }
};

// fp32 rows on the tf32 instructions, each factor as the sum of two (the
// split-precision product of Markidis et al., 2018, with rounded parts):
// x y = x_h y_h + x_h y_l + x_l y_h to about 2^-23.  K: the lane holds entries
// 16 y + 4 c .. + 3 of its slots; V: entries 4 g + 32 y .. + 3 of slots c,
// c + 4, c + 8, c + 12.  P reaches its layout by shuffles.
template <int D, bool QREG>
struct F32 {
  using T = float;
  static constexpr int kD = D;
  static constexpr int KB = D / 16, VS = D / 32, MT = D / 16;
  static constexpr int kRun = 0;  // (values adds outside the instruction)
  struct Q { float4 r[QREG ? KB : 1]; const T* p; };  // QREG: held in r, else read at p for every step (L1)
  struct K { uint4 r[2][KB]; };
  struct V { uint4 r[4][VS]; };

  // x = h + l, both rounded to tf32 (10 bits of significand).  h by an integer
  // addition (the instruction ignores the lower 13 bits); l by a conversion,
  // which keeps a NaN one
  static __device__ __forceinline__ void split(uint32_t x, uint32_t& h, uint32_t& l) {
    h = (x + 0x1000u) & 0xffffe000u;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(l) : "f"(__uint_as_float(x) - __uint_as_float(h)));
  }
  static __device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  }
  // A B in split precision (A split already): the full products into c, the
  // small ones into `small`.  The instruction cuts its sums off where fp32 additions round, so
  // c is a fresh accumulator, added outside, wherever a sum is long.
  struct Parts4 { uint32_t h[4], l[4]; };
  static __device__ __forceinline__ Parts4 split4(uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
    Parts4 p;
    split(a0, p.h[0], p.l[0]), split(a1, p.h[1], p.l[1]), split(a2, p.h[2], p.l[2]), split(a3, p.h[3], p.l[3]);
    return p;
  }
  static __device__ __forceinline__ void mma3(float (&c)[4], float (&small)[4], const Parts4& a, uint32_t b0, uint32_t b1) {
    uint32_t hb[2], lb[2];
    split(b0, hb[0], lb[0]), split(b1, hb[1], lb[1]);
    mma(c, a.h[0], a.h[1], a.h[2], a.h[3], hb[0], hb[1]);
    mma(small, a.l[0], a.l[1], a.l[2], a.l[3], hb[0], hb[1]);
    mma(small, a.h[0], a.h[1], a.h[2], a.h[3], lb[0], lb[1]);
  }

  // (p is a row of q whether `on` or not)
  static __device__ __forceinline__ void load_q(Q& q, const T* p, bool on, int c) {
    q.p = p + 4 * c;
    if (!QREG) return;
#pragma unroll
    for (int y = 0; y < KB; ++y) q.r[y] = on ? *(const float4*)(p + 16 * y + 4 * c) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  static __device__ __forceinline__ float4 q_at(const Q& q, int y) {
    if (QREG) return q.r[y];
    float4 v;  // (not to be held across steps)
    asm volatile("ld.global.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "l"(q.p + 16 * y));
    return v;
  }
  static __device__ __forceinline__ int k_base(int g, int c) { return g * D + 4 * c; }
  static constexpr __device__ int k_off(int i, int y) { return 8 * i * D + 16 * y; }
  static __device__ __forceinline__ int v_slot(int i, int c) { return c + 4 * i; }
  static __device__ __forceinline__ int v_base(int g, int c) { return c * D + 4 * g; }
  static constexpr __device__ int v_off(int i, int y) { return 4 * i * D + 32 * y; }
  template <int NH>
  static __device__ __forceinline__ void scores(float (&s)[NH][4], const K& k, const Q (&q)[NH]) {
    constexpr int kChains = NH == 1 ? 2 : 1;
    float small[kChains][NH][4] = {};
#pragma unroll
    for (int y = 0; y < KB; ++y) {
      const uint4 k0 = k.r[0][y], k1 = k.r[1][y];
      const Parts4 a0 = split4(k0.x, k1.x, k0.y, k1.y), a1 = split4(k0.z, k1.z, k0.w, k1.w);
#pragma unroll
      for (int x = 0; x < NH; ++x) {
        const float4 qy = q_at(q[x], y);
        float c0[4] = {}, c1[4] = {};
        mma3(c0, small[0][x], a0, __float_as_uint(qy.x), __float_as_uint(qy.y));
        mma3(c1, small[kChains - 1][x], a1, __float_as_uint(qy.z), __float_as_uint(qy.w));
#pragma unroll
        for (int i = 0; i < 4; ++i) s[x][i] += c0[i] + c1[i];
      }
    }
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[x][i] += kChains == 2 ? small[0][x][i] + small[kChains - 1][x][i] : small[0][x][i];
  }
  template <int NH>
  static __device__ __forceinline__ void values(float (&o)[NH][MT][4], const V& v, const float (&p)[NH][4], int g,
                                                int c) {
    // slots c, c + 4, c + 8, c + 12 of head g: from the lanes with that slot (and 8 on) and the head's pair
    uint32_t b[NH][4];
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int src = 4 * (c + 4 * i) + g / 2;
        const float e0 = __shfl_sync(0xffffffffu, p[x][0], src), e1 = __shfl_sync(0xffffffffu, p[x][1], src);
        const float e2 = __shfl_sync(0xffffffffu, p[x][2], src), e3 = __shfl_sync(0xffffffffu, p[x][3], src);
        b[x][i] = __float_as_uint(g % 2 ? e1 : e0), b[x][i + 2] = __float_as_uint(g % 2 ? e3 : e2);
      }
#pragma unroll
    for (int y = 0; y < MT; ++y) {
      // rows g and g + 8 of tile y: entry y % 4 of the lane's segments 2 (y / 4) and 2 (y / 4) + 1
      auto at = [&](int slot, int seg) { return ((const uint32_t*)&v.r[slot][2 * (y / 4) + seg])[y % 4]; };
      const Parts4 a = split4(at(0, 0), at(0, 1), at(1, 0), at(1, 1)), a2 = split4(at(2, 0), at(2, 1), at(3, 0), at(3, 1));
#pragma unroll
      for (int x = 0; x < NH; ++x) {
        float full[4] = {}, small[4] = {};
        mma3(full, small, a, b[x][0], b[x][1]);
        mma3(full, small, a2, b[x][2], b[x][3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[x][y][i] += full[i] + small[i];
      }
    }
  }
  static __device__ __forceinline__ int entry(int y, int g, int upper) {
    return 32 * (2 * (y / 4) + upper) + 4 * g + y % 4;
  }
  // entry 4 g + y of each 32 at 8 y + g
  static __device__ __forceinline__ int place(int e) { return (e & ~31) + 8 * (e & 3) + ((e >> 2) & 7); }
};

// how far a score may rise above the running maximum (in powers of two)
// before the sums are rescaled: 2^8 leaves fp32 its full precision
constexpr float kSlack = 8.f;

// The lane's keys and values of the 16 slots from `row` on (-1: none), zero
// behind the sequence (0 x NaN would not be).
template <class X>
__device__ __forceinline__ void load_k(typename X::K& k, const typename X::T* p, int row, int g, int c) {
  const typename X::T* at = p + (long long)row * X::kD + X::k_base(g, c);
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int y = 0; y < X::KB; ++y) k.r[i][y] = row < 0 ? make_uint4(0, 0, 0, 0) : ldg_once(at + X::k_off(i, y));
}
template <class X>
__device__ __forceinline__ void load_v(typename X::V& v, const typename X::T* p, int row, int left, int g, int c) {
  const typename X::T* at = p + (long long)row * X::kD + X::v_base(g, c);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int y = 0; y < X::VS; ++y)
      v.r[i][y] = row < 0 || X::v_slot(i, c) >= left ? make_uint4(0, 0, 0, 0) : ldg_once(at + X::v_off(i, y));
}

// A unit's heads as one warp holds them: queries, and the running maximum, sum
// and weighted values of its slots.
template <class X, int NH>
struct Unit {
  static constexpr int MT = X::MT;
  typename X::Q q[NH];
  // rise: the raw score from which the sums are rescaled
  float o[NH][MT][4], mx[NH][2], sum[NH][2], rise[NH][2];

  __device__ __forceinline__ void start(const typename X::T* q0, long long q_h, int heads, int g, int c) {
#pragma unroll
    for (int x = 0; x < NH; ++x) {
      const bool on = 8 * x + g < heads;
      X::load_q(q[x], q0 + (on ? 8 * x + g : 0) * q_h, on, c);
#pragma unroll
      for (int y = 0; y < MT; ++y)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[x][y][i] = 0.f;
      mx[x][0] = mx[x][1] = kNoMax;
      rise[x][0] = rise[x][1] = -INFINITY;
      sum[x][0] = sum[x][1] = 0.f;
    }
  }

  // The raw scores s of 16 slots become their weights; lo, hi: whether slots g
  // and g + 8 count (all: every slot does).  at: where the slots' scores go
  // (accumulation), slot 0's first head, of `left` slots.  so: where earlier
  // runs' values lie, if there were any.
  template <bool ACC>
  __device__ __forceinline__ void weigh(float (&s)[NH][4], float scale2, bool all, bool lo, bool hi, float* at, int G,
                                        int left, int heads, float* so, bool earlier, int g, int c) {
    if (!all) {
#pragma unroll
      for (int x = 0; x < NH; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[x][i] = (i < 2 ? lo : hi) ? s[x][i] : -INFINITY;
    }
    bool rises = false;
#pragma unroll
    for (int x = 0; x < NH; ++x) {
      if (ACC) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = g + 8 * (i >> 1), h = 8 * x + 2 * c + (i & 1);
          if (j < left && h < heads) at[(long long)j * G + h] = s[x][i];
        }
      }
      rises |= fmaxf(s[x][0], s[x][2]) > rise[x][0] || fmaxf(s[x][1], s[x][3]) > rise[x][1];
    }
    if (__any_sync(0xffffffffu, rises)) {
#pragma unroll
      for (int x = 0; x < NH; ++x)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float m = fmaxf(s[x][i], s[x][i + 2]);
#pragma unroll
          for (int z = 4; z < 32; z <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, z));
          m = fmaxf(m * scale2, mx[x][i]);
          const float f = part_scale(mx[x][i], m);
          mx[x][i] = m;
          if (m > kNoMax) rise[x][i] = (m + kSlack) / scale2;
          sum[x][i] *= f;
#pragma unroll
          for (int y = 0; y < MT; ++y) o[x][y][i] *= f, o[x][y][i + 2] *= f;
          if (X::kRun > 0 && earlier) {
#pragma unroll
            for (int y = 0; y < MT; ++y) so[at_so(x, i, y, 0, g, c)] *= f, so[at_so(x, i, y, 1, g, c)] *= f;
          }
        }
    }
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[x][i] = weight_of(s[x][i], scale2, mx[x][i & 1]);
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
      for (int i = 0; i < 2; ++i) sum[x][i] += s[x][i] + s[x][i + 2];
  }

  // where o[x][y][i] (upper: o[x][y][i + 2]) stands in this warp's so [8 NH][pitch]
  static __device__ __forceinline__ int at_so(int x, int i, int y, int upper, int g, int c) {
    return (8 * x + 2 * c + i) * kPitch<X::kD> + X::place(X::entry(y, g, upper));
  }
  // the values to shared memory, to what earlier runs left there if there were any
  __device__ __forceinline__ void put_values(float* so, bool earlier, int g, int c) {
    if (X::kRun > 0 && earlier) {
#pragma unroll
      for (int x = 0; x < NH; ++x)
#pragma unroll
        for (int y = 0; y < MT; ++y)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[x][y][i] += so[at_so(x, i & 1, y, i >> 1, g, c)];
    }
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
      for (int y = 0; y < MT; ++y)
#pragma unroll
        for (int i = 0; i < 4; ++i) so[at_so(x, i & 1, y, i >> 1, g, c)] = o[x][y][i];
  }
  // A run's values added up (each lane its own entries), for the next run to begin at zero.
  __device__ __forceinline__ void end_run(float* so, bool earlier, int g, int c) {
    put_values(so, earlier, g, c);
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
      for (int y = 0; y < MT; ++y)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[x][y][i] = 0.f;
  }

  // the unit's result to shared memory, so and sml [8 NH][2] of this warp
  __device__ __forceinline__ void put(float* so, float* sml, bool earlier, int g, int c) {
#pragma unroll
    for (int x = 0; x < NH; ++x)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int z = 4; z < 32; z <<= 1) sum[x][i] += __shfl_xor_sync(0xffffffffu, sum[x][i], z);
        const int h = 8 * x + 2 * c + i;
        if (g == 0) sml[h * 2] = mx[x][i], sml[h * 2 + 1] = sum[x][i];
      }
    put_values(so, earlier, g, c);
  }
};

// The weights of a key head's one tile, whose scores and sums the calling threads
// have just written: weight[slot] += sum over the group's heads of p = 2^(score -
// maximum) / sum, thread t of `threads` a slot after the other, as add_weights does for
// longer ones.  175 sequences of up to 38 slots, 16 heads: 22.5 us, 27 with
// these tiles in add_weights too (24.0 with the weights' third part).
__device__ __forceinline__ void add_one_tile(const DecodeArgs& a, int b, int hk, int n, int t, int threads) {
  for (int j = t; j < n; j += threads) {
    const int pg = a.pg.page_of(b, j / a.pg.page);
    if (pg < 0) continue;
    const int row = (int)a.pg.row(pg, hk, j % a.pg.page);
    float* at = a.weight + row;
    const float* x = scores_of(a, b, hk) + scores_row(a, j, row) * a.G;
    const float2* ml = a.ml_ws + (long long)b * a.Hq + hk * a.G;
    float w = 0.f;  // the group's sum, added once: of a heavy slot's weight, each head's part alone may be below half a step
#pragma unroll 4
    for (int g = 0; g < a.G; ++g) w = fmaf(weight_of(x[g], a.scale2, ml[g].x), ml[g].y, w);
    *at += w;
  }
}
// (a group of more heads than a unit's is summed over its units: add_weights)
__device__ __forceinline__ bool one_tile(const DecodeArgs& a, long long tiles) { return tiles == 1 && a.ngroups == 1; }

// A step's K registers are refilled for the next one as soon as the scores are
// done, V's when the values are, so that a warp has some 8 KB on their way all
// the time; page entries are read a step ahead of their rows.
template <class X, int NH, bool ACC, int BLOCKS>
__global__ void __launch_bounds__(kThreads, BLOCKS) decode_kernel(DecodeArgs a) {
  using T = typename X::T;
  constexpr int D = X::kD, GT = 8 * NH;
  begin();
  __shared__ float so[kWarps * GT * kPitch<D>], sml[kWarps * GT * 2];
  const int U = a.pg.Hk * a.ngroups;
  const Run run = my_run(a.pg, U, a.prefix);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, c = lane & 3;
  const T *kp = (const T*)a.k, *vp = (const T*)a.v;
  long long cur = run.s, pre = run.pre;
  int b = run.b0;
  while (cur < run.e) {
    int n = a.pg.length(b);
    const int nt = tiles_of(n);
    if (cur >= (pre + nt) * U) {
      pre += nt;
      ++b;
      continue;
    }
    int t0;
    int u = (int)div_rem(cur - pre * U, nt, &t0);
    const int t1 = (int)min((long long)nt, t0 + (run.e - cur));
    // Units of one tile that follow one another go to a warp each, 16 slots
    // after the other, and need no join of warps (175 sequences of up to 38 slots,
    // 16 heads, with weights: 35 us to 27); else the
    // warps share the unit's tiles, 16 slots of each.
    int units = 0, mb = b;  // such units, and this warp's sequence (n, u: its slots and unit)
    if (nt == 1) {
      long long before = pre;
      int s = b, len = n, tiles = nt, wn = n, wu = u;
      for (; units < kWarps && cur + units < run.e; ++units) {
        while (cur + units >= (before + tiles) * U) {
          before += tiles;
          len = a.pg.length(++s), tiles = tiles_of(len);
        }
        if (tiles != 1) break;
        if (units == warp) mb = s, wn = len, wu = (int)(cur + units - before * U);
      }
      if (units > 1) n = wn, u = wu;
    }
    const bool alone = units > 1;  // a unit a warp
    const int slot0 = alone ? 0 : t0 * kTile + warp * 16, stride = alone ? 16 : kTile;
    const int steps = alone ? (warp < units ? (n + 15) / 16 : 0) : t1 - t0;
    const int hk = u / a.ngroups, g0 = (u % a.ngroups) * GT;
    const int heads = alone && warp >= units ? 0 : min(GT, a.G - g0), h0 = hk * a.G + g0;
    Unit<X, NH> unit;
    unit.start((const T*)a.q + mb * a.q_b + h0 * a.q_h, a.q_h, heads, g, c);
    // row of the first slot of step st, or -1: past the end or without a page
    // (noted, and reported after the loop: a branch here would wait for the
    // entry)
    bool bad = false;
    auto first_row = [&](int st) -> int {
      const int j0 = slot0 + st * stride;
      const bool in = st < steps && j0 < n;
      const int pg = in ? a.pg.page_of(mb, (uint32_t)j0 / (uint32_t)a.pg.page) : -1;
      bad |= in && pg < 0;
      return pg < 0 ? -1 : (int)a.pg.row(pg, hk, (uint32_t)j0 % (uint32_t)a.pg.page);
    };
    typename X::K k;
    typename X::V v;
    int row = first_row(0), next = first_row(1);
    float *mine = so + warp * GT * kPitch<D>, *mine_ml = sml + warp * GT * 2;
    bool earlier = false;  // runs that have ended
    float* const scores = ACC ? scores_of(a, mb, hk) + g0 : nullptr;
    load_k<X>(k, kp, row, g, c);
    load_v<X>(v, vp, row, n - slot0, g, c);
    for (int st = 0; st < steps; ++st) {
      const int j0 = slot0 + st * stride, after = first_row(st + 2);
      float s[NH][4] = {};
      X::scores(s, k, unit.q);
      load_k<X>(k, kp, next, g, c);
      float* at = ACC ? scores + scores_row(a, j0, row) * a.G : nullptr;
      unit.template weigh<ACC>(s, a.scale2, row >= 0 && j0 + 16 <= n, row >= 0 && j0 + g < n, row >= 0 && j0 + g + 8 < n,
                               at, a.G, row >= 0 ? n - j0 : 0, heads, mine, earlier, g, c);
      X::values(unit.o, v, s, g, c);
      load_v<X>(v, vp, next, n - j0 - stride, g, c);
      row = next;
      next = after;
      if (X::kRun > 0 && (st + 1) % max(X::kRun, 1) == 0) unit.end_run(mine, earlier, g, c), earlier = true;
    }
    if (bad && lane == 0) *a.pg.err = 1;
    unit.put(mine, mine_ml, earlier, g, c);
    if (alone) {
      __syncwarp();
      finish_unit<X, GT, 1>(a, mine, mine_ml, mb, h0, heads, -1, lane);
      __syncwarp();
      if (ACC && warp < units && one_tile(a, 1)) add_one_tile(a, mb, hk, n, lane, 32);
      cur += units;
      continue;
    }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == nt;
    finish_unit<X, GT, kWarps>(a, so, sml, b, h0, heads, whole ? -1 : 2LL * blockIdx.x + (cur == run.s ? 0 : 1),
                               threadIdx.x);
    __syncthreads();
    if (ACC && one_tile(a, nt)) add_one_tile(a, b, hk, n, threadIdx.x, kThreads);
    cur += t1 - t0;
  }
}

// The CTA whose run holds tile x of the line (the run of CTA i of n is
// [i T / n, (i + 1) T / n)).
__device__ __forceinline__ int cta_of(long long x, long long T, int n) {
  const long long y = (x + 1) * n - 1;
  return (y | T) >> 32 ? (int)(y / T) : (int)((uint32_t)y / (uint32_t)T);
}

// The partials of a unit that lies in more than one run: CTAs c0 .. c1, the
// first one's slot; `one`: its only CTA has written the result itself.
struct Parts {
  int c0, c1;
  long long first;
  bool one;
  __device__ __forceinline__ long long slot(int c) const { return c == c0 ? first : 2LL * c; }
};
__device__ __forceinline__ Parts parts_of(long long pre, long long nt, long long total, int u, int U, int n) {
  const long long x0 = pre * U + u * nt, T = total * U;
  Parts p;
  p.c0 = cta_of(x0, T, n);
  p.c1 = cta_of(x0 + nt - 1, T, n);
  p.one = p.c0 == p.c1;
  // a CTA whose run begins in the unit (or before it with the unit as its first) used slot 0
  p.first = 2LL * p.c0 + (mul_div(T, p.c0, n) == x0 ? 0 : 1);
  return p;
}
// One warp: maximum and sum of head g's partials, the lanes side by side.
__device__ __forceinline__ void join_sums(const DecodeArgs& a, const Parts& p, int g, float& M, float& l) {
  const int lane = threadIdx.x & 31;
  M = kNoMax, l = 0.f;
  for (int c = p.c0 + lane; c <= p.c1; c += 32) {
    const float2 ml = *(const float2*)(a.part_ml + 2 * (p.slot(c) * a.GT + g));
    const float m = fmaxf(M, ml.x);
    l = l * part_scale(M, m) + ml.y * part_scale(ml.x, m);
    M = m;
  }
  const float m = warp_max(M);
  l = warp_sum(l * part_scale(M, m));
  M = m;
}

// Row i = (sequence, query head): joins the unit's partials, or writes the row
// of an empty sequence.  W warps share the partials: one where there are rows
// enough, the whole CTA for few.
template <typename T, int D, int W>
__device__ __forceinline__ void join_row(const DecodeArgs& a, long long i) {
  constexpr int E = D / 32;
  __shared__ float red[W > 1 ? W * D : 1];
  const int lane = threadIdx.x & 31, w = W > 1 ? threadIdx.x >> 5 : 0;
  const int b = (int)(i / a.Hq), h = (int)(i % a.Hq);
  const int hk = h / a.G, g = (h % a.G) % a.GT, u = hk * a.ngroups + (h % a.G) / a.GT;
  const long long pre = a.prefix[b], nt = a.prefix[b + 1] - pre;
  float o[E], M = kNoMax, l = 0.f;
#pragma unroll
  for (int x = 0; x < E; ++x) o[x] = 0.f;
  if (nt > 0) {
    const Parts p = parts_of(pre, nt, a.prefix[a.pg.B], u, a.pg.Hk * a.ngroups, (int)a.prefix[a.pg.B + 1]);
    if (p.one) return;  // (every warp of the row)
    join_sums(a, p, g, M, l);
#pragma unroll 8
    for (int c = p.c0 + w; c <= p.c1; c += W) {
      const long long s = p.slot(c) * a.GT + g;
      const float f = part_scale(a.part_ml[2 * s], M);
      const float* at = a.part_o + s * D + lane * E;
      if (E == 4) {
        const float4 v = *(const float4*)at;
        o[0] += f * v.x, o[1] += f * v.y, o[2] += f * v.z, o[3] += f * v.w;
      } else {
        const float2 v = *(const float2*)at;
        o[0] += f * v.x, o[1] += f * v.y;
      }
    }
    if (W > 1) {
#pragma unroll
      for (int x = 0; x < E; ++x) red[w * D + lane * E + x] = o[x];
      __syncthreads();
      if (w > 0) return;
#pragma unroll
      for (int r = 1; r < W; ++r)
#pragma unroll
        for (int x = 0; x < E; ++x) o[x] += red[r * D + lane * E + x];
    }
  }
  if (w > 0) return;
#pragma unroll
  for (int x = 0; x < E; ++x) ((T*)a.out)[i * D + lane * E + x] = from_f32<T>(l == 0.f ? 0.f : o[x] / l);
  if (a.lse && lane == 0) a.lse[i] = lse_of(M, l);
}

// Part `idx` of `count` of the tile line: weight[slot] += sum over the group's
// heads of p = 2^(score - maximum) / sum, these two from the partials again (so
// this need not wait for the joined rows).  A thread a slot: nothing is summed in an order
// that varies.
__device__ __forceinline__ void add_weights(const DecodeArgs& a, int idx, int count) {
  extern __shared__ float2 ml_of[];  // [G] maximum and 1 / sum
  __shared__ int found;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, Hk = a.pg.Hk, G = a.G;
  const long long total = a.prefix[a.pg.B], T = total * Hk;
  const int ctas = (int)a.prefix[a.pg.B + 1];  // of the decode kernel
  const int used = ctas_used(T, count);
  if (idx >= used) return;
  const long long s = mul_div(T, idx, used), e = mul_div(T, idx + 1, used);
  for (int b = tid; b < a.pg.B; b += kThreads)
    if (a.prefix[b] * Hk <= s && s < a.prefix[b + 1] * Hk) found = b;
  __syncthreads();
  int b = found;
  for (long long cur = s; cur < e;) {
    const long long pre = a.prefix[b], nt = a.prefix[b + 1] - pre;
    if (cur >= (pre + nt) * Hk) {
      ++b;
      continue;
    }
    if (one_tile(a, nt)) {  // added by the decode kernel
      cur = min(e, (pre + 1) * Hk);
      continue;
    }
    const long long local = cur - pre * Hk;
    int t0;
    const int hk = (int)div_rem(local, (int)nt, &t0), t1 = (int)min(nt, t0 + (e - cur));
    const int end = min(a.pg.length(b), t1 * kTile);
    constexpr int kSlots = 4;  // a thread's slots in flight; their pages are read an iteration ahead
    int j = t0 * kTile + tid, pg[kSlots];
    auto pages = [&](int j) {
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        const int ji = j + i * kThreads;
        pg[i] = ji < end ? a.pg.page_of(b, ji / a.pg.page) : -1;
      }
    };
    pages(j);
    // a unit's heads by a thread each where its parts are few, else by a warp each
    const Parts p0 = parts_of(pre, nt, total, hk * a.ngroups, Hk * a.ngroups, ctas);
    const bool few = p0.c1 - p0.c0 < 16;
    for (int g = few ? tid : warp; g < G; g += few ? kThreads : kWarps) {
      const Parts p = g < a.GT ? p0 : parts_of(pre, nt, total, hk * a.ngroups + g / a.GT, Hk * a.ngroups, ctas);
      float M = kNoMax, l = 0.f;
      if (p.one) {
        ml_of[g] = a.ml_ws[(long long)b * a.Hq + hk * G + g];
      } else if (few) {
#pragma unroll 4
        for (int c = p.c0; c <= p.c1; ++c) {
          const float2 ml = *(const float2*)(a.part_ml + 2 * (p.slot(c) * a.GT + g % a.GT));
          const float m = fmaxf(M, ml.x);
          l = l * part_scale(M, m) + ml.y * part_scale(ml.x, m);
          M = m;
        }
        ml_of[g] = make_float2(M, l == 0.f ? 0.f : 1.f / l);
      } else {
        join_sums(a, p, g % a.GT, M, l);
        if (lane == 0) ml_of[g] = make_float2(M, l == 0.f ? 0.f : 1.f / l);
      }
    }
    __syncthreads();
    const float* const scores = scores_of(a, b, hk);
    for (; j < end; j += kSlots * kThreads) {
      float w[kSlots], was[kSlots];  // the group's sum, added once to the stored weight
      const float* x[kSlots];
      float* at[kSlots];
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        const int ji = j + i * kThreads;
        const int row = (int)a.pg.row(max(pg[i], 0), hk, ji % a.pg.page);
        at[i] = pg[i] < 0 ? nullptr : a.weight + row;
        was[i] = at[i] ? *at[i] : 0.f;
        w[i] = 0.f;
        x[i] = scores + scores_row(a, min(ji, end - 1), row) * G;  // (without a page: any that can be read)
      }
      pages(j + kSlots * kThreads);
      auto add = [&](int i, float v, float2 ml) { w[i] = fmaf(weight_of(v, a.scale2, ml.x), ml.y, w[i]); };
      if (G % 4 == 0) {
#pragma unroll 1
        for (int g = 0; g < G; g += 4) {
          float4 v[kSlots];
#pragma unroll
          for (int i = 0; i < kSlots; ++i) v[i] = __ldg((const float4*)(x[i] + g));
#pragma unroll
          for (int i = 0; i < kSlots; ++i)
            add(i, v[i].x, ml_of[g]), add(i, v[i].y, ml_of[g + 1]), add(i, v[i].z, ml_of[g + 2]), add(i, v[i].w, ml_of[g + 3]);
        }
      } else {
#pragma unroll 2
        for (int g = 0; g < G; ++g) {
          float v[kSlots];
#pragma unroll
          for (int i = 0; i < kSlots; ++i) v[i] = __ldg(x[i] + g);
#pragma unroll
          for (int i = 0; i < kSlots; ++i) add(i, v[i], ml_of[g]);
        }
      }
#pragma unroll
      for (int i = 0; i < kSlots; ++i)
        if (at[i]) *at[i] = was[i] + w[i];
    }
    __syncthreads();
    cur += t1 - t0;
  }
}

// The first CTAs join; the others (accumulation) add the weights of units of
// more than one tile.  Eight CTAs an SM, all of a launch's: 4 x 131072 slots 290
// us, 296 with seven.
template <typename T, int D, int W>
__global__ void __launch_bounds__(kThreads, 8) decode_finish_kernel(DecodeArgs a, int join_ctas) {
  begin();
  if ((int)blockIdx.x < join_ctas) {
    const long long i = W > 1 ? blockIdx.x : (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
    if (i < (long long)a.pg.B * a.Hq) join_row<T, D, W>(a, i);
  } else {
    add_weights(a, blockIdx.x - join_ctas, gridDim.x - join_ctas);
  }
}

constexpr size_t kAlign = 256;
size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

// The scores that a call which accumulates keeps: of every slot of the table, or,
// since no page is in the table twice then, of the pool, where the table (as long
// as the longest allowed context) has more than twice the pool's slots.  32
// sequences of 32 heads with tables of 131,072 slots over 4096 pages of 64: 34 MB,
// 537 by the table.  The two take the same time (4 x 131072 slots 289 us each, 64
// x 2000 51).
double scores_by_table(const nats_paged_cache* c, int Hq) { return (double)c->B * Hq * c->max_pages * c->page; }
double scores_by_pool(const nats_paged_cache* c, int Hq) { return (double)c->n_pages * c->page * Hq; }
bool pooled(const nats_paged_cache* c, int Hq) { return scores_by_table(c, Hq) > 2 * scores_by_pool(c, Hq); }

size_t layout(const nats_paged_cache* c, int Hq, bool accumulate, char* base, DecodeArgs* a) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    char* p = base ? base + off : nullptr;
    off += align_up(bytes);
    return p;
  };
  DecodeArgs d = {};
  d.prefix = (long long*)take(8 * ((size_t)c->B + 2));
  d.ml_ws = (float2*)take(8 * (size_t)c->B * Hq);
  d.part_ml = (float*)take(4 * 2 * (size_t)kMaxCtas * kMaxHeads * 2);
  d.part_o = (float*)take(4 * 2 * (size_t)kMaxCtas * kMaxHeads * c->d);
  d.pooled = pooled(c, Hq);
  const size_t scores = (size_t)(d.pooled ? scores_by_pool(c, Hq) : scores_by_table(c, Hq));
  d.scores = accumulate ? (float*)take(4 * scores) : nullptr;
  if (a) *a = d;
  return off;
}

nats_status check_decode(const nats_paged_cache* c, int32_t Hq, int32_t accumulate) {
  const nats_status s = check_cache(c);
  if (s != NATS_OK) return s;
  if (Hq < 0 || Hq % c->Hk != 0) return NATS_ERR_SHAPE;
  // a group's maxima and sums fit shared memory
  if (Hq / c->Hk > 4096) return NATS_ERR_UNSUPPORTED;
  // rows of a pool and of the batch's queries are 32-bit
  if ((long long)c->B * Hq > (1LL << 31) - 1 || (double)c->n_pages * c->Hk * c->page > 2147483647.0)
    return NATS_ERR_UNSUPPORTED;
  if (accumulate && std::fmin(scores_by_table(c, Hq), scores_by_pool(c, Hq)) > 1099511627776.0) return NATS_ERR_UNSUPPORTED;
  return NATS_OK;
}

// BLOCKS: the CTAs an SM has registers for.
template <class X, int NH, int BLOCKS>
cudaError_t launch(DecodeArgs& a, cudaStream_t st) {
  using T = typename X::T;
  constexpr int D = X::kD;
  a.GT = 8 * NH;
  a.ngroups = (a.G + a.GT - 1) / a.GT;
  const bool acc = a.scores != nullptr;
  const int ctas = kSMs * BLOCKS;
  const cudaError_t e = acc ? after(decode_kernel<X, NH, true, BLOCKS>, ctas, kThreads, 0, st, 0, a)
                            : after(decode_kernel<X, NH, false, BLOCKS>, ctas, kThreads, 0, st, 0, a);
  if (e != cudaSuccess) return e;
  // a CTA a row while the rows are no more than two waves of CTAs, so that a
  // long unit's many partials (up to one a CTA) are read by four warps
  const long long rows = (long long)a.pg.B * a.Hq;
  const bool few = rows <= kSMs * 16;
  const int join = (int)(few ? rows : (rows + kWarps - 1) / kWarps);
  const unsigned grid = join + (acc ? kSMs * 8 : 0);
  const size_t smem = acc ? sizeof(float2) * (size_t)a.G : 0;
  return few ? after(decode_finish_kernel<T, D, kWarps>, grid, kThreads, smem, st, 0, a, join)
             : after(decode_finish_kernel<T, D, 1>, grid, kThreads, smem, st, 0, a, join);
}

// Units of eight heads; groups of more than eight in units of sixteen, whose
// rows are then read, and in fp32 split, once.  bf16, 16 x 16384 slots, 12 heads
// a group: 123 us (78 % of the copy rate, with two warps a scheduler); their
// heads dealt to several warps 161 us where this took 145.  fp32, 8 x 16384, 12
// heads a group: d 64 94 us (60 %), 123 in units of eight; d 128 206 us (56 %),
// 239; but only where there are some four tiles a CTA, since units of eight are
// twice as many to share out (14 x 86 slots, 4 key heads, d 128: 14.8 us, 12.6 in
// units of eight).  Lengths are on the device, so the table's capacity stands for
// them here: short sequences in long tables get units of sixteen.  Groups of more
// than sixteen read their rows once a unit (one key head, 1 x 131072 slots, d 128,
// bf16: 16 heads 41 us, 64 52, 128 83).  fp32 queries of 128 are read again for every step (F32's
// QREG; 8 x 16384, 4 heads a group: 134 us, 138 held in registers, some of them
// spilled), those of 64 held (70.5 against 71.6).
cudaError_t launch(DecodeArgs& a, int dtype, int d, cudaStream_t st) {
  if (dtype != NATS_BF16) {
    const long long tiles = (long long)a.pg.B * a.pg.Hk * ((a.pg.cap() + kTile - 1) / kTile);
    if (a.G > 8 && tiles >= 8 * kSMs)
      return d == 128 ? launch<F32<128, false>, 2, 2>(a, st) : launch<F32<64, true>, 2, 2>(a, st);
    return d == 128 ? launch<F32<128, false>, 1, 2>(a, st) : launch<F32<64, true>, 1, 3>(a, st);
  }
  if (a.G > 8) return d == 128 ? launch<Bf16<128>, 2, 2>(a, st) : launch<Bf16<64>, 2, 3>(a, st);
  return d == 128 ? launch<Bf16<128>, 1, 3>(a, st) : launch<Bf16<64>, 1, 4>(a, st);
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
  // (a stride that leads from nothing to nothing may be anything)
  if (cache->B == 1) q_stride_b = 0;
  if (Hq == 1) q_stride_h = 0;
  if (((uintptr_t)q | (uintptr_t)out | (uintptr_t)workspace) & 15u) return NATS_ERR_ALIGN;
  if ((q_stride_b * es) % 16 != 0 || (q_stride_h * es) % 16 != 0 || ((uintptr_t)lse & 3u)) return NATS_ERR_ALIGN;
  DecodeArgs a;
  if (workspace_bytes < layout(cache, Hq, accumulate != 0, (char*)workspace, &a)) return NATS_ERR_WORKSPACE;
  a.pg = view_of(cache);
  if (cache->n_pages == 0) a.pg.max_pages = 0;  // no slot can have a page
  a.k = cache->k_pages, a.v = cache->v_pages, a.weight = cache->weight;
  a.q = q, a.q_b = q_stride_b, a.q_h = q_stride_h, a.out = out, a.lse = lse;
  a.Hq = Hq, a.G = Hq / cache->Hk;
  a.scale2 = (scale > 0.f ? scale : 1.0f / std::sqrt((float)cache->d)) * kLog2e;
  cudaStream_t st = (cudaStream_t)stream;
  const cudaError_t e = launch(a, cache->dtype, cache->d, st);
  return (nats_status)record_cuda_error(e);
}

}  // extern "C"
