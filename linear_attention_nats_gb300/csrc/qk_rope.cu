// qk_rope.cu - RMSNorm of each head's query and key row with the rotary
// position rotation in the same pass (nats_qk_norm_rope), its gradient
// (nats_qk_norm_rope_bwd), and the same pass with the key and value rows
// going to the pages of a cache (nats_paged_append).
//
//   n = sqrt(mean(x^2) + eps),  z = w x / n,  y = R(p) z
//   u = R(p)^T dy,  dw = sum u x / n,  dx = (w u - x <w u, x> / (d n^2)) / n
//
// Bound by HBM: a row is read once and written once, its d entries held in
// the registers of d / 8 lanes (8 entries a lane), statistics and rotation in
// fp32.  A lane's entries are two quads chosen so that both members of each
// pair are its own and the rotation needs no exchange: quads l and l + rot/8
// for pairs (i, i + rot/2), quads 2l and 2l + 1 for pairs (2i, 2i + 1); in
// both, the lane's four pairs are 4l .. 4l + 3.  A warp keeps one token's
// cosines and sines and walks over the heads with them; where tokens are many
// and their rows few, each group of d / 8 lanes does so with a token of its own.
//
// Angles.  p f in fp32 is off by 2^-24 of the angle, whole radians at far
// positions, and fp64 is slow on this chip.  The frequency becomes a 64-bit
// fixed-point fraction of a turn, F = frac(f / 2 pi) 2^64, and the phase is
// p F mod 2^64, exact whole turns dropping out of the product by themselves;
// its upper 32 bits go to sincospif, rounded to fp32 (up to 1e-7 rad).
//
// Measured on one GB300 (4 x 8192 tokens, 16 query and 16 key heads of 128,
// bf16; HBM copy rate 6.8 TB/s): forward 88 us, 6.1 TB/s; gradient from fp32 to
// bf16 176 us, 6.1 TB/s; one token 2.8 us (position, angle and row are one
// chain of loads).  8 ragged prompts of up to 4096 tokens into a cache, 32 + 8
// + 8 heads: 99 us, 5.8 TB/s.
#include <cmath>
#include <type_traits>

#include "kernels.h"
#include "launch.cuh"
#include "paged.cuh"

namespace nats {
namespace {

constexpr int kWarps = 8;  // warps per CTA

// f / (2 pi) in turns times 2^64, modulo 2^64, from the bits of the double f:
// the 53-bit mantissa times 2^64 / (2 pi) rounded to an integer (62 bits),
// shifted by the exponent.  Integer work only.  2^64 / (2 pi) =
// 2935890503282001226.3...  An infinity or NaN has no turns: see turned_by.
__device__ __forceinline__ uint64_t turns_fixed(double f) {
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int e = (int)(bits >> 52) & 0x7ff;
  if (e == 0 || e == 0x7ff) return 0;  // below 2^-1022: no turn at any position
  const uint64_t m = (bits & 0xfffffffffffffull) | (1ull << 52);
  constexpr uint64_t kInv2Pi = 2935890503282001226ull;
  const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  const int s = 1075 - e;  // f = m 2^-s
  uint64_t r;
  if (s <= 0)
    r = -s >= 64 ? 0 : lo << -s;
  else if (s < 64)
    r = (lo >> s) | (hi << (64 - s));
  else
    r = s >= 128 ? 0 : hi >> (s - 64);
  return (bits >> 63) ? 0 - r : r;
}

// Whether f is an infinity or NaN.
__device__ __forceinline__ bool endless(double f) {
  return (((uint64_t)__double_as_longlong(f) >> 52) & 0x7ff) == 0x7ff;
}
// cos and sin of position p's turns of the frequency F; NaN, as the formula's,
// for one that is not finite (bad)
__device__ __forceinline__ void turned_by(uint64_t F, long long p, bool bad, float* c, float* s) {
  sincospif((float)(int32_t)((uint64_t)p * F >> 32) * 0x1p-31f, s, c);
  if (bad) *s = *c = __int_as_float(0x7fffffff);
}

struct Operand {
  const void* p;
  long long b, h, t;
};

// Four entries of a row as they are stored, and their conversions.
template <typename T, bool VEC>
struct Quad;
template <>
struct Quad<__nv_bfloat16, true> {
  uint2 u;
  __device__ __forceinline__ void zero() { u = make_uint2(0, 0); }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = __ldcs((const uint2*)p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *(uint2*)p = u; }
  __device__ __forceinline__ void get(float* o) const {
    o[0] = __uint_as_float(u.x << 16), o[1] = __uint_as_float(u.x & 0xffff0000u);
    o[2] = __uint_as_float(u.y << 16), o[3] = __uint_as_float(u.y & 0xffff0000u);
  }
  __device__ __forceinline__ void set(const float* o) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(o[0], o[1]), b = __floats2bfloat162_rn(o[2], o[3]);
    u.x = *(const uint32_t*)&a, u.y = *(const uint32_t*)&b;
  }
};
template <>
struct Quad<float, true> {
  float4 u;
  __device__ __forceinline__ void zero() { u = make_float4(0.f, 0.f, 0.f, 0.f); }
  __device__ __forceinline__ void load(const float* p) { u = __ldcs((const float4*)p); }
  __device__ __forceinline__ void store(float* p) const { *(float4*)p = u; }
  __device__ __forceinline__ void get(float* o) const { o[0] = u.x, o[1] = u.y, o[2] = u.z, o[3] = u.w; }
  __device__ __forceinline__ void set(const float* o) { u = make_float4(o[0], o[1], o[2], o[3]); }
};
template <typename T>
struct Quad<T, false> {
  T u[4];
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = from_f32<T>(0.f);
  }
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = p[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = u[i];
  }
  __device__ __forceinline__ void get(float* o) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = to_f32(u[i]);
  }
  __device__ __forceinline__ void set(const float* o) {
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = from_f32<T>(o[i]);
  }
};

// What a lane knows of its row: its two quads and its four pairs' turns.
struct LaneMap {
  int qa, qb;   // entry offsets of the two quads
  bool turned;  // whether the lane's entries are rotated at all
  int pair0;    // its first pair
};
template <bool INTER>
__device__ __forceinline__ LaneMap lane_map(int l, int rot) {
  LaneMap m;
  m.turned = 8 * l < rot;
  m.pair0 = 4 * l;
  if (INTER || !m.turned) {
    m.qa = 8 * l;  // the rows' entries from rot on lie in pairs of quads, as the lanes from rot / 8 on do
    m.qb = 8 * l + 4;
  } else {
    m.qa = 4 * l;
    m.qb = 4 * l + rot / 2;
  }
  return m;
}

// cos and sin of the lane's four pairs at position p (1 and 0 where nothing
// turns).  The 32 / LPR rows of a warp have the same pairs, so each of them
// works out its share of the four (F: that share's frequencies, bad: a bit for
// each that is not finite) and the lanes exchange them.
template <int LPR>
__device__ __forceinline__ void angles(const uint64_t* F, unsigned bad, bool turned, long long p, int l, float* c,
                                       float* s) {
  constexpr int N = 4 / (32 / LPR);
  float cm[N], sm[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    cm[i] = 1.f, sm[i] = 0.f;
    if (turned) turned_by(F[i], p, bad >> i & 1, &cm[i], &sm[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    c[i] = __shfl_sync(0xffffffffu, cm[i % N], LPR * (i / N) + l);
    s[i] = __shfl_sync(0xffffffffu, sm[i % N], LPR * (i / N) + l);
  }
}
// How a warp's 32 / LPR groups of lanes share the work: rows of one token side
// by side (angles above), or, where a token has few rows, a token each.
template <int LPR, bool EACH>
struct Share {
  static constexpr int kTokens = EACH ? 32 / LPR : 1;  // of a warp
  static constexpr int kRows = 32 / LPR / kTokens;     // of a token, side by side
  static constexpr int kPairs = EACH ? 4 : LPR / 8;    // of the lane's four, whose frequencies it holds
  uint64_t F[kPairs];
  unsigned bad = 0;
  __device__ __forceinline__ Share(const double* inv_freq, const LaneMap& m, int sub) {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const double f = m.turned ? inv_freq[m.pair0 + (EACH ? 0 : sub * kPairs) + i] : 0.0;
      F[i] = turns_fixed(f);
      bad |= (unsigned)endless(f) << i;
    }
  }
  __device__ __forceinline__ void at(bool turned, long long p, int l, float* c, float* s) const {
    if constexpr (EACH) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = 1.f, s[i] = 0.f;
        if (turned) turned_by(F[i], p, bad >> i & 1, &c[i], &s[i]);
      }
    } else {
      angles<LPR>(F, bad, turned, p, l, c, s);
    }
  }
};

// x[0..3] the lane's first quad, x[4..7] its second
template <bool INTER>
__device__ __forceinline__ void turn(float* x, const float* c, const float* s) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int a = INTER ? 2 * i : i, b = INTER ? 2 * i + 1 : i + 4;
    const float xa = x[a], xb = x[b];
    x[a] = xa * c[i] - xb * s[i];
    x[b] = xb * c[i] + xa * s[i];
  }
}

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

struct RopeArgs {
  Operand q, k, v;     // v: append only
  Operand qo, ko;      // outputs (ko: not for append)
  const float *wq, *wk;
  const double* inv_freq;
  const int64_t* pos;
  long long pos_b, pos0;
  int B, L, Hq, Hk, rot;
  int norm;
  float eps;
  int rows_per_item, items_per_token;  // a warp's share of a token's rows
  // append
  PagedView pg;
  void *k_pages, *v_pages;
  float* weight;
  const int32_t *start, *n_new;
};

// The lane's eight weights (ones without).
__device__ __forceinline__ void lane_weights(const float* w, const LaneMap& m, float* o) {
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = w ? w[(i < 4 ? m.qa : m.qb - 4) + i] : 1.f;
}

// Rows h0 .. h1 - 1 at src to L2, each of LANES lanes a 128-byte line: the whole
// item's reads are under way while its angles are still being formed.
template <typename T, int D, int LANES>
__device__ __forceinline__ void prefetch_rows(const T* src, long long stride_h, int h0, int h1, int lane) {
  constexpr int kLines = D * (int)sizeof(T) / 128;
  for (int i = lane; i < (h1 - h0) * kLines; i += LANES) {
    const T* p = src + (h0 + i / kLines) * stride_h + (i % kLines) * (128 / (int)sizeof(T));
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
  }
}

constexpr int kRowsAhead = 4;  // row loads a lane has in flight

// Rows h0 .. h1 - 1 of one token and one kind (query, key, or a value to
// copy), their first row at src, RPW of them side by side (this lane's from
// row `sub` on): kRowsAhead rows of every D / 8 lanes are requested together.  row_at(h) is the destination of row h, or NULL to
// leave it.  With the weights taken into the token's cosines and sines, a pair
// costs four products and the row's 1 / n two:
//   y_a = (x_a w_a c - x_b w_b s) / n,  y_b = (x_b w_b c + x_a w_a s) / n.
template <typename T, int D, int RPW, bool INTER, bool VEC, bool COPY, class RowAt>
__device__ __forceinline__ void fwd_rows(const T* src, long long stride_h, int h0, int h1, const float* w, bool norm,
                                         float eps, const LaneMap& m, const float* c, const float* s, int sub,
                                         RowAt row_at) {
  float ca[4], sa[4], cb[4], sb[4];
  if (!COPY) {
    float wl[8];
    lane_weights(w, m, wl);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float wa = wl[INTER ? 2 * i : i], wb = wl[INTER ? 2 * i + 1 : i + 4];
      ca[i] = wa * c[i], sa[i] = wa * s[i], cb[i] = wb * c[i], sb[i] = wb * s[i];
    }
  }
  const long long step = RPW * stride_h;
  const T *pa = src + (h0 + sub) * stride_h + m.qa, *pb = pa + (m.qb - m.qa);
  auto rows = [&](int h, auto full) {
    Quad<T, VEC> qa[kRowsAhead], qb[kRowsAhead];
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i) {
      if (full || h + i * RPW < h1) {
        qa[i].load(pa);
        qb[i].load(pb);
      } else {
        qa[i].zero(), qb[i].zero();
      }
      pa += step, pb += step;
    }
#pragma unroll
    for (int i = 0; i < kRowsAhead; ++i) {
      const int r = h + i * RPW;
      if (!full && r - sub >= h1) break;  // (none of the warp's rows)
      if (!COPY) {
        float x[8];
        qa[i].get(x), qb[i].get(x + 4);
        float rn = 1.f;
        if (norm) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss = fmaf(x[e], x[e], ss);
          rn = rsqrtf(fmaf(row_sum<D / 8>(ss), 1.f / D, eps));
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int ia = INTER ? 2 * e : e, ib = INTER ? 2 * e + 1 : e + 4;
          const float xa = x[ia], xb = x[ib];
          x[ia] = rn * fmaf(xa, ca[e], -(xb * sb[e]));
          x[ib] = rn * fmaf(xb, cb[e], xa * sa[e]);
        }
        qa[i].set(x), qb[i].set(x + 4);
      }
      if (!full && r >= h1) continue;
      T* dst = row_at(r);
      if (!dst) continue;
      qa[i].store(dst + m.qa);
      qb[i].store(dst + m.qb);
    }
  };
  int h = h0;
  for (; h + kRowsAhead * RPW <= h1; h += kRowsAhead * RPW) rows(h + sub, std::true_type{});
  if (h < h1) rows(h + sub, std::false_type{});
}

// One warp per item (a token and a run of its rows; EACH: as many tokens as it
// has groups of lanes): q rows, then k rows, then (append) v rows.  Three CTAs an SM, four rows of a lane requested
// together and the item's rows prefetched: 1.7 times the rate of one row at a
// time (151 us for the 4 x 8192 tokens above).
template <typename T, int D, bool INTER, bool PAGED, bool VEC, bool EACH>
__global__ void __launch_bounds__(kWarps * 32, 3) rope_fwd_kernel(RopeArgs a) {
  constexpr int LPR = D / 8;
  begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  using Sh = Share<LPR, EACH>;
  const int l = lane % LPR, group = lane / LPR, sub = EACH ? 0 : group, pl = EACH ? l : lane;
  const long long tokens = (long long)a.B * a.L;
  const long long item = ((long long)blockIdx.x * kWarps + warp) * Sh::kTokens + (EACH ? group : 0);
  long long tok = item / a.items_per_token;
  if (EACH ? item - group >= tokens : tok >= tokens) return;
  bool live = tok < tokens;  // (EACH: the last token again without writing, where a group has none)
  tok = min(tok, tokens - 1);
  const int b = (int)(tok / a.L), t = (int)(tok % a.L);
  const int rows = a.Hq + a.Hk + (PAGED ? a.Hk : 0);
  const int r0 = EACH ? 0 : (int)(item % a.items_per_token) * a.rows_per_item;
  const int r1 = EACH ? rows : min(rows, r0 + a.rows_per_item);
  if (PAGED && a.n_new) {
    live = live && t < a.n_new[b];
    if (!__any_sync(0xffffffffu, live)) return;
  }
  const int k0 = max(r0 - a.Hq, 0), k1 = min(r1 - a.Hq, a.Hk);
  const T *qs = (const T*)a.q.p + b * a.q.b + t * a.q.t, *ks = (const T*)a.k.p + b * a.k.b + t * a.k.t;
  constexpr int kLanes = EACH ? LPR : 32;
  prefetch_rows<T, D, kLanes>(qs, a.q.h, r0, min(r1, a.Hq), pl);
  prefetch_rows<T, D, kLanes>(ks, a.k.h, k0, k1, pl);
  const int v0 = max(r0 - a.Hq - a.Hk, 0), v1 = PAGED ? min(r1 - a.Hq - a.Hk, a.Hk) : 0;
  const T* vs = PAGED ? (const T*)a.v.p + b * a.v.b + t * a.v.t : nullptr;
  if (PAGED) prefetch_rows<T, D, kLanes>(vs, a.v.h, v0, v1, pl);
  long long p = a.pos0 + t;
  int pg = -1, slot = 0;
  if (PAGED) {
    const long long at = (long long)(a.start ? a.start[b] : a.pg.lens[b]) + t;
    p = at;
    if (at >= 0 && at < a.pg.cap()) {
      pg = a.pg.page_of(b, (int)at / a.pg.page);
      slot = (int)at % a.pg.page;
    }
    if (pg < 0 && live && pl == 0 && r0 == 0) *a.pg.err = 1;
    if (!live) pg = -1;
  }
  if (a.pos) p = a.pos[b * a.pos_b + t];
  const LaneMap m = lane_map<INTER>(l, a.rot);
  float c[4], s[4];
  Sh(a.inv_freq, m, sub).at(m.turned, p, l, c, s);
  constexpr int RPW = Sh::kRows;
  if (r0 < a.Hq) {
    T* dst = (T*)a.qo.p + b * a.qo.b + t * a.qo.t;
    fwd_rows<T, D, RPW, INTER, VEC, false>(qs, a.q.h, r0, min(r1, a.Hq), a.wq, a.norm, a.eps, m, c, s, sub,
                                           [&](int h) { return EACH && !live ? nullptr : dst + h * a.qo.h; });
  }
  if (k0 < k1) {
    if (PAGED) {
      fwd_rows<T, D, RPW, INTER, VEC, false>(ks, a.k.h, k0, k1, a.wk, a.norm, a.eps, m, c, s, sub, [&](int h) -> T* {
        if (pg < 0) return nullptr;
        const long long at = a.pg.row(pg, h, slot);
        if (a.weight && l == 0) a.weight[at] = 0.f;
        return (T*)a.k_pages + at * D;
      });
    } else {
      T* dst = (T*)a.ko.p + b * a.ko.b + t * a.ko.t;
      fwd_rows<T, D, RPW, INTER, VEC, false>(ks, a.k.h, k0, k1, a.wk, a.norm, a.eps, m, c, s, sub,
                                             [&](int h) { return EACH && !live ? nullptr : dst + h * a.ko.h; });
    }
  }
  if (PAGED) {
    if (v0 < v1 && (EACH || pg >= 0))
      fwd_rows<T, D, RPW, INTER, VEC, true>(vs, a.v.h, v0, v1, nullptr, false, 0.f, m, c, s, sub, [&](int h) -> T* {
        return EACH && pg < 0 ? nullptr : (T*)a.v_pages + a.pg.row(pg, h, slot) * D;
      });
  }
}

struct RopeBwdArgs {
  Operand gq, gk, q, k, dq, dk;
  const float *wq, *wk;
  const double* inv_freq;
  const int64_t* pos;
  long long pos_b, pos0;
  int B, L, Hq, Hk, rot, norm;
  float eps;
  int rows_per_item, items_per_token;
  float* part;  // [grid, 2, D] or NULL
};

constexpr int kWarpsBwd = 4;
// CTAs an SM has registers for, with eight rows of each warp in flight
template <typename T, typename GI>
constexpr int kBwdBlocks = sizeof(T) + sizeof(GI) == 4 ? 4 : 3;

// Gradients of rows h0 .. h1 - 1 of one token and one kind; acc gathers the
// lane's share of dw.
template <typename T, typename GI, typename GO, int D, int RPW, bool INTER, bool VEC>
__device__ __forceinline__ void bwd_rows(const GI* g, long long g_h, const T* src, long long x_h, GO* dst,
                                         long long d_h, int h0, int h1, const float* w, bool norm, float eps,
                                         const LaneMap& m, const float* c, const float* s, int sub, bool live, float* acc) {
  constexpr int kAhead = RPW > 1 ? 8 / RPW : 4;  // eight rows of a warp in flight (RPW 1: four of each token)
  float wl[8];
  lane_weights(w, m, wl);
  const int dq = m.qb - m.qa;
  const GI* pg = g + (h0 + sub) * g_h + m.qa;
  const T* px = src + (h0 + sub) * x_h + m.qa;
  GO* pd = dst + (h0 + sub) * d_h + m.qa;
  const long long sg = RPW * g_h, sx = RPW * x_h, sd = RPW * d_h;
  auto rows = [&](int h, auto full) {
    Quad<GI, VEC> ga[kAhead], gb[kAhead];
    Quad<T, VEC> xa[kAhead], xb[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const bool on = live && (full || h + i * RPW < h1);
      if (on) {
        ga[i].load(pg);
        gb[i].load(pg + dq);
      } else {
        ga[i].zero(), gb[i].zero();
      }
      if (on && norm) {
        xa[i].load(px);
        xb[i].load(px + dq);
      } else {
        xa[i].zero(), xb[i].zero();
      }
      pg += sg, px += sx;
    }
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const bool on = live && (full || h + i * RPW < h1);
      if (!full && h - sub + i * RPW >= h1) break;  // (none of the warp's rows)
      float u[8];
      ga[i].get(u), gb[i].get(u + 4);
      turn<INTER>(u, c, s);
      if (norm) {
        float x[8], ss = 0.f, gx = 0.f, t[8];
        xa[i].get(x), xb[i].get(x + 4);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          t[e] = u[e] * x[e];
          ss = fmaf(x[e], x[e], ss);
          gx = fmaf(t[e], wl[e], gx);
        }
        ss = row_sum<D / 8>(ss);
        gx = row_sum<D / 8>(gx);
        const float rn = rsqrtf(fmaf(ss, 1.f / D, eps));
        const float cx = gx * rn * rn * (1.f / D);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (on) acc[e] = fmaf(t[e], rn, acc[e]);
          u[e] = rn * fmaf(u[e], wl[e], -(cx * x[e]));
        }
      }
      if (on) {
        Quad<GO, VEC> o;
        o.set(u);
        o.store(pd);
        o.set(u + 4);
        o.store(pd + dq);
      }
      pd += sd;
    }
  };
  int h = h0;
  for (; h + kAhead * RPW <= h1; h += kAhead * RPW) rows(h + sub, std::true_type{});
  if (h < h1) rows(h + sub, std::false_type{});
}

// The same mapping on a fixed grid whose warps stride over the items and keep
// their shares of dw_q, dw_k in registers (8 entries of each a lane).  Bytes
// in flight bound it: 12 warps an SM with eight rows each 176 us, 16 with four
// 191 us; prefetching the next item to L2 as well 227 us (the prefetched rows
// push each other out).  EACH: items of as many tokens as a warp has groups.
template <typename T, typename GI, typename GO, int D, bool INTER, bool VEC, bool EACH>
__global__ void __launch_bounds__(kWarpsBwd * 32, kBwdBlocks<T, GI>) rope_bwd_kernel(RopeBwdArgs a) {
  constexpr int LPR = D / 8;
  __shared__ float red[kWarpsBwd][D];
  begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  using Sh = Share<LPR, EACH>;
  constexpr int RPW = Sh::kRows;
  const int l = lane % LPR, sub = lane / LPR, row0 = EACH ? 0 : sub;
  const LaneMap m = lane_map<INTER>(l, a.rot);
  const Sh share(a.inv_freq, m, sub);
  float aq[8], ak[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) aq[i] = ak[i] = 0.f;
  const int rows = a.Hq + a.Hk;
  const long long n_items = (long long)a.B * a.L * a.items_per_token;
  for (long long first = ((long long)blockIdx.x * kWarpsBwd + warp) * Sh::kTokens; first < n_items;
       first += (long long)gridDim.x * kWarpsBwd * Sh::kTokens) {
    const bool live = !EACH || first + sub < n_items;  // (else the last token again, for nothing)
    const long long item = EACH ? min(first + sub, n_items - 1) : first;
    const long long tok = item / a.items_per_token;
    const int b = (int)(tok / a.L), t = (int)(tok % a.L);
    const int r0 = EACH ? 0 : (int)(item % a.items_per_token) * a.rows_per_item;
    const int r1 = EACH ? rows : min(rows, r0 + a.rows_per_item);
    float c[4], s[4];
    share.at(m.turned, a.pos ? a.pos[b * a.pos_b + t] : a.pos0 + t, l, c, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = -s[i];
    if (r0 < a.Hq)
      bwd_rows<T, GI, GO, D, RPW, INTER, VEC>((const GI*)a.gq.p + b * a.gq.b + t * a.gq.t, a.gq.h,
                                              (const T*)a.q.p + b * a.q.b + t * a.q.t, a.q.h,
                                              (GO*)a.dq.p + b * a.dq.b + t * a.dq.t, a.dq.h, r0, min(r1, a.Hq), a.wq,
                                              a.norm, a.eps, m, c, s, row0, live, aq);
    const int k0 = max(r0 - a.Hq, 0), k1 = min(r1 - a.Hq, a.Hk);
    if (k0 < k1)
      bwd_rows<T, GI, GO, D, RPW, INTER, VEC>((const GI*)a.gk.p + b * a.gk.b + t * a.gk.t, a.gk.h,
                                              (const T*)a.k.p + b * a.k.b + t * a.k.t, a.k.h,
                                              (GO*)a.dk.p + b * a.dk.b + t * a.dk.t, a.dk.h, k0, k1, a.wk, a.norm, a.eps,
                                              m, c, s, row0, live, ak);
  }
  if (!a.part) return;
  // the CTA's sums: over the rows of a warp, then over the warps in order
#pragma unroll
  for (int which = 0; which < 2; ++which) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float v = which ? ak[i] : aq[i];
#pragma unroll
      for (int o = 16; o >= LPR; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
      if (sub == 0) red[warp][(i < 4 ? m.qa : m.qb - 4) + i] = v;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < D; e += kWarpsBwd * 32) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWarpsBwd; ++w) v += red[w][e];
      a.part[((long long)blockIdx.x * 2 + which) * D + e] = v;
    }
    __syncthreads();
  }
}

// dw[e] = sum over the partials, in order: 32 runs of partials per column
template <int D>
__global__ void rope_dw_kernel(const float* part, int n, float* dwq, float* dwk) {
  __shared__ float red[32][32];
  begin();
  const int col = blockIdx.x * 32 + threadIdx.x;  // of 2 D
  float v = 0.f;
#pragma unroll 8
  for (int i = threadIdx.y; i < n; i += 32) v += part[(long long)i * 2 * D + col];
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0) {
    v = 0.f;
#pragma unroll
    for (int y = 0; y < 32; ++y) v += red[y][threadIdx.x];
    float* o = col < D ? dwq : dwk;
    if (o) o[col % D] = v;
  }
}

constexpr int kSMs = 152;
constexpr int kBwdGrid = kSMs * 4;  // at most

// Rows a warp takes of one token: all of them when the tokens alone give
// `want` warps (those that run at once) their work, else an even share, so
// that short calls spread out but stay one wave.
void split_rows(long long tokens, int rows, int rpw, long long want, int* per_item, int* items) {
  const int most = (rows + rpw - 1) / rpw;
  long long n = tokens > 0 ? want / tokens : 1;
  if (n > most) n = most;
  if (n < 1) n = 1;
  int per = (most + (int)n - 1) / (int)n * rpw;
  *per_item = per;
  *items = (rows + per - 1) / per;
}

// (a stride that leads from nothing to nothing may be anything: 0)
Operand operand(const void* p, const nats_strides* s, int B, int H, int L) {
  return s ? Operand{p, B > 1 ? s->b : 0, H > 1 ? s->h : 0, L > 1 ? s->t : 0} : Operand{p, 0, 0, 0};
}

// quads of this operand start at multiples of their size
bool vec_ok(const Operand& o, int es) {
  if (!o.p) return true;
  return ((uintptr_t)o.p % (4 * es)) == 0 && o.b % 4 == 0 && o.h % 4 == 0 && o.t % 4 == 0;
}

bool elem_ok(const void* p, int es) { return ((uintptr_t)p % es) == 0; }

nats_status check_rope(const nats_rope_dims* d) {
  if (!d) return NATS_ERR_NULL;
  if (d->dtype != NATS_BF16 && d->dtype != NATS_F32) return NATS_ERR_DTYPE;
  if (d->B < 0 || d->L < 0 || d->Hq < 0 || d->Hk < 0) return NATS_ERR_SHAPE;
  if (d->d != 64 && d->d != 128) return NATS_ERR_UNSUPPORTED;
  if (d->rot < 0 || d->rot > d->d || d->rot % 8 != 0) return NATS_ERR_SHAPE;
  if (d->norm && (!std::isfinite(d->eps) || d->eps < 0.f)) return NATS_ERR_VALUE;
  if ((long long)d->Hq + 2LL * d->Hk > (1LL << 30)) return NATS_ERR_UNSUPPORTED;
  const double rows = (double)d->B * d->L * ((double)d->Hq + 2.0 * d->Hk);
  if (rows > 1099511627776.0 || (double)d->B * d->L > 4294967296.0) return NATS_ERR_UNSUPPORTED;
  return NATS_OK;
}

// Whether a warp's groups of lanes take a token each, its rows one after the
// other, in place of one token's rows side by side: where the tokens are more
// than the `wave` of warps that run at once and a token's rows are few, the
// chain from a position to a row is what a warp waits for, and two to four of
// them then run together.  `bytes`: of a token's rows, up to which the reads of
// a warp's tokens still follow one another closely enough (measured on both
// sides, time with a token each against without, 30,000 to 40,000 tokens):
//   forward  bf16 d 128: 1 + 1 heads 25 / 42 us, 12 + 4 58 / 69, 20 + 4 68 / 66
//            bf16 d 64: 1 + 1 14 / 36 us, 20 + 4 39 / 44, 16 + 16 63 / 61
//            fp32 d 128: 4 + 4 54 / 58 us, 8 + 2 67 / 66
//   gradient bf16 d 128: 1 + 1 39 / 66 us, 20 + 4 131 / 138, 24 + 4 151 / 150
//            fp32 d 128: 8 + 2 104 / 110 us, 16 + 4 148 / 146
// and with 3600 tokens (one wave) 12 + 4 heads 8.3 / 7.3 us forward.
bool token_each(long long tokens, long long wave, int rows, int row_bytes, int most_rows, int bytes, bool vec) {
  return vec && tokens > wave && rows <= most_rows && rows * row_bytes <= bytes;
}

template <bool PAGED>
cudaError_t launch_fwd(RopeArgs& a, int dtype, int d, bool inter, bool vec, cudaStream_t st) {
  const long long tokens = (long long)a.B * a.L;
  const int rows = a.Hq + a.Hk * (PAGED ? 2 : 1), rpw = 32 / (d / 8);
  const long long wave = (long long)kSMs * 3 * kWarps;
  split_rows(tokens, rows, rpw, wave, &a.rows_per_item, &a.items_per_token);
  const bool each = token_each(tokens, wave, rows, d * (dtype == NATS_BF16 ? 2 : 4), 24, 4096, vec);
  const long long warps = each ? (tokens + rpw - 1) / rpw : tokens * a.items_per_token;
  if (each) a.items_per_token = 1;
  const unsigned grid = (unsigned)((warps + kWarps - 1) / kWarps);
#define NATS_ROPE(T, D, I, V, E) after(rope_fwd_kernel<T, D, I, PAGED, V, E>, grid, kWarps * 32, 0, st, 0, a)
#define NATS_ROPE_V(T, D, I) \
  (each ? NATS_ROPE(T, D, I, true, true) : vec ? NATS_ROPE(T, D, I, true, false) : NATS_ROPE(T, D, I, false, false))
#define NATS_ROPE_I(T, D) (inter ? NATS_ROPE_V(T, D, true) : NATS_ROPE_V(T, D, false))
  if (dtype == NATS_BF16) return d == 128 ? NATS_ROPE_I(__nv_bfloat16, 128) : NATS_ROPE_I(__nv_bfloat16, 64);
  return d == 128 ? NATS_ROPE_I(float, 128) : NATS_ROPE_I(float, 64);
}

template <typename T, typename GI, typename GO>
cudaError_t launch_bwd(const RopeBwdArgs& a, int d, bool inter, bool vec, bool each, unsigned grid, cudaStream_t st) {
#define NATS_BWD(D, I, V, E) after(rope_bwd_kernel<T, GI, GO, D, I, V, E>, grid, kWarpsBwd * 32, 0, st, 0, a)
#define NATS_BWD_V(D, I) \
  (each ? NATS_BWD(D, I, true, true) : vec ? NATS_BWD(D, I, true, false) : NATS_BWD(D, I, false, false))
#define NATS_BWD_I(D) (inter ? NATS_BWD_V(D, true) : NATS_BWD_V(D, false))
  return d == 128 ? NATS_BWD_I(128) : NATS_BWD_I(64);
}

}  // namespace
}  // namespace nats

using namespace nats;

extern "C" {

nats_status nats_qk_norm_rope(const nats_rope_dims* dims, const void* q, const nats_strides* q_st, const void* k,
                              const nats_strides* k_st, const float* w_q, const float* w_k, const double* inv_freq,
                              const int64_t* pos, int64_t pos_stride_b, int64_t pos0, void* q_out,
                              const nats_strides* q_out_st, void* k_out, const nats_strides* k_out_st,
                              nats_stream_t stream) {
  const nats_status s = check_rope(dims);
  if (s != NATS_OK) return s;
  if (dims->B == 0 || dims->L == 0 || dims->Hq + dims->Hk == 0) return NATS_OK;
  if (dims->Hq > 0 && (!q || !q_st || !q_out || !q_out_st)) return NATS_ERR_NULL;
  if (dims->Hk > 0 && (!k || !k_st || !k_out || !k_out_st)) return NATS_ERR_NULL;
  if (dims->rot > 0 && !inv_freq) return NATS_ERR_NULL;
  const int es = dims->dtype == NATS_BF16 ? 2 : 4;
  RopeArgs a = {};
  const auto of = [&](const void* p, const nats_strides* st, int H) { return operand(p, st, dims->B, H, dims->L); };
  if (dims->Hq > 0) a.q = of(q, q_st, dims->Hq), a.qo = of(q_out, q_out_st, dims->Hq);
  if (dims->Hk > 0) a.k = of(k, k_st, dims->Hk), a.ko = of(k_out, k_out_st, dims->Hk);
  const Operand* ops[] = {&a.q, &a.k, &a.qo, &a.ko};
  bool vec = true;
  for (const Operand* o : ops) {
    if (!elem_ok(o->p, es)) return NATS_ERR_ALIGN;
    vec = vec && vec_ok(*o, es);
  }
  if (!elem_ok(w_q, 4) || !elem_ok(w_k, 4) || !elem_ok(inv_freq, 8) || !elem_ok(pos, 8)) return NATS_ERR_ALIGN;
  a.wq = dims->norm ? w_q : nullptr, a.wk = dims->norm ? w_k : nullptr;
  a.inv_freq = inv_freq, a.pos = pos, a.pos_b = pos_stride_b, a.pos0 = pos0;
  a.B = dims->B, a.L = dims->L, a.Hq = dims->Hq, a.Hk = dims->Hk, a.rot = dims->rot;
  a.norm = dims->norm, a.eps = dims->eps;
  return (nats_status)record_cuda_error(
      launch_fwd<false>(a, dims->dtype, dims->d, dims->interleaved != 0, vec, (cudaStream_t)stream));
}

nats_status nats_paged_append(const nats_paged_cache* cache, const nats_rope_dims* dims, const void* q,
                              const nats_strides* q_st, const void* k, const nats_strides* k_st, const void* v,
                              const nats_strides* v_st, const float* w_q, const float* w_k, const double* inv_freq,
                              const int32_t* start, const int32_t* n_new, const int64_t* pos, int64_t pos_stride_b,
                              void* q_out, const nats_strides* q_out_st, nats_stream_t stream) {
  nats_status s = check_cache(cache);
  if (s != NATS_OK) return s;
  s = check_rope(dims);
  if (s != NATS_OK) return s;
  if (dims->B != cache->B || dims->Hk != cache->Hk || dims->d != cache->d) return NATS_ERR_SHAPE;
  if (dims->dtype != cache->dtype) return NATS_ERR_DTYPE;
  if (dims->B == 0 || dims->L == 0) return NATS_OK;
  s = check_cache_pointers(cache);
  if (s != NATS_OK) return s;
  if (!k || !k_st || !v || !v_st) return NATS_ERR_NULL;
  if (dims->Hq > 0 && (!q || !q_st || !q_out || !q_out_st)) return NATS_ERR_NULL;
  if (dims->rot > 0 && !inv_freq) return NATS_ERR_NULL;
  const int es = dims->dtype == NATS_BF16 ? 2 : 4;
  RopeArgs a = {};
  const auto of = [&](const void* p, const nats_strides* st, int H) { return operand(p, st, dims->B, H, dims->L); };
  if (dims->Hq > 0) a.q = of(q, q_st, dims->Hq), a.qo = of(q_out, q_out_st, dims->Hq);
  a.k = of(k, k_st, dims->Hk), a.v = of(v, v_st, dims->Hk);
  const Operand* ops[] = {&a.q, &a.k, &a.v, &a.qo};
  bool vec = true;
  for (const Operand* o : ops) {
    if (!elem_ok(o->p, es)) return NATS_ERR_ALIGN;
    vec = vec && vec_ok(*o, es);
  }
  if (!elem_ok(w_q, 4) || !elem_ok(w_k, 4) || !elem_ok(inv_freq, 8) || !elem_ok(pos, 8) || !elem_ok(start, 4) ||
      !elem_ok(n_new, 4))
    return NATS_ERR_ALIGN;
  a.wq = dims->norm ? w_q : nullptr, a.wk = dims->norm ? w_k : nullptr;
  a.inv_freq = inv_freq, a.pos = pos, a.pos_b = pos_stride_b, a.pos0 = 0;
  a.B = dims->B, a.L = dims->L, a.Hq = dims->Hq, a.Hk = dims->Hk, a.rot = dims->rot;
  a.norm = dims->norm, a.eps = dims->eps;
  a.pg = view_of(cache), a.k_pages = cache->k_pages, a.v_pages = cache->v_pages, a.weight = cache->weight;
  a.start = start, a.n_new = n_new;
  return (nats_status)record_cuda_error(
      launch_fwd<true>(a, dims->dtype, dims->d, dims->interleaved != 0, vec, (cudaStream_t)stream));
}

size_t nats_qk_norm_rope_bwd_workspace_size(const nats_rope_dims* dims) {
  if (check_rope(dims) != NATS_OK) return 0;
  return sizeof(float) * kBwdGrid * 2 * dims->d;
}

nats_status nats_qk_norm_rope_bwd(const nats_rope_dims* dims, int32_t grad_dtype, int32_t dx_dtype,
                                  const void* dq_out, const nats_strides* dq_out_st, const void* dk_out,
                                  const nats_strides* dk_out_st, const void* q, const nats_strides* q_st,
                                  const void* k, const nats_strides* k_st, const float* w_q, const float* w_k,
                                  const double* inv_freq, const int64_t* pos, int64_t pos_stride_b, int64_t pos0,
                                  void* dq, const nats_strides* dq_st, void* dk, const nats_strides* dk_st,
                                  float* dw_q, float* dw_k, void* workspace, size_t workspace_bytes,
                                  nats_stream_t stream) {
  const nats_status s = check_rope(dims);
  if (s != NATS_OK) return s;
  if ((grad_dtype != NATS_BF16 && grad_dtype != NATS_F32) || (dx_dtype != NATS_BF16 && dx_dtype != NATS_F32))
    return NATS_ERR_DTYPE;
  if (dims->dtype == NATS_F32 && (grad_dtype != NATS_F32 || dx_dtype != NATS_F32)) return NATS_ERR_DTYPE;
  if (!dims->norm && (dw_q || dw_k)) return NATS_ERR_VALUE;
  const bool empty = dims->B == 0 || dims->L == 0 || dims->Hq + dims->Hk == 0;
  if (!empty) {
    if (dims->Hq > 0 && (!dq_out || !dq_out_st || !dq || !dq_st || (dims->norm && (!q || !q_st)))) return NATS_ERR_NULL;
    if (dims->Hk > 0 && (!dk_out || !dk_out_st || !dk || !dk_st || (dims->norm && (!k || !k_st)))) return NATS_ERR_NULL;
    if (dims->rot > 0 && !inv_freq) return NATS_ERR_NULL;
  }
  const int es = dims->dtype == NATS_BF16 ? 2 : 4, eg = grad_dtype == NATS_BF16 ? 2 : 4,
            eo = dx_dtype == NATS_BF16 ? 2 : 4;
  RopeBwdArgs a = {};
  const auto of = [&](const void* p, const nats_strides* st, int H) { return operand(p, st, dims->B, H, dims->L); };
  if (dims->Hq > 0)
    a.gq = of(dq_out, dq_out_st, dims->Hq), a.q = of(q, q_st, dims->Hq), a.dq = of(dq, dq_st, dims->Hq);
  if (dims->Hk > 0)
    a.gk = of(dk_out, dk_out_st, dims->Hk), a.k = of(k, k_st, dims->Hk), a.dk = of(dk, dk_st, dims->Hk);
  const Operand* ops[] = {&a.gq, &a.gk, &a.q, &a.k, &a.dq, &a.dk};
  const int sizes[] = {eg, eg, es, es, eo, eo};
  bool vec = true;
  for (int i = 0; i < 6; ++i) {
    if (!elem_ok(ops[i]->p, sizes[i])) return NATS_ERR_ALIGN;
    vec = vec && vec_ok(*ops[i], sizes[i]);
  }
  if (!elem_ok(w_q, 4) || !elem_ok(w_k, 4) || !elem_ok(dw_q, 4) || !elem_ok(dw_k, 4) || !elem_ok(inv_freq, 8) ||
      !elem_ok(pos, 8))
    return NATS_ERR_ALIGN;
  const bool dw = dw_q || dw_k;
  if (dw && !empty) {
    if (!workspace) return NATS_ERR_NULL;
    if ((uintptr_t)workspace & 15u) return NATS_ERR_ALIGN;
    if (workspace_bytes < nats_qk_norm_rope_bwd_workspace_size(dims)) return NATS_ERR_WORKSPACE;
  }
  cudaStream_t st = (cudaStream_t)stream;
  if (empty) {
    for (float* o : {dw_q, dw_k})
      if (o) {
        const int r = record_cuda_error(cudaMemsetAsync(o, 0, sizeof(float) * dims->d, st));
        if (r != NATS_OK) return (nats_status)r;
      }
    return NATS_OK;
  }
  a.wq = dims->norm ? w_q : nullptr, a.wk = dims->norm ? w_k : nullptr;
  a.inv_freq = inv_freq, a.pos = pos, a.pos_b = pos_stride_b, a.pos0 = pos0;
  a.B = dims->B, a.L = dims->L, a.Hq = dims->Hq, a.Hk = dims->Hk, a.rot = dims->rot;
  a.norm = dims->norm, a.eps = dims->eps;
  a.part = dw ? (float*)workspace : nullptr;
  const long long tokens = (long long)a.B * a.L;
  const int most = kSMs * (dims->dtype == NATS_BF16 && grad_dtype == NATS_BF16 ? kBwdBlocks<__nv_bfloat16, __nv_bfloat16>
                                                                             : kBwdBlocks<float, float>);
  split_rows(tokens, a.Hq + a.Hk, 32 / (dims->d / 8), most * kWarpsBwd, &a.rows_per_item, &a.items_per_token);
  const int rpw = 32 / (dims->d / 8);
  const bool each = token_each(tokens, most * kWarpsBwd, a.Hq + a.Hk, dims->d * es, 32, 6144, vec);
  if (each) a.items_per_token = 1;
  const long long warps = each ? (tokens + rpw - 1) / rpw : tokens * a.items_per_token;
  const long long ctas = (warps + kWarpsBwd - 1) / kWarpsBwd;
  const unsigned grid = (unsigned)(ctas < most ? ctas : most);
  const bool inter = dims->interleaved != 0;
  const int d = dims->d;
  cudaError_t e;
  if (dims->dtype == NATS_F32)
    e = launch_bwd<float, float, float>(a, d, inter, vec, each, grid, st);
  else if (grad_dtype == NATS_F32 && dx_dtype == NATS_F32)
    e = launch_bwd<__nv_bfloat16, float, float>(a, d, inter, vec, each, grid, st);
  else if (grad_dtype == NATS_F32)
    e = launch_bwd<__nv_bfloat16, float, __nv_bfloat16>(a, d, inter, vec, each, grid, st);
  else if (dx_dtype == NATS_F32)
    e = launch_bwd<__nv_bfloat16, __nv_bfloat16, float>(a, d, inter, vec, each, grid, st);
  else
    e = launch_bwd<__nv_bfloat16, __nv_bfloat16, __nv_bfloat16>(a, d, inter, vec, each, grid, st);
  const int r = record_cuda_error(e);
  if (r != NATS_OK || !dw) return (nats_status)r;
  const float* part = a.part;
  return (nats_status)record_cuda_error(after(d == 128 ? rope_dw_kernel<128> : rope_dw_kernel<64>, 2 * d / 32,
                                              dim3(32, 32), 0, st, 0, part, (int)grid, dw_q, dw_k));
}

}  // extern "C"
