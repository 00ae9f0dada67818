// decay_attn_tc.cu - linear attention with a decay for each head on the
// 5th-generation tensor cores (bf16 operands; decay.cuh has the mathematics).
//
// One CTA walks the 128-token chunks of one segment of one (scan, sequence,
// head) and 64 of the state's columns.  Per chunk, with Q, K, V its tiles, W
// the tokens' weights gamma^(n - 1 - j + e), all rows in memory order:
//   X  = Q K^T                    (128 x 128, K = d)
//   P  = X * gamma^|i - j| on the past side, bf16 in place of X in TMEM
//   Oi = Q S, Op = P V            (128 x 64)
//   o  = scale (Op + gamma^(..) Oi)
//   dS = K^T (W V)                (d x 64, K = 128), a fresh sum every chunk
//   S  <- gamma^n S + dS          (fp32, in registers; its bf16 copy feeds Oi)
// W V goes in as three bf16 numbers (their sum is its fp32 value), so dS is
// summed from exact products and the state is as good as an fp32 recurrence;
// P and the copy of S are rounded to bf16, half a step like the output's own.
//
// Roles (576 threads): warps 0-3 P, warps 4-7 state, warps 8-11 output, warps
// 12-15 W V, warp 16 TMA producer, warp 17 TMEM owner and MMA issuer.  The
// output takes the place of the chunk's V tile on its way out (TMA store).
// Every wait is bounded (tc::kWaitLimitNs); an expired one sets g_expired.
#include <cmath>
#include <mutex>

#include "decay.cuh"
#include "kernels.h"
#include "launch.cuh"
#include "tc.cuh"

namespace nats {
namespace decay {
namespace {

__device__ int g_expired;  // a wait of a kernel of this file gave up (nats_decay_attn_check)

constexpr int C = 128;
constexpr int kSplit = 3;  // bf16 numbers that make up an fp32 one

struct Maps {
  CUtensorMap q, k, v, o;
};
struct TcArgs {
  Args a;
  Maps m[kMaxOps];
};

template <int D, bool STATES>
struct Lay {
  static constexpr int kTile = C * D * 2;      // Q or K: D / 64 slabs of 128 lines of 128 bytes
  static constexpr int kV = C * kWidth * 2;    // 16 KiB
  static constexpr int kQ = STATES ? 0 : kTile;
  static constexpr int kStage = kQ + kTile + kV;
  static constexpr int kHalf = 64 * kWidth * 2;  // 64 tokens of one part of W V
  static constexpr int kStages = D == 128 && !STATES ? 2 : 3;
  static constexpr int offW = kStages * kStage;            // [half][part]
  static constexpr int offS = offW + 2 * kSplit * kHalf;   // D lines of 128 bytes
  static constexpr int offPow = offS + (STATES ? 0 : D * 128);  // gamma^m, m = 0 .. 128
  static constexpr int offBar = offPow + 136 * 4;
  static constexpr int kNumBars = 32;
  static constexpr int offTmem = offBar + kNumBars * 8;
  static constexpr int kBytes = offTmem + 16;
  static_assert(kBytes <= 232448, "shared memory");
};

enum {
  B_QK = 0,        // + stage: Q and K have landed
  B_V = 3,         // + stage: V has landed
  B_QKFREE = 6,    // + stage
  B_VFREE = 9,     // + stage
  B_X = 12,        // + chunk % 2: X is complete
  B_P = 14,        // + chunk % 2: P is in place
  B_W = 16,        // + half: W V is in place
  B_WFREE = 18,    // + half: its product with K is complete
  B_S = 20,        // the state ahead of the chunk is in place
  B_SREAD = 21,    // its product with Q is complete
  B_O = 22,        // Oi and Op are complete
  B_OREAD = 23,    // and read
  B_DONE = 24,
  B_D = 25,        // + chunk % 2: dS is complete
  B_DREAD = 27     // + chunk % 2: and read (without outputs; with them B_S of the next chunk says so)
};

// TMEM columns
constexpr uint32_t kColX = 0;     // two X / P buffers of 128
constexpr uint32_t kColOi = 256;  // 64
constexpr uint32_t kColOp = 320;  // 64
constexpr uint32_t kColD = 384;   // two dS buffers of 64

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int t, int h, int b, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::
          "r"(tc::smem_u32(dst)),
      "l"((uint64_t)map), "r"(x), "r"(t), "r"(h), "r"(b), "r"(tc::smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void tma_store_4d(const CUtensorMap* map, const void* src, int x, int t, int h, int b) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"((uint64_t)map),
               "r"(tc::smem_u32(src)), "r"(x), "r"(t), "r"(h), "r"(b)
               : "memory");
}

// 16-byte piece g of line r in a 128-byte-swizzled tile
__device__ __forceinline__ uint32_t piece(int r, int g) { return (uint32_t)(r * 128 + ((g ^ (r & 7)) << 4)); }

__device__ __forceinline__ float lo16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi16(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

template <int D, bool STATES>
__global__ void __launch_bounds__(576, 1) scan_tc_kernel(const __grid_constant__ TcArgs ta) {
  using M = Lay<D, STATES>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = (uint64_t*)(smem + M::offBar);
  uint32_t* tmem_slot = (uint32_t*)(smem + M::offTmem);
  float* pw = (float*)(smem + M::offPow);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < M::kNumBars; ++i) {
      const bool by_warps = i == B_P || i == B_P + 1 || i == B_W || i == B_W + 1 || i == B_S || i == B_OREAD || i == B_DREAD ||
                            i == B_DREAD + 1;
      tc::mbar_init(&bars[i], by_warps ? 4 : 1);
    }
    tc::fence_barrier_init();
  }
  if (warp == 17) {
    tc::tmem_alloc(tmem_slot, 512);
    tc::tmem_relinquish();
  }
  begin();
  const Args& a = ta.a;
  constexpr int kSlices = D / kWidth;
  const int segs = STATES ? a.segs - 1 : a.segs;
  int x = blockIdx.x;
  const int slice = x % kSlices;
  x /= kSlices;
  int seg = x % segs;
  x /= segs;
  const int bh = x % (a.B * a.H);
  const int iop = a.first_op + x / (a.B * a.H);
  const Op& op = a.op[iop];
  const Maps& maps = ta.m[iop];
  const int b = bh / a.H, h = bh % a.H;
  const bool back = op.back != 0;
  if (STATES && back) ++seg;  // (the first segment in the scan's order that another one follows)
  const int len = length(a, b);
  const int t0 = seg * a.seg, t1 = min(t0 + a.seg, a.L);
  const int n_seg = max(0, min(t1, len) - t0);
  const int N = (n_seg + C - 1) / C;
  const float g = a.g[h];
  const bool last_seg = seg == (back ? 0 : a.segs - 1);
  // chunks whose sums are wanted: all, or all but the last where no state goes on
  const int updates = STATES || (op.s_out && last_seg) ? N : N - 1;
  const auto chunk_at = [&](int c) { return back ? N - 1 - c : c; };
  const auto tokens_of = [&](int c) { return min(C, n_seg - chunk_at(c) * C); };
  if (threadIdx.x <= C) pw[threadIdx.x] = power(g, threadIdx.x);
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  int* err = &g_expired;

  if (warp == 16) {
    // ------------------------------------------------------------- producer
    if (lane == 0) {
      bool ok = true;
      int qk = 0, v = 0;
      for (int c = 0; c < N; ++c) {
        const int s = c % M::kStages, ph = ((c / M::kStages) & 1) ^ 1;
        const int t = t0 + chunk_at(c) * C;
        uint8_t* st = smem + s * M::kStage;
        if (!(ok = tc::mbar_wait(&bars[B_QKFREE + s], ph, err))) break;
        tc::mbar_arrive_expect_tx(&bars[B_QK + s], M::kQ + M::kTile);
        for (int y = 0; y < D / 64; ++y) {
          if (!STATES) tma_load_4d(st + y * 16384, &maps.q, 64 * y, t, h, b, &bars[B_QK + s]);
          tma_load_4d(st + M::kQ + y * 16384, &maps.k, 64 * y, t, h, b, &bars[B_QK + s]);
        }
        ++qk;
        if (!(ok = tc::mbar_wait(&bars[B_VFREE + s], ph, err))) break;
        tc::mbar_arrive_expect_tx(&bars[B_V + s], M::kV);
        tma_load_4d(st + M::kQ + M::kTile, &maps.v, kWidth * slice, t, h, b, &bars[B_V + s]);
        ++v;
      }
      // every copy issued has landed before the CTA may exit
      for (int s = 0; s < M::kStages; ++s) {
        const int nq = qk > s ? (qk - 1 - s) / M::kStages + 1 : 0, nv = v > s ? (v - 1 - s) / M::kStages + 1 : 0;
        if (nq > 0) tc::mbar_wait(&bars[B_QK + s], (nq - 1) & 1, nullptr);
        if (nv > 0) tc::mbar_wait(&bars[B_V + s], (nv - 1) & 1, nullptr);
      }
    }
  } else if (warp == 17) {
    // ------------------------------------------------------------------ MMA
    if (lane == 0 && N > 0) {
      constexpr uint32_t idX = tc::idesc_bf16_f32(128, 128, false, false), idO = tc::idesc_bf16_f32(128, 64, false, true),
                         idD = tc::idesc_bf16_f32(128, 64, true, true);
      const uint32_t s0 = tc::smem_u32(smem);
      const uint64_t qd0 = tc::smem_desc_sw128(s0, 16, 1024);
      const uint64_t kd0 = tc::smem_desc_sw128(s0 + M::kQ, 16, 1024);
      // K^T: features along M, 64 of them to a slab (for d = 64 rows 64 .. 127 are the V tile's: not read back)
      const uint64_t kt0 = tc::smem_desc_sw128(s0 + M::kQ, 16384, 1024);
      const uint64_t vd0 = tc::smem_desc_sw128(s0 + M::kQ + M::kTile, 16384, 1024);
      const uint64_t wd0 = tc::smem_desc_sw128(s0 + M::offW, 16384, 1024);
      const uint64_t sd0 = tc::smem_desc_sw128(s0 + M::offS, 16384, 1024);
      bool ok = true;
      const auto scores = [&](int c) {
        const int s = c % M::kStages;
        if (!tc::mbar_wait(&bars[B_QK + s], (c / M::kStages) & 1, err)) return false;
        tc::fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = s * M::kStage + (kk >> 2) * 16384 + (kk & 3) * 32;
          tc::mma_bf16(tmem + kColX + (c & 1) * 128, tc::desc_add(qd0, off), tc::desc_add(kd0, off), idX, kk > 0);
        }
        tc::mma_commit(&bars[B_X + (c & 1)]);
        return true;
      };
      if (!STATES) ok = scores(0);
      for (int c = 0; c < N && ok; ++c) {
        const int s = c % M::kStages;
        const uint32_t sb = s * M::kStage;
        if (STATES && !(ok = tc::mbar_wait(&bars[B_QK + s], (c / M::kStages) & 1, err))) break;
        // dS (its buffer was read before the state ahead of the last chunk was in place)
        if (STATES && c >= 2 && !(ok = tc::mbar_wait(&bars[B_DREAD + (c & 1)], ((c - 2) >> 1) & 1, err))) break;
#pragma unroll 1
        for (int hf = 0; hf < 2; ++hf) {
          if (!(ok = tc::mbar_wait(&bars[B_W + hf], c & 1, err))) break;
          if (c >= updates) continue;
          tc::fence_after();
#pragma unroll
          for (int p = 0; p < kSplit; ++p)
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc::mma_bf16(tmem + kColD + (c & 1) * 64, tc::desc_add(kt0, sb + hf * 8192 + kk * 2048),
                           tc::desc_add(wd0, (hf * kSplit + p) * M::kHalf + kk * 2048), idD, hf > 0 || p > 0 || kk > 0);
          tc::mma_commit(&bars[B_WFREE + hf]);
        }
        if (!ok) break;
        if (c < updates) tc::mma_commit(&bars[B_D + (c & 1)]);
        if (STATES) {
          tc::mma_commit(&bars[B_QKFREE + s]);
          continue;
        }
        // the next chunk's scores, into the buffer that the last one's P has left
        if (c + 1 < N) {
          if (c >= 1 && !(ok = tc::mbar_wait(&bars[B_O], (c - 1) & 1, err))) break;
          if (!(ok = scores(c + 1))) break;
        }
        if (!(ok = tc::mbar_wait(&bars[B_S], c & 1, err))) break;
        if (c >= 1 && !(ok = tc::mbar_wait(&bars[B_OREAD], (c - 1) & 1, err))) break;
        tc::fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          tc::mma_bf16(tmem + kColOi, tc::desc_add(qd0, sb + (kk >> 2) * 16384 + (kk & 3) * 32),
                       tc::desc_add(sd0, kk * 2048), idO, kk > 0);
        tc::mma_commit(&bars[B_SREAD]);
        tc::mma_commit(&bars[B_QKFREE + s]);
        if (!(ok = tc::mbar_wait(&bars[B_P + (c & 1)], (c >> 1) & 1, err))) break;
        tc::fence_after();
#pragma unroll
        for (int kk = 0; kk < C / 16; ++kk)
          tc::mma_bf16_ts(tmem + kColOp, tmem + kColX + (c & 1) * 128 + kk * 8, tc::desc_add(vd0, sb + kk * 2048), idO,
                          kk > 0);
        tc::mma_commit(&bars[B_O]);
      }
      tc::mma_commit(&bars[B_DONE]);
      tc::mbar_wait(&bars[B_DONE], 0, err);
    }
  } else if (warp < 4) {
    // -------------------------------------------------------------------- P
    if (!STATES) {
      const int w = warp;
      const uint32_t lane_off = (uint32_t)(32 * w) << 16;
      const int i = 32 * w + lane;
      // decays along a block's 32 columns, from the end next to the diagonal
      uint64_t cf[16];
#pragma unroll
      for (int j = 0; j < 16; ++j)
        cf[j] = back ? tc::f2_pack(pw[2 * j], pw[2 * j + 1]) : tc::f2_pack(pw[31 - 2 * j], pw[30 - 2 * j]);
      for (int c = 0; c < N; ++c) {
        const int n = tokens_of(c);
        if (!__all_sync(0xffffffffu, tc::mbar_wait(&bars[B_X + (c & 1)], (c >> 1) & 1, err))) break;
        tc::fence_after();
        const uint32_t tx = tmem + kColX + (c & 1) * 128 + lane_off;
#pragma unroll 1
        for (int blk = 0; blk < 4; ++blk) {
          uint32_t pk[16];
          if ((back ? blk >= w : blk <= w) && 32 * blk < n) {
            float s[32];
            tc::tmem_ld32(tx + 32 * blk, s);
            tc::tmem_ld_wait();
            if (blk != w) {
              const float rf = pw[back ? 32 * blk - i : i - 32 * blk - 31];
              const uint64_t r2 = tc::f2_pack(rf, rf);
#pragma unroll
              for (int j = 0; j < 16; ++j) {
                float p0, p1;
                tc::f2_unpack(tc::f2_mul(tc::f2_pack(s[2 * j], s[2 * j + 1]), tc::f2_mul(cf[j], r2)), p0, p1);
                s[2 * j] = p0, s[2 * j + 1] = p1;
              }
            } else {
#pragma unroll
              for (int j = 0; j < 32; ++j) {
                const int m = back ? j - lane : lane - j;
                s[j] = m >= 0 ? s[j] * pw[m & 31] : 0.f;
              }
            }
            // (scores with tokens behind the end may be anything)
            if (32 * blk + 32 > n)
#pragma unroll
              for (int j = 0; j < 32; ++j) s[j] = 32 * blk + j < n ? s[j] : 0.f;
#pragma unroll
            for (int j = 0; j < 16; ++j) pk[j] = tc::pack_bf16x2(s[2 * j], s[2 * j + 1]);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) pk[j] = 0u;
          }
          tc::tmem_st16u(tx + 16 * blk, pk);  // over columns of X that have been read
        }
        tc::tmem_st_wait();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars[B_P + (c & 1)]);
      }
    }
  } else if (warp < 8) {
    // ---------------------------------------------------------------- state
    const int w = warp - 4, r = 32 * w + lane;
    const uint32_t lane_off = (uint32_t)(32 * w) << 16;
    const bool has = r < D;  // (warp-uniform)
    float S[kWidth];
    const long long at = (long long)bh * D * D;
    if (STATES || !has) {
#pragma unroll
      for (int i = 0; i < kWidth; ++i) S[i] = 0.f;
    } else if (a.segs > 1) {
      const float* p = op.part + ((long long)bh * a.segs + seg) * D * D;
#pragma unroll
      for (int i = 0; i < kWidth; ++i) {
        const int col = slice * kWidth + i;
        S[i] = p[op.part_t ? r * D + col : col * D + r];
      }
    } else {
#pragma unroll
      for (int i = 0; i < kWidth; ++i)
        S[i] = op.s_in ? op.s_in[at + r * op.s_r + (slice * kWidth + i) * op.s_c] * op.in_scale : 0.f;
    }
    const auto publish = [&]() {  // the bf16 copy that the queries meet
      if (has) {
        uint8_t* line = smem + M::offS;
#pragma unroll
        for (int gg = 0; gg < 8; ++gg)
          *(uint4*)(line + piece(r, gg)) =
              make_uint4(tc::pack_bf16x2(S[8 * gg], S[8 * gg + 1]), tc::pack_bf16x2(S[8 * gg + 2], S[8 * gg + 3]),
                         tc::pack_bf16x2(S[8 * gg + 4], S[8 * gg + 5]), tc::pack_bf16x2(S[8 * gg + 6], S[8 * gg + 7]));
        tc::fence_proxy_async_smem();
      }
      tc::fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars[B_S]);
    };
    if (!STATES) publish();
    bool ok = true;
    const Carry whole(g, C);
    for (int c = 0; c < updates; ++c) {
      const int n = tokens_of(c);
      if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait(&bars[B_D + (c & 1)], (c >> 1) & 1, err)))) break;
      tc::fence_after();
      const Carry carry = n == C ? whole : Carry(g, n);
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        float d[32];
        tc::tmem_ld32(tmem + kColD + (c & 1) * 64 + 32 * hf + lane_off, d);
        tc::tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) S[32 * hf + i] = carry(S[32 * hf + i], d[i]);
      }
      if (STATES) {
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars[B_DREAD + (c & 1)]);
      } else if (c + 1 < N) {
        if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait(&bars[B_SREAD], c & 1, err)))) break;
        publish();
      }
    }
    if (ok && has) {
      if (STATES) {
        float* p = op.part + ((long long)bh * a.segs + (back ? seg - 1 : seg + 1)) * D * D;
#pragma unroll
        for (int i = 0; i < kWidth; ++i) p[(slice * kWidth + i) * D + r] = S[i];
      } else if (op.s_out && last_seg) {
#pragma unroll
        for (int i = 0; i < kWidth; ++i) op.s_out[at + r * op.s_r + (slice * kWidth + i) * op.s_c] = S[i] * op.out_scale;
      }
    }
  } else if (warp < 12) {
    // --------------------------------------------------------------- output
    if (!STATES) {
      const int w = warp - 8, i = 32 * w + lane;
      const uint32_t lane_off = (uint32_t)(32 * w) << 16;
      bool ok = true;
      for (int c = 0; c < N; ++c) {
        const int s = c % M::kStages, n = tokens_of(c);
        if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait(&bars[B_O], c & 1, err)))) break;
        tc::fence_after();
        uint8_t* tile = smem + s * M::kStage + M::kQ + M::kTile;
        const float wi = i < n ? pw[back ? n - 1 - i : i + 1] * a.scale : 0.f;
        uint32_t o[32];
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          float oi[32], po[32];
          tc::tmem_ld32(tmem + kColOi + 32 * hf + lane_off, oi);
          tc::tmem_ld32(tmem + kColOp + 32 * hf + lane_off, po);
          tc::tmem_ld_wait();
          if (hf == 1) {
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[B_OREAD]);
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            const float x0 = fmaf(oi[2 * j], wi, po[2 * j] * a.scale), x1 = fmaf(oi[2 * j + 1], wi, po[2 * j + 1] * a.scale);
            o[16 * hf + j] = i < n ? tc::pack_bf16x2(x0, x1) : 0u;
          }
        }
#pragma unroll
        for (int gg = 0; gg < 8; ++gg)
          *(uint4*)(tile + piece(i, gg)) = make_uint4(o[4 * gg], o[4 * gg + 1], o[4 * gg + 2], o[4 * gg + 3]);
        tc::fence_proxy_async_smem();
        tc::named_barrier(1, 128);
        if (threadIdx.x == 256) {
          tma_store_4d(&maps.o, tile, kWidth * slice, t0 + chunk_at(c) * C, h, b);
          tc::bulk_commit();
          tc::bulk_wait_read_all();
          tc::mbar_arrive(&bars[B_VFREE + s]);
        }
      }
      if (threadIdx.x == 256) tc::bulk_wait_all();
      // rows behind the sequence's end
      __nv_bfloat16* o = (__nv_bfloat16*)op.o.p + b * op.o.b + h * op.o.h + slice * kWidth;
      for (int e = threadIdx.x - 256; e < (t1 - t0 - N * C) * (kWidth / 8); e += 128)
        *(uint4*)(o + (t0 + N * C + e / (kWidth / 8)) * op.o.t + (e % (kWidth / 8)) * 8) = make_uint4(0, 0, 0, 0);
    }
  } else {
    // ------------------------------------------------------------------ W V
    const int el = threadIdx.x - 384;
    bool ok = true;
    for (int c = 0; c < N && ok; ++c) {
      const int s = c % M::kStages, n = tokens_of(c);
      uint8_t* kt = smem + s * M::kStage + M::kQ;
      uint8_t* vt = kt + M::kTile;
      // tokens behind the end that the loads have brought along are taken out of K and V
      const bool ragged = n < C && t0 + chunk_at(c) * C + n < a.L;
      if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait(&bars[B_V + s], (c / M::kStages) & 1, err)))) break;
      if (ragged) {
        // (K once its scores are complete)
        uint64_t* ready = STATES ? &bars[B_QK + s] : &bars[B_X + (c & 1)];
        const uint32_t ph = STATES ? (c / M::kStages) & 1 : (c >> 1) & 1;
        if (!(ok = __all_sync(0xffffffffu, tc::mbar_wait(ready, ph, err)))) break;
        for (int e = el; e < (C - n) * 8; e += 128) {
          *(uint4*)(vt + (n + e / 8) * 128 + (e % 8) * 16) = make_uint4(0, 0, 0, 0);
          for (int y = 0; y < D / 64; ++y) *(uint4*)(kt + y * 16384 + (n + e / 8) * 128 + (e % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
        tc::named_barrier(2, 128);
      }
#pragma unroll 1
      for (int hf = 0; hf < 2; ++hf) {
        // (also ahead of a chunk without a sum: B_W must not run two chunks ahead of the products)
        if (c > 0 && !(ok = __all_sync(0xffffffffu, tc::mbar_wait(&bars[B_WFREE + hf], (c - 1) & 1, err)))) break;
        if (c < updates) {
          uint8_t* dst = smem + M::offW + hf * kSplit * M::kHalf;
#pragma unroll
          for (int it = 0; it < 4; ++it) {
            const int row = it * 16 + (el >> 3), j = 64 * hf + row, gg = el & 7;
            const float wj = j < n ? pw[back ? j + 1 : n - 1 - j] : 0.f;
            const uint4 in = *(const uint4*)(vt + piece(j, gg));
            const uint32_t u[4] = {in.x, in.y, in.z, in.w};
            uint32_t p[kSplit][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              float x0 = lo16(u[e]) * wj, x1 = hi16(u[e]) * wj;
#pragma unroll
              for (int y = 0; y < kSplit; ++y) {
                const uint32_t z = tc::pack_bf16x2(x0, x1);
                p[y][e] = z;
                x0 -= lo16(z), x1 -= hi16(z);
              }
            }
#pragma unroll
            for (int y = 0; y < kSplit; ++y)
              *(uint4*)(dst + y * M::kHalf + piece(row, gg)) = make_uint4(p[y][0], p[y][1], p[y][2], p[y][3]);
          }
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars[B_W + hf]);
      }
      if (STATES && ok) {
        tc::named_barrier(2, 128);
        if (el == 0) tc::mbar_arrive(&bars[B_VFREE + s]);
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  if (warp == 17) {
    tc::fence_after();
    tc::tmem_dealloc(tmem, 512);
  }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = (EncodeTiledFn)ptr;
  });
  return fn;
}

// [B, H, L, d] as boxes of 128 tokens x 64 entries of one head, 128-byte
// swizzle; rows behind L read as zero and are not written.
bool make_map(CUtensorMap* map, const Tokens& x, const Args& a, int d) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const auto stride = [](int extent, long long s) { return (cuuint64_t)(extent == 1 ? 16 : 2 * s); };
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)a.L, (cuuint64_t)a.H, (cuuint64_t)a.B};
  const cuuint64_t strides[3] = {stride(a.L, x.t), stride(a.H, x.h), stride(a.B, x.b)};
  const cuuint32_t box[4] = {64, C, 1, 1}, estr[4] = {1, 1, 1, 1};
  return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, x.p, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool STATES>
cudaError_t launch(const TcArgs& ta, cudaStream_t st) {
  auto kern = scan_tc_kernel<D, STATES>;
  const int smem = Lay<D, STATES>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const Args& a = ta.a;
  const long long grid = (long long)(a.last_op - a.first_op) * a.B * a.H * (D / kWidth) * (STATES ? a.segs - 1 : a.segs);
  return after(kern, (unsigned)grid, dim3(576), smem, st, 0, ta);
}

}  // namespace

cudaError_t launch_tc(const Args& a, int d, bool states_only, cudaStream_t st) {
  TcArgs ta;
  ta.a = a;
  for (int i = a.first_op; i < a.last_op; ++i)
    if (!make_map(&ta.m[i].q, a.op[i].q, a, d) || !make_map(&ta.m[i].k, a.op[i].k, a, d) ||
        !make_map(&ta.m[i].v, a.op[i].v, a, d) || !make_map(&ta.m[i].o, a.op[i].o, a, d))
      return cudaErrorInvalidValue;
  if (states_only) return d == 64 ? launch<64, true>(ta, st) : launch<128, true>(ta, st);
  return d == 64 ? launch<64, false>(ta, st) : launch<128, false>(ta, st);
}

cudaError_t expired_waits(int* out, cudaStream_t st) {
  cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_expired, sizeof(int), 0, cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  const int zero = 0;
  if (e == cudaSuccess && *out) {
    e = cudaMemcpyToSymbolAsync(g_expired, &zero, sizeof(int), 0, cudaMemcpyHostToDevice, st);
    if (e == cudaSuccess) e = cudaStreamSynchronize(st);
  }
  return e;
}

}  // namespace decay
}  // namespace nats
