// decay_attn_tc.cu - linear attention with a decay for each head on the
// 5th-generation tensor cores (bf16 operands; decay.cuh has the mathematics).
//
// One CTA walks the 128-token chunks of one segment of one (scan, sequence,
// head) and 64 of the state's columns.  Per chunk, with Q, K, V its tiles, W
// the tokens' weights x gamma^(n - 1 - j + e), all rows in memory order:
//   X  = Q K^T                    (128 x 128, K = d)
//   P  = X * gamma^|i - j| on the past side, bf16, in TMEM
//   Oi = Q S, Op = P V            (128 x 64)
//   o  = scale Op + y gamma^(..) Oi
//   dS = K^T (W V)                (d x 64, K = 128), a fresh sum every chunk
//   S  <- gamma^n S + dS          (fp32, in registers; its bf16 copy feeds Oi)
// W V goes in as three bf16 numbers whose sum is its fp32 value, so dS is
// summed from exact products and a state that is given out is as good as an
// fp32 recurrence's (two numbers, 2^-16, where it is not); P and the copy of S
// that meets the queries are rounded to bf16, half a step each like the
// output's own.
//
// Roles: four warps for P, four for the state, four for the output, eight for
// W V, one for the loads, two that issue MMAs (X, Oi, Op; dS).
// Every wait on an mbarrier is bounded; an expired one sets g_expired.  A
// barrier of several warps is met by all of them whether their waits have
// ended or not (W V's, the output's), so that it ends too.
//
// Measured on one GB300, 4 x 16 heads of 8192 tokens, d = 128: 117 to 121 us, 4.5
// TB/s of the tensors' own bytes (HBM copy rate 6.7), 1.8 us a chunk; the three
// scans of its gradient 344 to 355 us; d = 64 88 and 191 us.  Bound by shared memory
// and the chain of a chunk's steps: 370 to 410 KB a chunk, 2900 to 3200 of its 3300
// cycles at 128 bytes each (tensor pipe 45 %, issue slots 42 %).  64
// columns a CTA so that few heads fill the GPU and two stages of tiles fit; 128
// tokens a chunk because an MMA of 64 rows takes as long as one of 128.
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
struct Maps {
  CUtensorMap q, k, v, o;
};
struct TcArgs {
  Args a;
  Maps m[kMaxOps];
};

// Decays between tokens.  Entry y of the table is gamma^m with m = 127 - y
// forward, y - 31 backward, and 0 where m < 0, so that the decays from row i to
// columns j, j + 1, .. are the entries from y = kFrom - i + j on (kFrom 127 or
// 31) and the future's are zero.  It is held four times, the copy s shifted by s
// entries, for reads of four entries wherever a row starts; kCopy puts the
// copies' pieces in different banks.
constexpr int kCopy = 168;
constexpr int kPowBytes = 4 * kCopy * 4;
constexpr int kPow128 = 160;  // gamma^128 (copy 0)

// Shared memory.  PARTS: the bf16 numbers that make up an entry of W V.
template <int D, bool STATES, int PARTS>
struct Lay {
  static constexpr int kTile = C * D * 2;      // Q or K: D / 64 slabs of 128 lines of 128 bytes
  static constexpr int kV = C * kWidth * 2;    // 16 KiB
  static constexpr int kQ = STATES ? 0 : kTile;
  static constexpr int kStage = kQ + kTile + kV;
  static constexpr int kStages = D == 128 && !STATES ? 2 : 3;
  // tokens of W V that are held of each half of a chunk: all, or half of them at a time where there is no room
  static constexpr int kStep = D == 128 && !STATES && PARTS == 3 ? 32 : 64;
  static constexpr int kSteps = 64 / kStep;
  static constexpr int kPart = kStep * kWidth * 2;
  static constexpr int offW = kStages * kStage;               // [half][part]
  static constexpr int offS = offW + 2 * PARTS * kPart;       // D lines of 128 bytes
  static constexpr int offO = offS + (STATES ? 0 : D * 128);  // the output's tile
  static constexpr int offPow = offO + (STATES ? 0 : kV);
  static constexpr int offBar = offPow + kPowBytes;
  static constexpr int kNumBars = 32;
  static constexpr int offTmem = offBar + kNumBars * 8;
  static constexpr int kBytes = offTmem + 16;
  static_assert(kBytes <= 232448, "shared memory");
};

enum {
  B_QK = 0,      // + stage: Q and K have landed
  B_V = 3,       // + stage: V has landed
  B_QKFREE = 6,  // + stage
  B_VFREE = 9,   // + stage
  B_W = 15,      // + half: W V is in place
  B_WFREE = 17,  // + half: its product with K is complete
  B_X = 19,      // X is complete
  B_XREAD = 20,  // and read
  B_P = 21,      // P is in place
  B_S = 22,      // the state ahead of the chunk is in place
  B_SREAD = 23,  // its product with Q is complete
  B_O = 24,      // Oi and Op are complete
  B_OREAD = 25,  // and read
  B_D = 26,      // dS is complete
  B_DREAD = 27,  // and read
  // of the chunk that holds tokens behind the end (at most one of a segment): its scores have been read; the tokens
  // are out of K and V
  B_RAGGED = 28,
  B_CLEAN = 29,
  B_DONE = 30,   // + MMA warp
};

// TMEM columns
constexpr uint32_t kColX = 0;     // 128
constexpr uint32_t kColP = 128;   // 64: two bf16 to a column
constexpr uint32_t kColOi = 192;  // 64
constexpr uint32_t kColOp = 256;  // 64
constexpr uint32_t kColD = 320;   // 64 for each part of W V
// (without outputs there is room for two dS, of chunks c % 2)
template <bool STATES>
__device__ __forceinline__ uint32_t col_d(int c) { return STATES ? (c & 1) * 192 : kColD; }
template <bool STATES>
__device__ __forceinline__ int bar_d(int c) { return STATES && (c & 1) ? B_X : B_D; }
template <bool STATES>
__device__ __forceinline__ int bar_dread(int c) { return STATES && (c & 1) ? B_XREAD : B_DREAD; }

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

// The warp's first lane issues; the others go along, so that the descriptors
// stay in uniform registers.
__device__ __forceinline__ void mma_if(uint32_t leader, uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void mma_ts_if(uint32_t leader, uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc), "r"(leader)
      : "memory");
}
__device__ __forceinline__ void commit_if(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(tc::smem_u32(bar)),
      "r"(leader)
      : "memory");
}
// Waits for the phase of parity `parity` to complete, asleep up to 10 us a
// try; gives up after 2^17 tries (5 ms at the least, 1.3 s at most; the waits
// of a CTA are for its own work, microseconds).  The
// loop is kept short: the roles' code goes through one instruction cache, and
// what is unrolled is fetched again for every chunk (4 x 16 heads of 8192 tokens:
// 125 us; unrolled by four 226, with a clock read in the loop 165; with the
// limit an argument of the launch 131,072 tokens of 8 heads 328 -> 347 us).
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity) {
  const uint32_t at = tc::smem_u32(bar);
  uint32_t ok = 0;
#pragma unroll 1
  for (int i = 0; i < (1 << 17) && !ok; ++i)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(at), "r"(parity), "r"(10000u)
        : "memory");
  return ok;
}
__device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait(bar, parity));
}

// 16-byte piece g of line r in a 128-byte-swizzled tile
__device__ __forceinline__ uint32_t piece(int r, int g) { return (uint32_t)(r * 128 + ((g ^ (r & 7)) << 4)); }

__device__ __forceinline__ float lo16(uint32_t x) { return __uint_as_float(x << 16); }
__device__ __forceinline__ float hi16(uint32_t x) { return __uint_as_float(x & 0xffff0000u); }

// First warp of each role (P from warp 0).  The four warps of a warpgroup share
// a register budget: the launch's 80 a thread, 480 in six warpgroups, are dealt
// out as 80 (P), 152 (state), 72 (output), 64 and 64 (W V), 40 (loads, MMAs).
// Nothing that a role calls may stay a function of its own: it would be compiled
// for more registers than the warp has left.
constexpr int kThreads = 768;
constexpr int kState = 4, kOut = 8, kW = 12, kLoad = 20, kMma = 21, kMmaD = 22;
template <int R>
__device__ __forceinline__ void registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R));
}
template <int R>
__device__ __forceinline__ void registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R));
}

template <int D, bool STATES, int PARTS>
__global__ void __launch_bounds__(kThreads, 1) scan_tc_kernel(const __grid_constant__ TcArgs ta) {
  using M = Lay<D, STATES, PARTS>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = (uint64_t*)(smem + M::offBar);
  uint32_t* tmem_slot = (uint32_t*)(smem + M::offTmem);
  float* tab = (float*)(smem + M::offPow);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < M::kNumBars; ++i) {
      const bool four = i == B_W || i == B_W + 1 || i == B_XREAD || i == B_P || i == B_S || i == B_OREAD || i == B_DREAD ||
                        i == B_RAGGED;                                 // the warps of a role
      const bool two = !STATES && i >= B_QKFREE && i < B_QKFREE + 3;  // both MMA warps
      const bool vfree = i >= B_VFREE && i < B_VFREE + 3;             // both W V groups, and P V
      tc::mbar_init(&bars[i], vfree ? (STATES ? 8 : 9) : i == B_CLEAN ? 8 : four ? 4 : two ? 2 : 1);
    }
    tc::fence_barrier_init();
  }
  if (warp == kMma) {
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
  // the one chunk that may hold fewer than C tokens
  const int part_c = back ? 0 : N - 1, part_n = n_seg - (N - 1) * C;
  const auto tokens_of = [&](int c) { return c == part_c ? part_n : C; };
  // a chunk whose tile holds tokens behind the sequence's end
  const int ragged_c = part_n < C && t0 + n_seg < a.L ? part_c : -1;
  const auto ragged_at = [&](int c) { return c == ragged_c; };
  for (int e = threadIdx.x; e < 4 * kCopy; e += kThreads) {
    const int y = e % kCopy + e / kCopy, m = back ? y - 31 : 127 - y;
    tab[e] = e == kPow128 ? power(g, 128) : m >= 0 ? power(g, m) : 0.f;
  }
  const auto pw = [&](int m) { return m == 128 ? tab[kPow128] : tab[back ? m + 31 : 127 - m]; };
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = *tmem_slot;
  // whether this warp's waits have all ended; a role that one left goes to the end, where it is recorded
  bool ok = true;

  if (warp >= kLoad) {
    registers_down<40>();
    if (warp == kLoad && lane == 0) {
      // ----------------------------------------------------------- producer
      int qk = 0, v = 0;
      for (int c = 0; c < N; ++c) {
        const int s = c % M::kStages, ph = ((c / M::kStages) & 1) ^ 1;
        const int t = t0 + chunk_at(c) * C;
        uint8_t* st = smem + s * M::kStage;
        if (!(ok = wait(&bars[B_QKFREE + s], ph))) break;
        tc::mbar_arrive_expect_tx(&bars[B_QK + s], M::kQ + M::kTile);
        for (int y = 0; y < D / 64; ++y) {
          tma_load_4d(st + M::kQ + y * 16384, &maps.k, 64 * y, t, h, b, &bars[B_QK + s]);
          if (!STATES) tma_load_4d(st + y * 16384, &maps.q, 64 * y, t, h, b, &bars[B_QK + s]);
        }
        ++qk;
        if (!(ok = wait(&bars[B_VFREE + s], ph))) break;
        tc::mbar_arrive_expect_tx(&bars[B_V + s], M::kV);
        tma_load_4d(st + M::kQ + M::kTile, &maps.v, kWidth * slice, t, h, b, &bars[B_V + s]);
        ++v;
      }
      // every copy issued has landed before the CTA may exit
      for (int s = 0; s < M::kStages; ++s) {
        const int nq = qk > s ? (qk - 1 - s) / M::kStages + 1 : 0, nv = v > s ? (v - 1 - s) / M::kStages + 1 : 0;
        if (nq > 0) wait(&bars[B_QK + s], (nq - 1) & 1);
        if (nv > 0) wait(&bars[B_V + s], (nv - 1) & 1);
      }
    } else if (!STATES && warp == kMma && N > 0) {
      // --------------------------------------------------- MMA: X, Oi and Op
      const uint32_t leader = lane == 0;
      constexpr uint32_t idX = tc::idesc_bf16_f32(128, 128, false, false), idO = tc::idesc_bf16_f32(128, 64, false, true);
      const uint32_t s0 = tc::smem_u32(smem);
      const uint64_t qd0 = tc::smem_desc_sw128(s0, 16, 1024);
      const uint64_t kd0 = tc::smem_desc_sw128(s0 + M::kQ, 16, 1024);
      const uint64_t vd0 = tc::smem_desc_sw128(s0 + M::kQ + M::kTile, 16384, 1024);
      const uint64_t sd0 = tc::smem_desc_sw128(s0 + M::offS, 16384, 1024);
      const auto scores = [&](int s, int phase) {
        if (!wait_all(&bars[B_QK + s], phase)) return false;
        tc::fence_after();
        const uint64_t qd = tc::desc_add(qd0, s * M::kStage), kd = tc::desc_add(kd0, s * M::kStage);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * 16384 + (kk & 3) * 32;
          mma_if(leader, tmem + kColX, tc::desc_add(qd, off), tc::desc_add(kd, off), idX, kk > 0);
        }
        commit_if(leader, &bars[B_X]);
        return true;
      };
      ok = scores(0, 0);
      int s = 0, phase = 0;
      for (int c = 0; c < N && ok; ++c) {
        const uint32_t sb = s * M::kStage;
        const int s1 = s + 1 == M::kStages ? 0 : s + 1, phase1 = s1 == 0 ? phase ^ 1 : phase;
        if (!(ok = wait_all(&bars[B_S], c & 1))) break;
        if (c >= 1 && !(ok = wait_all(&bars[B_OREAD], (c - 1) & 1))) break;
        tc::fence_after();
        const uint64_t qd = tc::desc_add(qd0, sb), vd = tc::desc_add(vd0, sb);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_if(leader, tmem + kColOi, tc::desc_add(qd, (kk >> 2) * 16384 + (kk & 3) * 32), tc::desc_add(sd0, kk * 2048), idO,
                 kk > 0);
        commit_if(leader, &bars[B_SREAD]);
        commit_if(leader, &bars[B_QKFREE + s]);
        // the next chunk's scores as soon as the last one's have been read
        if (c + 1 < N) {
          if (!(ok = wait_all(&bars[B_XREAD], c & 1))) break;
          if (!(ok = scores(s1, phase1))) break;
        }
        if (ragged_at(c) && !(ok = wait_all(&bars[B_CLEAN], 0))) break;
        if (!(ok = wait_all(&bars[B_V + s], phase))) break;
        if (!(ok = wait_all(&bars[B_P], c & 1))) break;
        tc::fence_after();
#pragma unroll
        for (int kk = 0; kk < C / 16; ++kk)
          mma_ts_if(leader, tmem + kColOp, tmem + kColP + kk * 8, tc::desc_add(vd, kk * 2048), idO, kk > 0);
        commit_if(leader, &bars[B_O]);
        commit_if(leader, &bars[B_VFREE + s]);
        s = s1, phase = phase1;
      }
      commit_if(leader, &bars[B_DONE]);
      ok = wait_all(&bars[B_DONE], 0) && ok;
    } else if (warp == kMmaD && N > 0) {
      // --------------------------------------------------------- MMA: dS
      const uint32_t leader = lane == 0;
      constexpr uint32_t idD = tc::idesc_bf16_f32(128, 64 * PARTS, true, true);
      const uint32_t s0 = tc::smem_u32(smem);
      // K^T: features along M, 64 of them to a slab (for d = 64 rows 64 .. 127 are the V tile's: not read back);
      // the parts of W V side by side along N
      const uint64_t kt0 = tc::smem_desc_sw128(s0 + M::kQ, 16384, 1024);
      const uint64_t wd0 = tc::smem_desc_sw128(s0 + M::offW, M::kPart, 1024);
      int s = 0, phase = 0;
      for (int c = 0; c < N; ++c) {
        if (!(ok = wait_all(&bars[B_QK + s], phase))) break;
        if (c < updates) {
          if (STATES) {
            if (c >= 2 && !(ok = wait_all(&bars[bar_dread<true>(c)], ((c - 2) >> 1) & 1))) break;
          } else if (c >= 1 && !(ok = wait_all(&bars[B_DREAD], (c - 1) & 1))) {
            break;
          }
          const uint64_t kt = tc::desc_add(kt0, s * M::kStage);
#pragma unroll
          for (int x = 0; x < 2 * M::kSteps && ok; ++x) {
            const int q = x >> 1, hf = x & 1;
            if (!(ok = wait_all(&bars[B_W + hf], (c * M::kSteps + q) & 1))) break;
            tc::fence_after();
#pragma unroll
            for (int kk = 0; kk < M::kStep / 16; ++kk)
              mma_if(leader, tmem + col_d<STATES>(c), tc::desc_add(kt, hf * 8192 + q * M::kStep * 128 + kk * 2048),
                     tc::desc_add(wd0, hf * PARTS * M::kPart + kk * 2048), idD, x > 0 || kk > 0);
            commit_if(leader, &bars[B_WFREE + hf]);
          }
          if (!ok) break;
          commit_if(leader, &bars[bar_d<STATES>(c)]);
        }
        commit_if(leader, &bars[B_QKFREE + s]);
        s = s + 1 == M::kStages ? 0 : s + 1;
        phase ^= s == 0;
      }
      commit_if(leader, &bars[B_DONE + 1]);
      ok = wait_all(&bars[B_DONE + 1], 0) && ok;
    }
  } else if (warp < kState) {
    // -------------------------------------------------------------------- P
    if (!STATES) {
      const int w = warp;
      const uint32_t lane_off = (uint32_t)(32 * w) << 16;
      const uint32_t tx = tmem + kColX + lane_off, tp = tmem + kColP + lane_off;
      // row i's decays: entry kFrom - i + j of the table for column j
      const int from = (back ? 31 : 127) - (32 * w + lane);
      const float* row = tab + (from & 3) * kCopy + (from & ~3);
      uint32_t pk[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) pk[j] = 0u;
      // blocks of 32 columns on the far side of the diagonal stay zero
      for (int blk = 0; blk < 4; ++blk)
        if (back ? blk < w : blk > w) tc::tmem_st16u(tp + 16 * blk, pk);
      const int first = back ? w : 0, last = back ? 3 : w;
      for (int c = 0; c < N; ++c) {
        const int n = tokens_of(c);
        if (!(ok = wait_all(&bars[B_X], c & 1))) break;
        tc::fence_after();
#pragma unroll 1
        for (int blk = first; blk <= last; ++blk) {
          float s[32];
          tc::tmem_ld32(tx + 32 * blk, s);
          tc::tmem_ld_wait();
          if (blk == last) {
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
              tc::mbar_arrive(&bars[B_XREAD]);
              if (ragged_at(c)) tc::mbar_arrive(&bars[B_RAGGED]);
            }
          }
#pragma unroll
          for (int j = 0; j < 32; j += 4) {
            const float4 f = *(const float4*)(row + 32 * blk + j);
            float p0, p1, p2, p3;
            tc::f2_unpack(tc::f2_mul(tc::f2_pack(s[j], s[j + 1]), tc::f2_pack(f.x, f.y)), p0, p1);
            tc::f2_unpack(tc::f2_mul(tc::f2_pack(s[j + 2], s[j + 3]), tc::f2_pack(f.z, f.w)), p2, p3);
            s[j] = p0, s[j + 1] = p1, s[j + 2] = p2, s[j + 3] = p3;
          }
          // (scores with tokens behind the end may be anything)
          if (32 * blk + 32 > n)
#pragma unroll
            for (int j = 0; j < 32; ++j) s[j] = 32 * blk + j < n ? s[j] : 0.f;
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[j] = tc::pack_bf16x2(s[2 * j], s[2 * j + 1]);
          if (blk == first && c > 0) {  // the last chunk's P has been used
            if (!(ok = wait_all(&bars[B_O], (c - 1) & 1))) break;
            tc::fence_after();
          }
          tc::tmem_st16u(tp + 16 * blk, pk);
        }
        if (!ok) break;
        tc::tmem_st_wait();
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive(&bars[B_P]);
      }
    }
  } else if (warp < kOut) {
    // ---------------------------------------------------------------- state
    registers_up<152>();
    const int w = warp - kState, r = 32 * w + lane;
    const uint32_t lane_off = (uint32_t)(32 * w) << 16;
    const bool has = 32 * w < D;
    float S[kWidth];
    // entry (r, column i) of a state is p[i * s_c]; as offsets of 32 bits from one address, which are less code than
    // an address each (prompt 121 -> 117 us, 131,072 tokens of 8 heads 356 -> 328)
    const auto column0 = [&](long long base, long long s_r, long long s_c) {
      return base + r * s_r + slice * kWidth * s_c;
    };
#pragma unroll
    for (int i = 0; i < kWidth; ++i) S[i] = 0.f;
    if (!STATES && has && (a.segs > 1 || op.s_in)) {
      const bool cut = a.segs > 1;
      const long long s_r = cut ? (op.part_t ? D : 1) : op.s_r, s_c = cut ? (op.part_t ? 1 : D) : op.s_c;
      const float* p = (cut ? op.part : op.s_in) + column0((cut ? (long long)bh * a.segs + seg : bh) * D * D, s_r, s_c);
#pragma unroll
      for (int i = 0; i < kWidth; ++i) S[i] = p[i * (int)s_c];
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
    for (int c = 0; c < updates; ++c) {
      const Carry carry(g, tokens_of(c));
      // the sum of the old state's part and dS's: gamma^n S first, while dS is on its way
      const uint64_t m2 = tc::f2_pack(carry.m, carry.m);
      if (carry.slow) {
#pragma unroll
        for (int i = 0; i < kWidth; i += 2) {
          const uint64_t s2 = tc::f2_pack(S[i], S[i + 1]);
          tc::f2_unpack(tc::f2_fma(s2, m2, s2), S[i], S[i + 1]);
        }
      } else {
#pragma unroll
        for (int i = 0; i < kWidth; i += 2)
          tc::f2_unpack(tc::f2_mul(tc::f2_pack(S[i], S[i + 1]), m2), S[i], S[i + 1]);
      }
      if (!(ok = wait_all(&bars[bar_d<STATES>(c)], STATES ? (c >> 1) & 1 : c & 1))) break;
      tc::fence_after();
#pragma unroll
      for (int o = 0; o < kWidth; o += 16) {
        float d[PARTS][16];
#pragma unroll
        for (int p = 0; p < PARTS; ++p) tc::tmem_ld16(tmem + col_d<STATES>(c) + 64 * p + o + lane_off, d[p]);
        tc::tmem_ld_wait();
        if (o + 16 == kWidth) {
          tc::fence_before();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&bars[bar_dread<STATES>(c)]);
        }
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          uint64_t x2 = tc::f2_pack(d[PARTS - 1][i], d[PARTS - 1][i + 1]);
#pragma unroll
          for (int p = PARTS - 2; p >= 0; --p) x2 = tc::f2_add(x2, tc::f2_pack(d[p][i], d[p][i + 1]));
          tc::f2_unpack(tc::f2_add(tc::f2_pack(S[o + i], S[o + i + 1]), x2), S[o + i], S[o + i + 1]);
        }
      }
      if (!STATES && c + 1 < N) {
        if (!(ok = wait_all(&bars[B_SREAD], c & 1))) break;
        publish();
      }
    }
    if (ok && has && (STATES || (op.s_out && last_seg))) {
      float* p = STATES ? op.part + column0(((long long)bh * a.segs + (back ? seg - 1 : seg + 1)) * D * D, 1, D)
                        : op.s_out + column0((long long)bh * D * D, op.s_r, op.s_c);
      const long long s_c = STATES ? D : op.s_c;
#pragma unroll
      for (int i = 0; i < kWidth; ++i) p[i * (int)s_c] = S[i];
    }
  } else if (warp < kW) {
    // --------------------------------------------------------------- output
    registers_down<72>();
    if (!STATES) {
      const int el = threadIdx.x - 32 * kOut, i = el;
      const uint32_t lane_off = (uint32_t)(el & 96) << 16;
      uint8_t* tile = smem + M::offO;
      const uint64_t sc2 = tc::f2_pack(a.scale, a.scale);
      const float read = op.scaled ? 1.f : a.scale;
      for (int c = 0; c < N; ++c) {
        const int n = tokens_of(c);
        const float wi = i < n ? pw(back ? n - 1 - i : i + 1) * read : 0.f;
        const uint64_t wi2 = tc::f2_pack(wi, wi);
        ok = wait_all(&bars[B_O], c & 1);
        if (el == 0) tc::bulk_wait_read_all();  // the last chunk's tile has left
        if (!(ok = tc::group_all(1, 128, ok))) break;
        tc::fence_after();
#pragma unroll
        for (int qt = 0; qt < 4; ++qt) {
          float oi[16], po[16];
          tc::tmem_ld16(tmem + kColOi + 16 * qt + lane_off, oi);
          tc::tmem_ld16(tmem + kColOp + 16 * qt + lane_off, po);
          tc::tmem_ld_wait();
          if (qt == 3) {
            tc::fence_before();
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&bars[B_OREAD]);
          }
          uint32_t o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            float x0, x1;
            tc::f2_unpack(tc::f2_fma(tc::f2_pack(oi[2 * j], oi[2 * j + 1]), wi2,
                                     tc::f2_mul(tc::f2_pack(po[2 * j], po[2 * j + 1]), sc2)),
                          x0, x1);
            o[j] = tc::pack_bf16x2(x0, x1);
          }
          if (i >= n)
#pragma unroll
            for (int j = 0; j < 8; ++j) o[j] = 0u;
#pragma unroll
          for (int gg = 0; gg < 2; ++gg)
            *(uint4*)(tile + piece(i, 2 * qt + gg)) = make_uint4(o[4 * gg], o[4 * gg + 1], o[4 * gg + 2], o[4 * gg + 3]);
        }
        tc::fence_proxy_async_smem();
        tc::named_barrier(1, 128);
        if (el == 0) {
          tma_store_4d(&maps.o, tile, kWidth * slice, t0 + chunk_at(c) * C, h, b);
          tc::bulk_commit();
        }
      }
      if (el == 0) tc::bulk_wait_all();
      // rows behind the sequence's end
      __nv_bfloat16* o = (__nv_bfloat16*)op.o.p + b * op.o.b + h * op.o.h + slice * kWidth;
      for (int e = el; e < (t1 - t0 - N * C) * (kWidth / 8); e += 128)
        *(uint4*)(o + (t0 + N * C + e / (kWidth / 8)) * op.o.t + (e % (kWidth / 8)) * 8) = make_uint4(0, 0, 0, 0);
    }
  } else {
    // ---------------------------------------- W V, a warpgroup to each half
    registers_down<64>();
    const int el = threadIdx.x - 32 * kW, hf = el >> 7, e0 = el & 127;
    // the weights of this thread's rows, 64 hf + 16 it + e0 / 8
    const float add = op.scaled ? a.scale : 1.f;
    const auto weight = [&](int it, int n) {
      const int j = 64 * hf + 16 * it + (e0 >> 3);
      return j < n ? pw(back ? j + 1 : n - 1 - j) * add : 0.f;
    };
    float w[4];
#pragma unroll
    for (int it = 0; it < 4; ++it) w[it] = weight(it, C);
    int s = 0, phase = 0;
    // The eight warps meet once, ahead of the ragged chunk, whether their waits have ended or not: one that leaves
    // the loop earlier is there too (behind it), so that the others' barrier ends.
    bool meets = ragged_c >= 0;
    for (int c = 0; c < N && ok; ++c) {
      const int n = tokens_of(c);
      uint8_t* kt = smem + s * M::kStage + M::kQ;
      uint8_t* vt = kt + M::kTile;
      ok = wait_all(&bars[B_V + s], phase) && !(c == a.expire && warp == kW);
      if (!ragged_at(c) && !ok) break;
      if (ragged_at(c)) {
        // tokens behind the end that the loads have brought along are taken out of K (once its scores have been
        // read) and V
        ok = ok && (STATES ? wait_all(&bars[B_QK + s], phase) : wait_all(&bars[B_RAGGED], 0));
        meets = false;
        if (!(ok = tc::group_all(2, 256, ok))) break;
        for (int e = el; e < (C - n) * 8; e += 256) {
          *(uint4*)(vt + (n + e / 8) * 128 + (e % 8) * 16) = make_uint4(0, 0, 0, 0);
          for (int y = 0; y < D / 64; ++y) *(uint4*)(kt + y * 16384 + (n + e / 8) * 128 + (e % 8) * 16) = make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async_smem();
        tc::named_barrier(2, 256);
        if (lane == 0) tc::mbar_arrive(&bars[B_CLEAN]);
      }
      if (c < updates) {
        uint8_t* dst = smem + M::offW + hf * PARTS * M::kPart;
        constexpr int kIts = M::kStep / 16;  // 16-byte pieces of a thread in a step
        if (n < C)
#pragma unroll
          for (int it = 0; it < 4; ++it) w[it] = weight(it, n);
#pragma unroll
        for (int q = 0; q < M::kSteps; ++q) {
          uint4 in[kIts];
#pragma unroll
          for (int it = 0; it < kIts; ++it) in[it] = *(const uint4*)(vt + piece(64 * hf + (q * kIts + it) * 16 + (e0 >> 3), e0 & 7));
          if ((c > 0 || q > 0) && !(ok = wait_all(&bars[B_WFREE + hf], (c * M::kSteps + q - 1) & 1))) break;
#pragma unroll
          for (int it = 0; it < kIts; ++it) {
            const float wj = w[q * kIts + it];
            const uint64_t w2 = tc::f2_pack(wj, wj);
            const uint32_t u[4] = {in[it].x, in[it].y, in[it].z, in[it].w};
            uint32_t p[PARTS][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              uint64_t x2 = tc::f2_mul(tc::f2_pack(lo16(u[e]), hi16(u[e])), w2);
#pragma unroll
              for (int y = 0; y < PARTS; ++y) {
                float x0, x1;
                tc::f2_unpack(x2, x0, x1);
                const uint32_t z = tc::pack_bf16x2(x0, x1);
                p[y][e] = z;
                if (y + 1 < PARTS) x2 = tc::f2_sub(x2, tc::f2_pack(lo16(z), hi16(z)));
              }
            }
#pragma unroll
            for (int y = 0; y < PARTS; ++y)
              *(uint4*)(dst + y * M::kPart + piece(it * 16 + (e0 >> 3), e0 & 7)) = make_uint4(p[y][0], p[y][1], p[y][2], p[y][3]);
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(&bars[B_W + hf]);
        }
        if (!ok) break;
        if (n < C)
#pragma unroll
          for (int it = 0; it < 4; ++it) w[it] = weight(it, C);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bars[B_VFREE + s]);
      s = s + 1 == M::kStages ? 0 : s + 1;
      phase ^= s == 0;
    }
    if (meets) tc::group_all(2, 256, false);
  }
  if (!ok && lane == 0) g_expired = 1;
  tc::fence_before();
  __syncthreads();
  if (warp == kMma) {
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

template <int D, bool STATES, int PARTS>
cudaError_t launch(const TcArgs& ta, cudaStream_t st) {
  auto kern = scan_tc_kernel<D, STATES, PARTS>;
  const int smem = Lay<D, STATES, PARTS>::kBytes;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const Args& a = ta.a;
  const long long grid = (long long)(a.last_op - a.first_op) * a.B * a.H * (D / kWidth) * (STATES ? a.segs - 1 : a.segs);
  return after(kern, (unsigned)grid, dim3(kThreads), smem, st, 0, ta);
}

}  // namespace

cudaError_t launch_tc(const Args& a, int d, bool states_only, cudaStream_t st) {
  TcArgs ta;
  ta.a = a;
  for (int i = a.first_op; i < a.last_op; ++i)
    if (!make_map(&ta.m[i].q, a.op[i].q, a, d) || !make_map(&ta.m[i].k, a.op[i].k, a, d) ||
        !make_map(&ta.m[i].v, a.op[i].v, a, d) || !make_map(&ta.m[i].o, a.op[i].o, a, d))
      return cudaErrorInvalidValue;
  // a state that is given out is as good as fp32 makes it; one that only meets the queries, in bf16, does with two parts
  bool out = false;
  for (int i = a.first_op; i < a.last_op; ++i) out = out || a.op[i].s_out;
  if (states_only && out) return d == 64 ? launch<64, true, 3>(ta, st) : launch<128, true, 3>(ta, st);
  if (states_only) return d == 64 ? launch<64, true, 2>(ta, st) : launch<128, true, 2>(ta, st);
  if (out) return d == 64 ? launch<64, false, 3>(ta, st) : launch<128, false, 3>(ta, st);
  return d == 64 ? launch<64, false, 2>(ta, st) : launch<128, false, 2>(ta, st);
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
