// paged_evict.cu - eviction from a paged key / value cache by accumulated
// attention weight (nats_paged_evict): every key head of a sequence with more
// than `budget` slots keeps the first `sinks`, the last `recent` and the
// budget - sinks - recent heaviest of those between (ties to the lower slot),
// and its kept rows go, in order, to fresh pages.
//
// Two kernels.  Selection, a cluster of CTAs per (sequence, key head), each
// with a contiguous share of the slots: the weights are read once, as
// order-preserving integers, into shared memory; the threshold is found
// exactly by a radix select over their bits (11, 11 and 10 of them, a
// histogram in every CTA's shared memory, summed over the cluster through
// distributed shared memory), then the kept slots' indexes are written in
// order, each warp counting its own run of slots first so that the places
// follow from one scan.  The copy, a CTA per 64 kept rows of a head, moves them with 16-byte
// accesses and is the floor: a kept row is read once and written once.
// Measured on one GB300: 32 x 8 heads from 2112 to 2048 slots of 128 bf16
// entries 72 us, of which the copy 57 (6.8 TB/s, the HBM copy rate); 4 x 8 heads
// from up to 131,072 to 32,768 slots 193 us, the copy 162.  Requesting rows to
// L2, or copying recent ones, beside the selection gained nothing (72 us to 74,
// and 72 to 72): what the copy then reads earlier it writes no faster.
#include <cooperative_groups.h>

#include "kernels.h"
#include "launch.cuh"
#include "paged.cuh"

namespace nats {
namespace {

constexpr int kBins = 2048;
constexpr int kKeysHeld = 32768;       // slots of a CTA's share in shared memory; a longer share is read again
constexpr int kSMs = 152;
constexpr int kMaxCluster = 8;
constexpr int kFusedRows = 512, kFusedBytes = 65536;  // of a head's keys that the selecting CTA copies itself (launch_select)
constexpr int kShortShare = 8192, kShortThreads = 512;  // slots of a share, threads of its CTA
constexpr int kCopyRows = 64;
constexpr int kCopyThreads = 256;

struct EvictArgs {
  PagedView pg;
  char *k, *v;
  float* weight;
  const int32_t* out_table;
  int out_pages;
  int budget, recent, sinks;
  int32_t* lens_out;
  int32_t* keep;  // [B, Hk, budget] (the caller's, or scratch)
  int row_bytes;
};

// An integer that orders as the weight does; NaN as -inf, -0 as +0.
__device__ __forceinline__ uint32_t order_bits(float w) {
  if (!(w == w)) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Inclusive sum over the CTA's threads in thread order; *total gets all of it.
template <int WARPS>
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int w = lane < WARPS ? warp_sums[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += y;
  }
  const int before = __shfl_sync(0xffffffffu, w, warp) - __shfl_sync(0xffffffffu, warp_sums[warp], 0);
  *total = __shfl_sync(0xffffffffu, w, 31);
  __syncthreads();
  return x + before;
}

// One warp: of 32 PER counts in every CTA of the cluster, summed over them, the
// index of the one that holds the rest-th from the top; *above, the sum of those above it.
template <int PER>
__device__ __forceinline__ int find_from_top(cooperative_groups::cluster_group& cluster, int* counts, int C, int rest,
                                             int* above) {
  const int lane = threadIdx.x & 31;
  int v[PER] = {};  // from the top: lane 0 has the highest
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r)
    if (r < C) {
      const int* c = cluster.map_shared_rank(counts, r) + 32 * PER - 1 - PER * lane;
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] += c[-i];
    }
  int mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) mine += v[i];
  int upto = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, upto, o);
    if (lane >= o) upto += y;
  }
  int before = upto - mine, at = 32 * PER - 1 - PER * lane;
  const bool here = before < rest && rest <= upto;
  if (PER == 2 && here && rest > before + v[0]) before += v[0], --at;
  const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  *above = __shfl_sync(0xffffffffu, before, src);
  return __shfl_sync(0xffffffffu, at, src);
}

// Rows i0 .. i0 + rows - 1 kept of one head, slot src[i - i0] each: keys, values
// and weights.  from, to: shared memory for `rows` of them.
template <int THREADS>
__device__ __forceinline__ void copy_rows(const EvictArgs& a, int b, int h, int i0, int rows, const int32_t* src,
                                          long long* from, long long* to) {
  const int tid = threadIdx.x;
  for (int i = tid; i < rows; i += THREADS) {
    const int j = src[i], k = i0 + i;
    const int pf = a.pg.page_of(b, j / a.pg.page);
    const int pt = a.out_table[(long long)b * a.out_pages + k / a.pg.page];
    const bool ok = pf >= 0 && (unsigned)pt < (unsigned)a.pg.n_pages;
    from[i] = ok ? a.pg.row(pf, h, j % a.pg.page) : -1;
    to[i] = ok ? a.pg.row(pt, h, k % a.pg.page) : -1;
    if (ok)
      a.weight[to[i]] = a.weight[from[i]];
    else
      *a.pg.err = 1;
  }
  __syncthreads();
  const int per = a.row_bytes / 16, total = rows * per;
#pragma unroll 4
  for (int x = tid; x < total; x += THREADS) {
    const int r = x / per, c = x % per;
    if (from[r] < 0) continue;
    const long long f = from[r] * a.row_bytes + c * 16, t = to[r] * a.row_bytes + c * 16;
    const uint4 kk = *(const uint4*)(a.k + f), vv = *(const uint4*)(a.v + f);
    *(uint4*)(a.k + t) = kk;
    *(uint4*)(a.v + t) = vv;
  }
}

// COPY (one CTA a head, a small budget): it also copies the head's rows, and no
// second kernel follows.
template <int THREADS, bool COPY>
__global__ void __launch_bounds__(THREADS, 2048 / THREADS) evict_select_kernel(EvictArgs a, int held) {
  namespace cg = cooperative_groups;
  constexpr int kSelThreads = THREADS, kSelWarps = THREADS / 32;
  begin();
  extern __shared__ uint32_t keys[];  // the share's first `held` weights, as order_bits
  __shared__ int hist[3][kBins], groups[3][kBins / 32];
  __shared__ int sums[kSelWarps], pick[2], counts[2];
  __shared__ long long from[COPY ? kFusedRows : 1], to[COPY ? kFusedRows : 1];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int bh = blockIdx.x / C, b = bh / a.pg.Hk, h = bh % a.pg.Hk;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.pg.length(b);
  int32_t* keep = a.keep + (long long)bh * a.budget;
  const int left = min(n, a.budget);
  if (tid == 0 && rank == 0) {
    if (h == 0) a.lens_out[b] = left;
    if (a.pg.lens[b] != n) *a.pg.err = 1;
  }
  for (int i = left + rank * kSelThreads + tid; i < a.budget; i += C * kSelThreads) keep[i] = -1;
  if (n <= a.budget) {  // (the whole cluster)
    for (int i = rank * kSelThreads + tid; i < n; i += C * kSelThreads) keep[i] = i;
    if constexpr (COPY) {
      __syncthreads();
      copy_rows<THREADS>(a, b, h, 0, n, keep, from, to);
    }
    return;
  }
  // the candidates are the slots m0 <= j < m1, of which `need` stay; the others
  // stay whatever they weigh: their image is above every weight's
  const int m0 = a.sinks, m1 = n - a.recent, need = a.budget - a.sinks - a.recent;
  constexpr uint32_t kAlways = 0xffffffffu;
  // this CTA's share and, of it, this warp's run: contiguous, 128 slots or a multiple
  const int run = (n + C * kSelWarps * 128 - 1) / (C * kSelWarps * 128) * 128;
  const int s0 = min((long long)n, (long long)rank * run * kSelWarps);
  const int w0 = min((long long)n, s0 + (long long)warp * run), w1 = min(n, w0 + run);
  const bool counted = C == 1 && n <= THREADS;  // ranked by counting: no histogram
  if (!counted) {
    for (int i = tid; i < 3 * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
    __syncthreads();
  }
  // the images of slots j .. j + 3 (j a multiple of 4, so of one page); 0, below
  // every weight's, behind the last
  auto image4 = [&](int j) {
    const int pg = a.pg.page_of(b, j / a.pg.page);
    const float4 w = pg < 0 ? make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY)  // no page: the lowest
                            : *(const float4*)(a.weight + a.pg.row(pg, h, j % a.pg.page));
    uint32_t u[4] = {order_bits(w.x), order_bits(w.y), order_bits(w.z), order_bits(w.w)};
    if (j < m0 || j + 3 >= m1) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (j + i < m0 || j + i >= m1) u[i] = j + i < n ? kAlways : 0;
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  };
  auto key4 = [&](int j) { return j - s0 < held ? *(const uint4*)(keys + (j - s0)) : image4(j); };
  if (counted) {
    // a slot a thread: it stays if fewer than `budget` are heavier or, as heavy, before it
    for (int j = 4 * tid; j < n; j += 4 * THREADS) *(uint4*)(keys + j) = image4(j);
    __syncthreads();
    bool stays = false;
    if (tid < n) {
      const uint32_t mine = keys[tid];
      const int own = tid & ~3;
      int ahead = 0;
      for (int j = 0; j < own; j += 4) {
        const uint4 u = *(const uint4*)(keys + j);
        ahead += (u.x >= mine) + (u.y >= mine) + (u.z >= mine) + (u.w >= mine);
      }
      for (int j = own; j < own + 4; ++j) ahead += j < tid ? keys[j] >= mine : keys[j] > mine;
      for (int j = own + 4; j < n; j += 4) {
        const uint4 u = *(const uint4*)(keys + j);
        ahead += (u.x > mine) + (u.y > mine) + (u.z > mine) + (u.w > mine);
      }
      stays = ahead < a.budget;
    }
    int total;
    const int upto = block_scan<kSelWarps>(stays, sums, &total);
    if (stays) keep[upto - 1] = tid;
    if constexpr (COPY) {
      __syncthreads();
      copy_rows<THREADS>(a, b, h, 0, a.budget, keep, from, to);
    }
    return;
  }
  {
#pragma unroll 2
    for (int j = w0 + 4 * lane; j < w1; j += 128) {
      const uint4 u = image4(j);
      if (j - s0 < held) *(uint4*)(keys + (j - s0)) = u;  // (held is a multiple of 4)
      if (need > 0) {
        if (u.x + 1 > 1) atomicAdd(&hist[0][u.x >> 21], 1);  // neither 0 nor kAlways
        if (u.y + 1 > 1) atomicAdd(&hist[0][u.y >> 21], 1);
        if (u.z + 1 > 1) atomicAdd(&hist[0][u.z >> 21], 1);
        if (u.w + 1 > 1) atomicAdd(&hist[0][u.w >> 21], 1);
      }
    }
    __syncwarp();
  }
  uint32_t prefix = need > 0 ? 0 : kAlways - 1, mask = 0;  // no candidate stays: only kAlways is above
  int rest = need;  // of the candidates that share the prefix, how many stay
  if (need > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
      if (pass > 0)
        for (int j = w0 + 4 * lane; j < w1; j += 128) {
          const uint4 u = key4(j);
          // (kAlways, should the prefix be its own, is no weight; the prefix is never 0's)
          if ((u.x & mask) == prefix && u.x != kAlways) atomicAdd(&hist[pass][(u.x >> shift) & (bins - 1)], 1);
          if ((u.y & mask) == prefix && u.y != kAlways) atomicAdd(&hist[pass][(u.y >> shift) & (bins - 1)], 1);
          if ((u.z & mask) == prefix && u.z != kAlways) atomicAdd(&hist[pass][(u.z >> shift) & (bins - 1)], 1);
          if ((u.w & mask) == prefix && u.w != kAlways) atomicAdd(&hist[pass][(u.w >> shift) & (bins - 1)], 1);
        }
      // sums of 32 bins each, so that the search reads little of the other CTAs
      __syncthreads();
#pragma unroll
      for (int i = warp; i < kBins / 32; i += kSelWarps) {
        const int sum = __reduce_add_sync(0xffffffffu, hist[pass][32 * i + lane]);
        if (lane == 0) groups[pass][i] = sum;
      }
      cluster.sync();
      if (warp == 0) {
        // the group from the top in which the rest-th lies, then the bin within it
        int above, more;
        const int gr = find_from_top<2>(cluster, groups[pass], C, rest, &above);
        const int bin = find_from_top<1>(cluster, hist[pass] + 32 * gr, C, rest - above, &more);
        if (lane == 0) pick[0] = 32 * gr + bin, pick[1] = rest - above - more;
      }
      __syncthreads();
      prefix |= (uint32_t)pick[0] << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      rest = pick[1];
    }
  }
  // threshold `prefix`: heavier slots stay, and the first `rest` equal ones
  int nsure = 0, ntie = 0;
  for (int j = w0 + 4 * lane; j < w1; j += 128) {
    const uint4 u = key4(j);
    nsure += (u.x > prefix) + (u.y > prefix) + (u.z > prefix) + (u.w > prefix);
    ntie += (u.x == prefix) + (u.y == prefix) + (u.z == prefix) + (u.w == prefix);
  }
  nsure = __reduce_add_sync(0xffffffffu, nsure), ntie = __reduce_add_sync(0xffffffffu, ntie);
  int total_sure, total_tie;
  const int sure_upto = block_scan<kSelWarps>(lane == 0 ? nsure : 0, sums, &total_sure);
  const int tie_upto = block_scan<kSelWarps>(lane == 0 ? ntie : 0, sums, &total_tie);
  if (tid == 0) counts[0] = total_sure, counts[1] = total_tie;
  cluster.sync();
  int sure0 = __shfl_sync(0xffffffffu, sure_upto, 0) - nsure, tie0 = __shfl_sync(0xffffffffu, tie_upto, 0) - ntie;
#pragma unroll
  for (int r = 0; r < kMaxCluster - 1; ++r)
    if (r < rank) {
      const int* c = cluster.map_shared_rank(counts, r);
      sure0 += c[0], tie0 += c[1];
    }
  cluster.sync();  // no CTA leaves while another reads its counts
  for (int j0 = w0; j0 < w1; j0 += 128) {
    const int j = j0 + 4 * lane;
    uint4 u = make_uint4(0, 0, 0, 0);
    if (j < w1) u = key4(j);
    // sure ones (upper half) and ties (lower half) before this lane's four slots
    uint32_t mine = (u.x > prefix) + (u.y > prefix) + (u.z > prefix) + (u.w > prefix);
    mine = mine << 16 | ((u.x == prefix) + (u.y == prefix) + (u.z == prefix) + (u.w == prefix));
    uint32_t upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += y;
    }
    int sure = sure0 + (int)((upto - mine) >> 16), ties = tie0 + (int)((upto - mine) & 0xffff);
    const uint32_t all = __shfl_sync(0xffffffffu, upto, 31);
    const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // kept before slot j + i: the sure ones, and of the ties the first `rest`
      const int at = sure + min(ties, rest);
      if (v[i] > prefix) keep[at] = j + i, ++sure;
      if (v[i] == prefix) {
        if (ties < rest) keep[at] = j + i;
        ++ties;
      }
    }
    sure0 += all >> 16;
    tie0 += all & 0xffff;
  }
  if constexpr (COPY) {
    __syncthreads();
    copy_rows<THREADS>(a, b, h, 0, a.budget, keep, from, to);
  }
}

// Kept rows i0 .. i0 + 63 of one head.
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(EvictArgs a, int tiles) {
  __shared__ long long from[kCopyRows], to[kCopyRows];
  begin();
  const int bh = blockIdx.x / tiles, i0 = (blockIdx.x % tiles) * kCopyRows;
  const int b = bh / a.pg.Hk, h = bh % a.pg.Hk;
  const int left = min(a.pg.length(b), a.budget);
  if (i0 >= left) return;
  copy_rows<kCopyThreads>(a, b, h, i0, min(kCopyRows, left - i0), a.keep + (long long)bh * a.budget + i0, from, to);
}

template <int THREADS, bool COPY>
cudaError_t launch_select(const EvictArgs& a, long long cap, int C, cudaStream_t st) {
  const long long warps = C * THREADS / 32, share = (cap + warps * 128 - 1) / (warps * 128) * 128 * (THREADS / 32);
  const int held = (int)(share < kKeysHeld ? share : kKeysHeld);
  auto kernel = evict_select_kernel<THREADS, COPY>;
  if (held * 4 > 8192) {  // beyond what a kernel has without asking
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysHeld * 4);
    if (e != cudaSuccess) return e;
  }
  return after(kernel, (unsigned)((long long)a.pg.B * a.pg.Hk * C), THREADS, (size_t)held * 4, st, C, a, held);
}

// CTAs of a head: as many as fill the GPU, while a share is worth its part of
// the cluster's barriers (2048 slots: 16 heads of 9199 34 us, 41 with shares of
// 4096; with 1024 32 heads of 5000 29 us, 25 with 2048; clusters of 16 gain
// only past 8 x 32768 slots, 66 to 40 us for 2 heads of 400,000, and cost the
// others 2 us).  Short shares by small CTAs, since a warp's fixed steps
// (barriers, scans) then outweigh its slots': 64 x 8 heads of 1000 slots 55.6
// us with 512 threads, 64.0 with 1024 (and the copy apart); long ones by large CTAs: one head
// of 131,072 34.5 us with 1024, 37.5 with 512.  *copied: the kernel copies too,
// which pays while a CTA's rows are few, more of them where every SM has CTAs
// that select while others copy (64 x 16 heads of 700 slots to 400: 75 us, 90
// with the copy apart; but 32 x 8 of 2112 to 2048, 91 against 72).  Lengths are on
// the device: all of this goes by the table's capacity, and short sequences in
// long tables are evicted by what suits the longest (64 x 8 heads of 1000 slots
// to 900: 86 us, in tables of 131,072 slots 157).
cudaError_t launch_select(const EvictArgs& a, long long cap, bool* copied, cudaStream_t st) {
  const long long heads = (long long)a.pg.B * a.pg.Hk;
  int C = 1;
  while (C < kMaxCluster && heads * C < kSMs && cap / (2 * C) >= 2048) C *= 2;
  *copied = C == 1 && a.budget <= kFusedRows &&
            (heads >= 2 * kSMs || (long long)a.budget * a.row_bytes <= kFusedBytes);
  if (cap / C > kShortShare) {
    *copied = false;
    return launch_select<1024, false>(a, cap, C, st);
  }
  return *copied ? launch_select<kShortThreads, true>(a, cap, C, st) : launch_select<kShortThreads, false>(a, cap, C, st);
}

nats_status check_evict(const nats_paged_cache* c, int32_t budget) {
  const nats_status s = check_cache(c);
  if (s != NATS_OK) return s;
  if (budget < 0) return NATS_ERR_SHAPE;
  if ((double)c->B * c->Hk * ((budget + kCopyRows - 1.0) / kCopyRows) > 2147483647.0) return NATS_ERR_UNSUPPORTED;
  return NATS_OK;
}

}  // namespace
}  // namespace nats

using namespace nats;

extern "C" {

size_t nats_paged_evict_workspace_size(const nats_paged_cache* cache, int32_t budget) {
  if (check_evict(cache, budget) != NATS_OK) return 0;
  return 4 * (size_t)cache->B * cache->Hk * budget + 16;
}

nats_status nats_paged_evict(const nats_paged_cache* cache, const int32_t* out_table, int32_t out_max_pages,
                             int32_t budget, int32_t recent, int32_t sinks, int32_t* lens_out, int32_t* keep,
                             void* workspace, size_t workspace_bytes, nats_stream_t stream) {
  nats_status s = check_evict(cache, budget);
  if (s != NATS_OK) return s;
  if (out_max_pages < 0 || (long long)out_max_pages * cache->page < budget) return NATS_ERR_SHAPE;
  if (recent < 0 || sinks < 0 || (long long)recent + sinks > budget) return NATS_ERR_VALUE;
  if (cache->B == 0) return NATS_OK;
  s = check_cache_pointers(cache);
  if (s != NATS_OK) return s;
  if (!lens_out || !workspace || (budget > 0 && !out_table) || (cache->n_pages > 0 && !cache->weight)) return NATS_ERR_NULL;
  if ((out_table && out_table == cache->table) || lens_out == cache->lens) return NATS_ERR_VALUE;
  if (((uintptr_t)workspace & 15u) || (((uintptr_t)out_table | (uintptr_t)lens_out | (uintptr_t)keep) & 3u))
    return NATS_ERR_ALIGN;
  if (workspace_bytes < nats_paged_evict_workspace_size(cache, budget)) return NATS_ERR_WORKSPACE;
  EvictArgs a = {};
  a.pg = view_of(cache), a.k = (char*)cache->k_pages, a.v = (char*)cache->v_pages, a.weight = cache->weight;
  a.out_table = out_table, a.out_pages = out_max_pages;
  a.budget = budget, a.recent = recent, a.sinks = sinks;
  a.lens_out = lens_out, a.keep = keep ? keep : (int32_t*)workspace;
  a.row_bytes = cache->d * (cache->dtype == NATS_BF16 ? 2 : 4);
  cudaStream_t st = (cudaStream_t)stream;
  bool copied = false;
  const int r = record_cuda_error(launch_select(a, (long long)cache->max_pages * cache->page, &copied, st));
  if (r != NATS_OK || budget == 0 || copied) return (nats_status)r;
  const int tiles = (budget + kCopyRows - 1) / kCopyRows;
  return (nats_status)record_cuda_error(after(
      evict_copy_kernel, (unsigned)((long long)cache->B * cache->Hk * tiles), kCopyThreads, 0, st, 0, a, tiles));
}

}  // extern "C"
