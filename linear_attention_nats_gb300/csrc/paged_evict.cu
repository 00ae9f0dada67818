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
#include <cooperative_groups.h>

#include "kernels.h"
#include "paged.cuh"

namespace nats {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;            // two a thread
constexpr int kKeysHeld = 32768;       // slots of a CTA's share in shared memory; a longer share is read again
constexpr int kSMs = 152;
constexpr int kMaxCluster = 8;
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

// The weight's image of slot j (a slot without a page counts as the lowest).
__device__ __forceinline__ uint32_t slot_bits(const EvictArgs& a, int b, int h, int j) {
  const int pg = a.pg.page_of(b, j / a.pg.page);
  return pg < 0 ? order_bits(-INFINITY) : order_bits(a.weight[a.pg.row(pg, h, j % a.pg.page)]);
}

// Inclusive sum over the CTA's threads in thread order; *total gets all of it.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int w = warp_sums[lane];
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

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a, int held) {
  namespace cg = cooperative_groups;
  extern __shared__ uint32_t keys[];  // the share's first `held` weights, as order_bits
  __shared__ int hist[3][kBins];
  __shared__ int sums[kSelWarps], pick[2], counts[2];
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
    return;
  }
  // the candidates are the slots m0 <= j < m1, of which `need` stay
  const int m0 = a.sinks, m1 = n - a.recent, need = a.budget - a.sinks - a.recent;
  // this CTA's share and, of it, this warp's run: contiguous, whole warps wide
  const int run = (n + C * kSelThreads - 1) / (C * kSelThreads) * 32;
  const int s0 = min((long long)n, (long long)rank * run * kSelWarps), w0 = s0 + warp * run;
  const int w1 = min(n, w0 + run);
  for (int i = tid; i < 3 * kBins; i += kSelThreads) (&hist[0][0])[i] = 0;
  __syncthreads();
  auto key = [&](int j) { return j - s0 < held ? keys[j - s0] : slot_bits(a, b, h, j); };
  uint32_t prefix = 0, mask = 0;
  int rest = need;  // of the candidates that share the prefix, how many stay
  if (need > 0) {
#pragma unroll 4
    for (int j = w0 + lane; j < w1; j += 32) {
      const uint32_t u = slot_bits(a, b, h, j);
      if (j - s0 < held) keys[j - s0] = u;
      if (j >= m0 && j < m1) atomicAdd(&hist[0][u >> 21], 1);
    }
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : kBins;
      if (pass > 0)
        for (int j = w0 + lane; j < w1; j += 32) {
          const uint32_t u = key(j);
          if (j >= m0 && j < m1 && (u & mask) == prefix) atomicAdd(&hist[pass][(u >> shift) & (bins - 1)], 1);
        }
      cluster.sync();
      // bins from the top, two a thread, summed over the cluster
      int hi = 0, lo = 0;
      const int top = bins - 1 - 2 * tid;
      if (top > 0)
        for (int r = 0; r < C; ++r) {
          const int2 v = *(const int2*)cluster.map_shared_rank(&hist[pass][top - 1], r);
          hi += v.y, lo += v.x;
        }
      int total;
      const int upto = block_scan(hi + lo, sums, &total);
      const int before = upto - hi - lo;
      if (before < rest && rest <= upto) {
        const bool in_hi = rest <= before + hi;
        pick[0] = in_hi ? top : top - 1;
        pick[1] = rest - (in_hi ? before : before + hi);
      }
      __syncthreads();
      prefix |= (uint32_t)pick[0] << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      rest = pick[1];
    }
  }
  // threshold `prefix`: heavier candidates stay, and the first `rest` equal ones
  auto look = [&](int j, bool& sure, bool& tie) {
    sure = j < w1 && (j < m0 || j >= m1), tie = false;
    if (need > 0 && j < w1 && j >= m0 && j < m1) {
      const uint32_t u = key(j);
      sure = u > prefix, tie = u == prefix;
    }
  };
  int nsure = 0, ntie = 0;
  for (int j = w0 + lane; j - lane < w1; j += 32) {
    bool sure, tie;
    look(j, sure, tie);
    nsure += __popc(__ballot_sync(0xffffffffu, sure));
    ntie += __popc(__ballot_sync(0xffffffffu, tie));
  }
  int total_sure, total_tie;
  const int sure_upto = block_scan(lane == 0 ? nsure : 0, sums, &total_sure);
  const int tie_upto = block_scan(lane == 0 ? ntie : 0, sums, &total_tie);
  if (tid == 0) counts[0] = total_sure, counts[1] = total_tie;
  cluster.sync();
  int sure0 = __shfl_sync(0xffffffffu, sure_upto, 0) - nsure, tie0 = __shfl_sync(0xffffffffu, tie_upto, 0) - ntie;
  for (int r = 0; r < rank; ++r) {
    const int* c = cluster.map_shared_rank(counts, r);
    sure0 += c[0], tie0 += c[1];
  }
  cluster.sync();  // no CTA leaves while another reads its counts
  const uint32_t lower = (1u << lane) - 1;
  for (int j = w0 + lane; j - lane < w1; j += 32) {
    bool sure, tie;
    look(j, sure, tie);
    const uint32_t bs = __ballot_sync(0xffffffffu, sure), bt = __ballot_sync(0xffffffffu, tie);
    // kept before slot j: the sure ones, and of the ties before it the first `rest`
    const int ties = tie0 + __popc(bt & lower);
    const int at = sure0 + __popc(bs & lower) + min(ties, rest);
    if (sure || (tie && ties < rest)) keep[at] = j;
    sure0 += __popc(bs);
    tie0 += __popc(bt);
  }
}

// Kept rows i0 .. i0 + 63 of one head: keys, values and weights.
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(EvictArgs a, int tiles) {
  __shared__ long long from[kCopyRows], to[kCopyRows];
  const int bh = blockIdx.x / tiles, i0 = (blockIdx.x % tiles) * kCopyRows;
  const int b = bh / a.pg.Hk, h = bh % a.pg.Hk;
  const int left = min(a.pg.length(b), a.budget);
  if (i0 >= left) return;
  const int rows = min(kCopyRows, left - i0);
  const int tid = threadIdx.x;
  if (tid < rows) {
    const int i = i0 + tid, j = a.keep[(long long)bh * a.budget + i];
    const int pf = a.pg.page_of(b, j / a.pg.page);
    const int pt = a.out_table[(long long)b * a.out_pages + i / a.pg.page];
    const bool ok = pf >= 0 && (unsigned)pt < (unsigned)a.pg.n_pages;
    from[tid] = ok ? a.pg.row(pf, h, j % a.pg.page) : -1;
    to[tid] = ok ? a.pg.row(pt, h, i % a.pg.page) : -1;
    if (ok)
      a.weight[to[tid]] = a.weight[from[tid]];
    else
      *a.pg.err = 1;
  }
  __syncthreads();
  const int per = a.row_bytes / 16, total = rows * per;
#pragma unroll 4
  for (int x = tid; x < total; x += kCopyThreads) {
    const int r = x / per, c = x % per;
    if (from[r] < 0) continue;
    const long long f = from[r] * a.row_bytes + c * 16, t = to[r] * a.row_bytes + c * 16;
    const uint4 kk = *(const uint4*)(a.k + f), vv = *(const uint4*)(a.v + f);
    *(uint4*)(a.k + t) = kk;
    *(uint4*)(a.v + t) = vv;
  }
}

// CTAs of a head: as many as fill the GPU, while a share is worth its part of
// the cluster's barriers (4096 slots).
cudaError_t launch_select(const EvictArgs& a, long long cap, cudaStream_t st) {
  const long long heads = (long long)a.pg.B * a.pg.Hk;
  int C = 1;
  while (C < kMaxCluster && heads * C < kSMs && cap / (2 * C) >= 4096) C *= 2;
  const long long share = (cap + C * kSelThreads - 1) / (C * kSelThreads) * kSelThreads;
  const int held = (int)(share < kKeysHeld ? share : kKeysHeld);
  if (held * 4 > 16384) {  // beyond what a kernel has without asking
    const cudaError_t e =
        cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kKeysHeld * 4);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(heads * C));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = (size_t)held * 4;
  cfg.stream = st;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim = {(unsigned)C, 1, 1};
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel, a, held);
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
  if (!lens_out || !workspace || (budget > 0 && (!out_table || (cache->n_pages > 0 && !cache->weight)))) return NATS_ERR_NULL;
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
  const int r = record_cuda_error(launch_select(a, (long long)cache->max_pages * cache->page, st));
  if (r != NATS_OK || budget == 0) return (nats_status)r;
  const int tiles = (budget + kCopyRows - 1) / kCopyRows;
  evict_copy_kernel<<<(unsigned)((long long)cache->B * cache->Hk * tiles), kCopyThreads, 0, st>>>(a, tiles);
  return (nats_status)record_cuda_error(cudaGetLastError());
}

}  // extern "C"
