// paged_evict.cu - eviction from a paged key / value cache by accumulated
// attention weight (nats_paged_evict): every key head of a sequence with more
// than `budget` slots keeps the first `sinks`, the last `recent` and the
// budget - sinks - recent heaviest of those between (ties to the lower slot),
// and its kept rows go, in order, to fresh pages.
//
// Two kernels.  Selection, a CTA per (sequence, key head): the threshold is
// found exactly by a radix select on the weights' bits (four passes of eight
// bits over an order-preserving integer image of the float, each a histogram
// in shared memory), then one pass in slot order writes the kept slots'
// indexes, ranks taken by ballots and a scan over the CTA's warps.  The copy,
// a CTA per 64 kept rows of a head, moves them with 16-byte accesses.  The
// copy is the floor: a kept row is read once and written once.
#include "kernels.h"
#include "paged.cuh"

namespace nats {
namespace {

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
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

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(EvictArgs a) {
  __shared__ int hist[256], scan[2][kSelWarps];
  __shared__ int pick[2];
  const int b = blockIdx.x / a.pg.Hk, h = blockIdx.x % a.pg.Hk;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n = a.pg.length(b);
  int32_t* keep = a.keep + (long long)blockIdx.x * a.budget;
  const int left = min(n, a.budget);
  if (tid == 0) {
    if (h == 0) a.lens_out[b] = left;
    if (a.pg.lens[b] != n) *a.pg.err = 1;
  }
  for (int i = left + tid; i < a.budget; i += kSelThreads) keep[i] = -1;
  if (n <= a.budget) {
    for (int i = tid; i < n; i += kSelThreads) keep[i] = i;
    return;
  }
  // the candidates are the slots m0 <= j < m1, of which `need` stay
  const int m0 = a.sinks, m1 = n - a.recent, need = a.budget - a.sinks - a.recent;
  uint32_t prefix = 0, mask = 0;
  int rest = need;  // of the candidates that share the prefix, how many stay
  if (need > 0) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      for (int i = tid; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int j = m0 + tid; j < m1; j += kSelThreads) {
        const uint32_t u = slot_bits(a, b, h, j);
        if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & 255], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int above = 0, d = 255;
        while (d > 0 && above + hist[d] < rest) above += hist[d--];
        pick[0] = d, pick[1] = rest - above;
      }
      __syncthreads();
      prefix |= (uint32_t)pick[0] << shift;
      mask |= 255u << shift;
      rest = pick[1];
    }
  }
  // threshold `prefix`: heavier candidates stay, and the first `rest` equal ones
  int kept0 = 0, ties0 = 0;
  for (int j0 = 0; j0 < n; j0 += kSelThreads) {
    const int j = j0 + tid;
    bool sure = j < n && (j < m0 || j >= m1), tie = false;
    if (need > 0 && j >= m0 && j < m1) {
      const uint32_t u = slot_bits(a, b, h, j);
      sure = u > prefix;
      tie = u == prefix;
    }
    const uint32_t bt = __ballot_sync(0xffffffffu, tie);
    if (lane == 0) scan[0][warp] = __popc(bt);
    __syncthreads();
    int before = ties0, ties = 0;
    for (int w = 0; w < kSelWarps; ++w) {
      if (w < warp) before += scan[0][w];
      ties += scan[0][w];
    }
    const uint32_t lower = (1u << lane) - 1;
    const bool stays = sure || (tie && before + __popc(bt & lower) < rest);
    const uint32_t bk = __ballot_sync(0xffffffffu, stays);
    if (lane == 0) scan[1][warp] = __popc(bk);
    __syncthreads();
    int at = kept0, kept = 0;
    for (int w = 0; w < kSelWarps; ++w) {
      if (w < warp) at += scan[1][w];
      kept += scan[1][w];
    }
    if (stays) keep[at + __popc(bk & lower)] = j;
    kept0 += kept;
    ties0 += ties;
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
  evict_select_kernel<<<(unsigned)(cache->B * cache->Hk), kSelThreads, 0, st>>>(a);
  const int r = record_cuda_error(cudaGetLastError());
  if (r != NATS_OK || budget == 0) return (nats_status)r;
  const int tiles = (budget + kCopyRows - 1) / kCopyRows;
  evict_copy_kernel<<<(unsigned)((long long)cache->B * cache->Hk * tiles), kCopyThreads, 0, st>>>(a, tiles);
  return (nats_status)record_cuda_error(cudaGetLastError());
}

}  // extern "C"
