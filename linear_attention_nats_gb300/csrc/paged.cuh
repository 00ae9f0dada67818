// paged.cuh - the paged key / value cache as its kernels see it, and the
// checks of its fields that the entry points share.
#pragma once

#include <stdint.h>

#include "../../include/nats.h"
#include "common.cuh"

namespace nats {

// Row j of sequence b and key head h lies at row (page * Hk + h) * page_size +
// j % page_size of the pools; 64-bit, a pool may hold more than 2^31 entries.
struct PagedView {
  const int32_t* table;
  const int32_t* lens;
  int32_t* err;
  int n_pages, page, Hk, B, max_pages;

  __host__ __device__ __forceinline__ int cap() const { return max_pages * page; }
  // lens[b] brought into 0 .. cap
  __device__ __forceinline__ int length(int b) const { return min(max(lens[b], 0), cap()); }
  // the page of slot block `i` of sequence b, or -1 when the entry is not one
  // of the pool's
  __device__ __forceinline__ int page_of(int b, int i) const {
    const int pg = table[(long long)b * max_pages + i];
    return (unsigned)pg < (unsigned)n_pages ? pg : -1;
  }
  __device__ __forceinline__ long long row(int pg, int h, int slot) const {
    return ((long long)pg * Hk + h) * page + slot;
  }
};

inline PagedView view_of(const nats_paged_cache* c) {
  return PagedView{c->table, c->lens, c->err, c->n_pages, c->page, c->Hk, c->B, c->max_pages};
}

// Fields of the cache (api part of nats_paged_*): extents first, so that an
// empty cache passes with its pointers unset.
inline nats_status check_cache(const nats_paged_cache* c) {
  if (!c) return NATS_ERR_NULL;
  if (c->dtype != NATS_BF16 && c->dtype != NATS_F32) return NATS_ERR_DTYPE;
  if (c->n_pages < 0 || c->Hk <= 0 || c->B < 0 || c->max_pages < 0 || c->page <= 0 || c->page % 16 != 0)
    return NATS_ERR_SHAPE;
  if (c->d != 64 && c->d != 128) return NATS_ERR_UNSUPPORTED;
  // slots are 32-bit (with room for a tile behind the last one); so are heads x sequences (grids)
  if ((long long)c->max_pages * c->page > (1LL << 30) || (long long)c->B * c->Hk > (1LL << 30) ||
      (long long)c->B * c->max_pages > (1LL << 40))
    return NATS_ERR_UNSUPPORTED;
  return NATS_OK;
}

inline nats_status check_cache_pointers(const nats_paged_cache* c) {
  if (!c->lens || !c->err) return NATS_ERR_NULL;
  if (c->max_pages > 0 && !c->table) return NATS_ERR_NULL;
  if (c->n_pages > 0 && (!c->k_pages || !c->v_pages)) return NATS_ERR_NULL;
  if (((uintptr_t)c->k_pages | (uintptr_t)c->v_pages | (uintptr_t)c->weight) & 15u) return NATS_ERR_ALIGN;
  if (((uintptr_t)c->table | (uintptr_t)c->lens | (uintptr_t)c->err) & 3u) return NATS_ERR_ALIGN;
  return NATS_OK;
}

}  // namespace nats
