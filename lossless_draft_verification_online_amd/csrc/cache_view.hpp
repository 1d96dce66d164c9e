// What the kernels over the paged cache share: the cache's places, the request of a row, and the
// checks of a call's cache arguments.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/sdv.h"
#include "launch.hpp"
#include "sdv_device.hpp"

namespace sdv {

constexpr int kMaxNodes = SDV_MAX_DEPTH;

struct CacheView {
  char* keys;
  char* values;
  const int32_t* table;
  const int32_t* len;
  int64_t n_pages;
  int32_t max_pages, page_log2, n_heads;

  // The page that holds slot s of request i, or -1.
  __device__ __forceinline__ int32_t page(int32_t i, int64_t s) const {
    const int64_t k = s >> page_log2;
    if (s < 0 || k >= max_pages) return -1;
    const int32_t p = table[(int64_t)i * max_pages + k];
    return p >= 0 && p < n_pages ? p : -1;
  }
  // Row (of head_dim values) of a slot in its page.
  __device__ __forceinline__ int64_t row(int32_t page, int32_t head, int64_t s) const {
    return (((int64_t)page * n_heads + head) << page_log2) + (s & ((1 << page_log2) - 1));
  }
};

// The last i in [0, n) with f(i) <= key, for a non-decreasing f: every lane tests one of 64 evenly
// spread places, so a batch of 4096 requests takes two rounds of loads.  -1 if f(0) > key, or if the
// answers show that f decreases.  The result is the same in every lane.
template <class F>
__device__ __forceinline__ int32_t find_last(int32_t n, int64_t key, F f) {
  const int lane = threadIdx.x & (kWave - 1);
  int64_t lo = 0, left = n;
  for (bool first = true; left > 1 || first; first = false) {
    const int64_t step = (left + kWave - 1) / kWave;
    const int64_t at = (int64_t)lane * step;
    const uint64_t yes = __ballot(at < left && f((int32_t)(lo + at)) <= key);
    if (!yes || (yes & (yes + 1))) return -1;
    const int64_t hop = (int64_t)(63 - __builtin_clzll(yes)) * step;
    lo += hop;
    left = left - hop < step ? left - hop : step;
  }
  return (int32_t)lo;
}

// The first i in [0, n) with f(i), or -1: every request looked at, 64 at a time.
template <class F>
__device__ __forceinline__ int32_t find_among(int32_t n, F f) {
  for (int32_t i0 = 0; i0 < n; i0 += kWave) {
    const int32_t i = i0 + (int32_t)(threadIdx.x & (kWave - 1));
    const uint64_t yes = __ballot(i < n && f(i));
    if (yes) return i0 + __ffsll((unsigned long long)yes) - 1;
  }
  return -1;
}

// Whether the positions of a request of K + 1 rows behind len cached slots are 32-bit numbers, with room for a tile.
__device__ __forceinline__ bool len_fits(int32_t len, int32_t k) { return len >= 0 && len < INT32_MAX - 1024 - k; }

struct Request {
  int32_t index, first, k;  // its number, its first draft row cu[i], its K; index -1: offsets not valid
  int64_t row0;             // cu[i] + i
};

__device__ __forceinline__ Request request_at(const int32_t* cu, int32_t i, int64_t n_d) {
  Request r;
  r.index = -1;
  r.first = r.k = 0;
  r.row0 = 0;
  if (i < 0) return r;
  const int32_t lo = cu[i], hi = cu[i + 1];
  if (lo < 0 || hi < lo || hi > n_d) return r;
  r.index = i;
  r.first = lo;
  r.k = hi - lo;
  r.row0 = (int64_t)lo + i;
  return r;
}

// The request of a row.  One offset that is not valid makes its two requests invalid, and can mislead the search for
// others' rows: where the search meets answers out of order or ends at a request that is not valid, every
// request is looked at.  (Where it ends at a valid one, that one's end is the next one's start, which it found to lie behind
// the row.)  A batch without such offsets pays 1% of 10467 rows' 22.6 us for the test.
__device__ __forceinline__ Request request_of_row(const int32_t* cu, int32_t B, int64_t n_d, int64_t row) {
  Request r = request_at(cu, find_last(B, row, [&](int32_t i) { return (int64_t)cu[i] + i; }), n_d);
  if (__builtin_expect(r.index < 0, 0))
    r = request_at(cu, find_among(B, [&](int32_t i) {
                     const Request q = request_at(cu, i, n_d);
                     return q.index >= 0 && row >= q.row0 && row <= q.row0 + q.k;
                   }), n_d);
  return r;
}

// A tree's depths, by rows (row 0 the last committed token, row n + 1 node n): the first wave stages the
// parents in shared memory and each lane walks its node's path.  False if the tree is not valid.
// All threads of the workgroup call it; depth holds kMaxNodes + 1 values.
__device__ __forceinline__ bool tree_depths(const int32_t* parents, const Request& r, int32_t* parent_s,
                                            int32_t* depth) {
  if (r.k > kMaxNodes) return false;
  const int t = threadIdx.x;
  bool ok = true;
  if (t < kWave) {
    int32_t p = -1;
    if (t < r.k) {
      p = parents[r.first + t];
      ok = p >= -1 && p < t;
    }
    ok = __ballot(!ok) == 0;
    parent_s[t] = ok ? p : -1;
    if (t == 0) depth[0] = ok ? 0 : -1;
  }
  __syncthreads();
  ok = depth[0] == 0;
  if (t < r.k) {
    int32_t d = 1;
    for (int32_t p = parent_s[t]; p >= 0; p = parent_s[p]) ++d;
    depth[t + 1] = d;
  }
  __syncthreads();
  return ok;
}

inline int log2_of(int32_t n) {
  int k = 0;
  while ((1 << k) < n) ++k;
  return k;
}

inline bool overlap(const void* a, int64_t a_bytes, const void* b, int64_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y ? y - x < (uintptr_t)a_bytes : x - y < (uintptr_t)b_bytes;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Checks what every call over a cache has in common.
inline int check_cache(const sdv_cache* c, int32_t B, int64_t n_d, const int32_t* cu) {
  if (!c) return SDV_ERR_INVALID_ARG;
  if (c->dtype != SDV_BF16 && c->dtype != SDV_FP32) return SDV_ERR_UNSUPPORTED;
  if (!c->keys || !c->values || !c->page_table || !c->cache_len || !cu || B < 1 || n_d < 0 || c->n_pages < 1 ||
      c->max_pages < 1 || c->n_kv_heads < 1 || c->page_size < 1 || c->page_size > 1024 ||
      (c->page_size & (c->page_size - 1)) || (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) ||
      !aligned16(c->keys) || !aligned16(c->values))
    return SDV_ERR_INVALID_ARG;
  if (n_d + B > INT32_MAX - 1024 || c->n_kv_heads > 1024 || c->n_pages > INT32_MAX) return SDV_ERR_LIMIT;
  return SDV_OK;
}

inline CacheView view_of(const sdv_cache* c) {
  CacheView v;
  v.keys = static_cast<char*>(c->keys);
  v.values = static_cast<char*>(c->values);
  v.table = c->page_table;
  v.len = c->cache_len;
  v.n_pages = c->n_pages;
  v.max_pages = c->max_pages;
  v.page_log2 = log2_of(c->page_size);
  v.n_heads = c->n_kv_heads;
  return v;
}

}  // namespace sdv
