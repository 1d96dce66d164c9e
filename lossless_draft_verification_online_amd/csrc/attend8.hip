// Attention of a ragged batch's rows over a paged cache of e4m3 codes with a power-of-two scale for each block of tokens and
// head: sdv_attend8.
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdlib.h>

#include "attend_rows.hpp"

namespace attend8_impl {

using namespace sdv;
using namespace attend_impl;

enum Mode { kUnits, kFewUnits, kRanges, kSmallPages, kRows };

static int64_t kManyColumns_() { const char* e = getenv("KC"); return e ? atoll(e) : 96; }
constexpr int64_t kManyWorkgroups = 128;

constexpr int64_t kShort = 32, kSomeUnits = 64;
constexpr int64_t kManyUnits = 2048;
constexpr int64_t kUnpaired = 128;
// Eight waves for a unit instead of four, up to as many units of 16 columns: a wave waits 1 us for each of its tiles (one row of 17 tiles
// 9.3 us for 10.2, 16 trees of 33 tiles 14.5 for 17.3, 64 units of 32 tiles 11.6 for 13.8; 256 units of 16 tiles 17.7 for 13.0).
constexpr int64_t kEightWaves = 128;
constexpr int kFewWaves = 8;
static int64_t places() { const char* e = getenv("KP"); return e ? atoll(e) : 512; }

struct Plan {
  int qb;
  Mode mode;
  int32_t ranges;
  int32_t pieces;  // of a unit, about
  int64_t tiles;
  bool many;  // cut into more than a few
  size_t part_bytes, stat_bytes, bytes;
};

inline size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

inline Plan plan_of(const sdv_cache* c, int32_t B, int64_t n_d, int32_t n_q, int32_t window, int32_t sinks,
                    bool tree) {
  const int64_t G = n_q / c->n_kv_heads, rows = n_d + B, mean = (rows * G + B - 1) / B;
  int64_t seen = (int64_t)c->max_pages * c->page_size;
  if (window && (int64_t)window + sinks + rows / B < seen) seen = (int64_t)window + sinks + rows / B;
  const int64_t tokens = (seen + kTile - 1) / kTile;
  auto units_of = [&](int64_t columns) { return (mean + columns - 1) / columns * B * c->n_kv_heads; };
  Plan p = {};
  p.qb = 1;
  if (!tree && c->dtype == SDV_BF16 && c->head_dim <= 128 && c->page_size >= 16 && mean >= kManyColumns_() &&
      units_of(kRowsColumns) >= kManyWorkgroups) {
    p.mode = kRows;
    p.tiles = rows * G / kRowsColumns + B;
    return p;
  }
  const bool pairs = mean > 16 && !(c->dtype == SDV_FP32 && c->head_dim > 64);
  const bool split = tokens > (units_of(16) < kSomeUnits ? kShort : 2 * kShort) && B <= 512 &&
                     rows <= 64 * (int64_t)B && units_of(32) < kManyUnits;
  p.mode = c->page_size < 16 ? kSmallPages : (split ? kRanges : kUnits);
  if (pairs && (p.mode == kRanges || units_of(16) > kUnpaired)) p.qb = 2;
  if (p.mode == kUnits && p.qb == 1 && c->head_dim <= 128 && units_of(16) <= kEightWaves) p.mode = kFewUnits;
  p.tiles = rows * G / (16 * p.qb) + B;
  if (p.mode == kRanges) {
    const int64_t units = units_of(16 * p.qb) / c->n_kv_heads, groups = (units * tokens + kStreamWaves - 1) / kStreamWaves;
    const int64_t most = places() / c->n_kv_heads > 0 ? places() / c->n_kv_heads : 1;
    p.ranges = (int32_t)(groups < most ? groups : most);
    p.pieces = (int32_t)((p.ranges + units - 1) / units) + 1;
    const size_t n = (size_t)2 * p.ranges * c->n_kv_heads * 16 * p.qb;
    p.part_bytes = up256(n * c->head_dim * 4);
    p.stat_bytes = up256(n * 8);
    p.many = p.pieces > 16;
    const size_t cuts = (size_t)(p.many ? p.tiles : p.ranges) * c->n_kv_heads + 1;
    p.bytes = p.part_bytes + p.stat_bytes + up256(cuts * sizeof(Cut));
  }
  return p;
}

template <class E, int D, int QB>
int launch(const AttendArgs& a, const Plan& p, hipStream_t s) {
  const dim3 units((unsigned)(a.tiles * a.cache.n_heads)), threads(kStreamWaves * kWave);
  if constexpr (QB == 1 && D <= 128) {
    if (p.mode == kFewUnits) {
      hipLaunchKernelGGL((attend_units<E, D, QB, kFewWaves, true, true>), units, dim3(kFewWaves * kWave), 0, s, a);
      return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
    }
  }
  if (p.mode == kSmallPages) {
    hipLaunchKernelGGL((attend_units<E, D, QB, kStreamWaves, false, true>), units, threads, 0, s, a);
  } else if (p.mode == kUnits) {
    hipLaunchKernelGGL((attend_units<E, D, QB, kStreamWaves, true, true>), units, threads, 0, s, a);
  } else {
    hipLaunchKernelGGL((attend_ranges<E, D, QB, true>), dim3((unsigned)(a.ranges * a.cache.n_heads)), threads, 0, s, a);
    if (a.ranges == 1) return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
    if (p.many)
      hipLaunchKernelGGL((join<E, D, QB, true, true>), dim3(units.x, 16 * QB), dim3(kJoinWaves * kWave), 0, s, a);
    else
      hipLaunchKernelGGL((join<E, D, QB, false, true>), dim3((unsigned)(a.ranges * a.cache.n_heads), 16 * QB / kJoin), dim3(kJoinWaves * kWave), 0, s, a);
  }
  return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
}

template <class E, int D>
int launch_columns(const AttendArgs& a, const Plan& p, hipStream_t s) {
  if constexpr (E::kBytes == 2 && D <= 128) {
    if (p.mode == kRows) {
      hipLaunchKernelGGL((attend_rows<D, true>), dim3((unsigned)(a.tiles * a.cache.n_heads)), dim3(kRowsWaves * kWave), 0, s, a);
      return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
    }
  }
  if constexpr (E::kBytes == 2 || D <= 64) {
    if (p.qb == 2) return launch<E, D, 2>(a, p, s);
  }
  return launch<E, D, 1>(a, p, s);
}

template <class E>
int launch_dim(const AttendArgs& a, int32_t D, const Plan& p, hipStream_t s) {
  return D == 64 ? launch_columns<E, 64>(a, p, s)
                 : (D == 128 ? launch_columns<E, 128>(a, p, s) : launch_columns<E, 256>(a, p, s));
}

inline int check(const sdv_cache* c, int32_t B, int64_t n_d, int32_t n_q, int32_t window, int32_t sinks) {
  if (n_q < 1 || n_q % c->n_kv_heads || window < 0 || sinks < 0) return SDV_ERR_INVALID_ARG;
  if (n_q > 1024 || (n_d + B) * (n_q / c->n_kv_heads) > INT32_MAX - 1024) return SDV_ERR_LIMIT;
  return plan_of(c, B, n_d, n_q, window, sinks, true).tiles * c->n_kv_heads > INT32_MAX ? SDV_ERR_LIMIT : SDV_OK;
}

}  // namespace attend8_impl

extern "C" size_t sdv_attend8_workspace_bytes(const sdv_cache8* cache, int32_t B, int64_t n_draft_rows,
                                              int32_t n_q_heads, int32_t window, int32_t sinks) {
  using namespace attend8_impl;
  if (!cache || B < 1 || n_draft_rows < 0 || cache->cache.n_kv_heads < 1 || cache->cache.max_pages < 1 ||
      cache->cache.page_size < 1 || n_draft_rows + B > INT32_MAX ||
      check(&cache->cache, B, n_draft_rows, n_q_heads, window, sinks) != SDV_OK)
    return 0;
  return plan_of(&cache->cache, B, n_draft_rows, n_q_heads, window, sinks, true).bytes;  // without a tree: that or less
}

extern "C" int sdv_attend8(const sdv_cache8* cache, int32_t B, int64_t n_draft_rows, const int32_t* ragged_offsets,
                           const int32_t* parents, const void* queries, int64_t query_stride, int32_t n_q_heads,
                           float scale, int32_t window, int32_t sinks, void* out, void* workspace,
                           size_t workspace_bytes, void* stream) {
  using namespace attend8_impl;
  int rc = check_cache8(cache, B, n_draft_rows, ragged_offsets);
  if (rc != SDV_OK) return rc;
  const sdv_cache* const c = &cache->cache;
  rc = check(c, B, n_draft_rows, n_q_heads, window, sinks);
  if (rc != SDV_OK) return rc;
  const int64_t per = c->dtype == SDV_BF16 ? 8 : 4;
  if (!queries || !out || out == queries || !aligned16(queries) || !aligned16(out) || query_stride % per ||
      query_stride < (int64_t)n_q_heads * c->head_dim || !(scale - scale == 0.0f))
    return SDV_ERR_INVALID_ARG;
  if (query_stride > ((int64_t)1 << 31)) return SDV_ERR_LIMIT;
  const Plan p = plan_of(c, B, n_draft_rows, n_q_heads, window, sinks, parents != nullptr);
  static_assert(kStreamWaves == kJoinWaves && kStreamWaves == kRowsWaves, "one bound for every launch");
  if (too_many(p.tiles * c->n_kv_heads, (p.mode == kFewUnits ? kFewWaves : kStreamWaves) * kWave)) return SDV_ERR_LIMIT;
  if (p.bytes > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < p.bytes)) return SDV_ERR_WORKSPACE;
  AttendArgs a;
  a.cache = view_of(c);
  a.B = B;
  a.n_q = n_q_heads;
  a.G = n_q_heads / c->n_kv_heads;
  a.ranges = p.ranges;
  a.window = window;
  a.sinks = sinks;
  a.n_d = n_draft_rows;
  a.query_stride = query_stride;
  a.tiles = p.tiles;
  a.scale2 = fmaxf(fabsf(scale) * 1.4426950408889634f, 0x1p-126f);
  a.flip = scale < 0 ? (c->dtype == SDV_BF16 ? 0x80008000u : 0x80000000u) : 0u;
  a.cu = ragged_offsets;
  a.parents = parents;
  a.queries = static_cast<const char*>(queries);
  a.out = static_cast<char*>(out);
  a.part = static_cast<float*>(workspace);
  a.stats = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.part_bytes);
  a.many = p.many;
  a.cuts = reinterpret_cast<Cut*>(static_cast<char*>(workspace) + p.part_bytes + p.stat_bytes);
  a.key_scales = cache->key_scales;
  a.value_scales = cache->value_scales;
  a.block_log2 = log2_of(cache->block);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return c->dtype == SDV_BF16 ? launch_dim<Bf16>(a, c->head_dim, p, s) : launch_dim<F32>(a, c->head_dim, p, s);
}

