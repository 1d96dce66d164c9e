// Attention of a ragged batch's rows over a paged cache of e4m3 codes with a power-of-two scale for each block of tokens and
// head: sdv_attend8.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "attend_rows.hpp"

namespace attend8_impl {

using namespace sdv;
using namespace attend_impl;

enum Mode { kUnits, kFewUnits, kRanges, kSmallPages, kRows };

// The rules, by what the host knows: the batch's mean columns of a request, and for its lengths the page table's width (under a
// window, the window).  Times of 8 heads of 128 values, bf16 rows, for one side and the other, each that of a call in a replayed
// graph (from Python a call takes 5 us at least); a tile is of 32 tokens, a unit of 16 columns on one head.
//
// attend_rows from this many columns of a request and this many workgroups on: 16 requests of 256 columns on 1000 tokens 47.9 us for
// 50.6 by units, of 512 on 4000 181 for 293, one of 4096 on 1000 59 for 86; 64 of 128 on 4000 340 for 316, 4 of 512 on 4000
// (128 workgroups) 113 for 76 by ranges.
constexpr int64_t kManyColumns = 256, kManyWorkgroups = 256;

// Eight waves for a unit instead of four, up to as many units: a wave waits 1 us for each of its tiles (one request of 47 tiles 15.2 us
// for 18.0, 16 of 63 20.3 for 25.9, 24 of 63 22.0 for 30.7).  A second round of such workgroups costs more than they gain (32
// requests of 20 columns on 16 tiles, 512 units, 19.1 for 14.8).  The bound is lower than it could be: at 256 units, 32 requests
// of 16 columns, eight waves take 13.8, 17.5, 26.6 and 52.3 on 16, 32, 63 and 125 tiles for the 15.1, 20.0, 32.7 and 61.3 of the plans
// taken; binary32 rows of 64 values, 16 of 32 columns on 125 tiles, 31.7 for 39.8.
constexpr int64_t kEightWaves = 192;
constexpr int kFewWaves = 8;

// Units of 16 columns up to which they are not paired (32 requests of 32 columns on 1000 tokens, 512 units, 21.0 us for 25.3 in
// pairs, 40 of them 25.5 for 26.2, 64 42.3 for 31.3).  Ranges are in pairs: they read the cache again for each column tile (64 of 20
// columns on 4000 tokens 105 us for 190).  Heads of 256 values never are: a pair takes the registers of all waves (16 of 64 columns
// on 4000 tokens 69 us by ranges and 85 by units, 95 in pairs by units; 16 of 32 columns 51, 61 and 94; 64 of 32 columns on 1000 tokens
// 42, 35 and 39, but on 4000 136, 117 and 112, of which the rule takes the ranges), nor are binary32 ones above 64.
constexpr int64_t kUnpaired = 640;

// Ranges from more tiles on than this: one request on 47 tiles 15.6 us for 15.2 by units, on 63 12.5 for 17.9; 16 (128 units) on 126
// 34.3 for 33.7, on 94 29.1 for 26.4; 32 (256 units) on 63 35.0 for 32.1, on 126 61 for 66; 64 (512 units) on 31 30.2 for 28.9, on 63
// 58.0 for 60.6; 256 (2048 units) on 31 122 either way, on 63 213 for 228.
inline int64_t short_of(int64_t units) {
  if (units <= kEightWaves) return units > 48 ? units : 48;
  return units < 512 ? 96 : 48;
}

// Requests of several column tiles run by units, whose tiles read the cache at one time, but for few of them (64 of 64 columns on 4000
// tokens 167 us for 214 by ranges, 16 of 128 74 for 80; 16 of 64 69 for 57, 4 of 512 111 for 76, one of 512 57 for 41).
constexpr int64_t kFewPairs = 256, kFewRequests = 4;

// Ranges take all of a request's tokens for each of its rows: rows up to this part of the tokens.
constexpr int64_t kRowsOfTokens = 8;

// Workgroups at once: two per compute unit.
constexpr int64_t kPlaces = 512;

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
  if (!tree && c->dtype == SDV_BF16 && c->head_dim <= 128 && c->page_size >= 16 && mean >= kManyColumns &&
      units_of(kRowsColumns) >= kManyWorkgroups) {
    p.mode = kRows;
    p.tiles = rows * G / kRowsColumns + B;
    return p;
  }
  const int64_t units = units_of(16);
  const bool pairs = mean > 16 && c->head_dim <= (c->dtype == SDV_FP32 ? 64 : 128);
  const bool split = tokens > short_of(units) && B <= 512 && rows * kRowsOfTokens <= tokens * kTile * B &&
                     (mean <= 32 || units_of(32) <= kFewPairs || B <= kFewRequests);
  p.mode = c->page_size < 16 ? kSmallPages : (split ? kRanges : kUnits);
  if (pairs && (p.mode == kRanges || units > kUnpaired)) p.qb = 2;
  if (p.mode == kUnits && p.qb == 1 && c->head_dim <= 128 && units <= kEightWaves) p.mode = kFewUnits;
  p.tiles = rows * G / (16 * p.qb) + B;
  if (p.mode == kRanges) {
    const int64_t per_head = units_of(16 * p.qb) / c->n_kv_heads;
    const int64_t groups = (per_head * tokens + kStreamWaves - 1) / kStreamWaves;
    const int64_t most = kPlaces / c->n_kv_heads > 0 ? kPlaces / c->n_kv_heads : 1;
    p.ranges = (int32_t)(groups < most ? groups : most);
    p.pieces = (int32_t)((p.ranges + per_head - 1) / per_head) + 1;
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
      hipLaunchKernelGGL((join<E, D, QB, false, true>), dim3((unsigned)(a.ranges * a.cache.n_heads), 16 * QB / kJoin),
                         dim3(kJoinWaves * kWave), 0, s, a);
  }
  return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
}

template <class E, int D>
int launch_columns(const AttendArgs& a, const Plan& p, hipStream_t s) {
  if constexpr (E::kBytes == 2 && D <= 128) {
    if (p.mode == kRows) {
      hipLaunchKernelGGL((attend_rows<D, true>), dim3((unsigned)(a.tiles * a.cache.n_heads)), dim3(kRowsWaves * kWave), 0, s,
                         a);
      return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
    }
  }
  if constexpr (D <= (E::kBytes == 2 ? 128 : 64)) {
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

