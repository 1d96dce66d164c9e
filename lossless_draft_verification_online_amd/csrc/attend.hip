// Attention of a ragged batch's rows over the paged cache, with a sliding window and first tokens
// that stay visible: sdv_attend.
//
// out = sum_s p_s v_s / sum_s p_s with p_s = 2^(c <q, k_s> - m), c = scale log2(e) and m the running
// maximum: one pass over the keys and values.  The query heads that share a key/value head, times the
// rows of a request, are the columns of one product: with G = n_q_heads / n_kv_heads column r is
// row r / G, head r % G.
//
// Scores are computed transposed, S^T = K Q^T (matrix instructions of 16 tokens x 16 columns): a
// lane then holds four consecutive tokens of one column, so the statistics of a column are a lane's
// own values and two swaps across the wave, and the probabilities are, as they lie, the B operand
// of O^T = V^T P^T.  The contraction's token order is free as long as both operands agree, so
// nothing is moved between the two products.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "cache_view.hpp"

namespace attend_impl {

using namespace sdv;

constexpr int kTile = 32;  // tokens a wave takes at a time

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

struct AttendArgs {
  CacheView cache;
  int32_t B, n_q, G, window, sinks;
  int32_t ranges;  // the ranges that the batch's work is cut into
  int64_t n_d, query_stride, tiles;
  float scale2;  // |scale| log2(e), at least 2^-126: a masked -inf stays one; the sign goes to the queries
  uint32_t flip;  // sign bits of a word of queries, set for a negative scale
  const int32_t* cu;
  const int32_t* parents;
  const char* queries;
  char* out;
  float* part;   // [2 ranges][columns][D] sums of a piece of a unit, in the frame of its maxima
  float* stats;  // [2 ranges][columns][2] maximum and sum of weights
};

// First tile number of request i: its columns take at most ceil((K + 1) G / columns) tiles from there.
__device__ __forceinline__ int64_t first_tile(const int32_t* cu, int32_t i, int32_t G, int32_t columns) {
  return (uint32_t)(cu[i] + i) * (uint32_t)G / (uint32_t)columns + i;  // below 2^31, as n_draft_rows + B times G is
}

struct TileOf {
  Request r;
  int32_t c0;  // its first column within the request
};

// The tile of request r, whose index is -1 if it does not have that one.
template <int kColumns>
__device__ __forceinline__ TileOf tile_in(const AttendArgs& a, const Request& r, int64_t tile) {
  TileOf t;
  t.r = r;
  t.c0 = 0;
  if (r.index < 0) return t;
  const int64_t c0 = (tile - first_tile(a.cu, r.index, a.G, kColumns)) * kColumns;
  if (c0 < 0 || c0 >= (int64_t)(r.k + 1) * a.G) t.r.index = -1;
  t.c0 = (int32_t)c0;
  return t;
}

// The request of a tile by a look at every one: for batches with offsets that are not valid (as in request_of_row).
template <int kColumns>
__device__ __forceinline__ int32_t tile_among(const AttendArgs& a, int64_t tile) {
  return find_among(a.B, [&](int32_t q) {
    return tile_in<kColumns>(a, request_at(a.cu, q, a.n_d), tile).r.index >= 0;
  });
}

template <int kColumns>
__device__ __forceinline__ TileOf tile_of(const AttendArgs& a, int64_t tile) {
  const int32_t i =
      find_last(a.B, tile, [&](int32_t q) { return first_tile(a.cu, q, a.G, kColumns); });
  Request r = request_at(a.cu, i, a.n_d);
  if (__builtin_expect(r.index < 0, 0)) r = request_at(a.cu, tile_among<kColumns>(a, tile), a.n_d);
  return tile_in<kColumns>(a, r, tile);
}

// Workgroups go to the 8 XCDs in turn.  Each XCD takes a run of neighbouring units instead: the heads of one page
// lie next to each other, so an XCD then reads whole pages (paged reads 5.0 -> 6.0 TB/s), and tiles
// of one request share its L2.
__device__ __forceinline__ int64_t unit_of_block(int64_t block, int64_t n) {
  const int64_t x = block & 7, q = n >> 3, r = n & 7;
  return x * q + (x < r ? x : r) + (block >> 3);
}

// The token tiles that rows j_lo .. j_hi of a request see: [0, near_end) and [lo, hi).
struct Span {
  int32_t lo, hi, near_end, t_lo, n_near, n;
};
__device__ __forceinline__ Span span_of(int32_t len, int32_t pos_lo, int32_t pos_hi, int32_t window, int32_t sinks) {
  Span s;
  s.hi = len + pos_hi + 1;
  s.lo = window && len + pos_lo >= window ? len + pos_lo - window + 1 : 0;
  s.near_end = s.lo < sinks ? s.lo : sinks;
  s.t_lo = s.lo / kTile;
  s.n_near = (s.near_end + kTile - 1) / kTile;
  if (s.t_lo <= s.n_near) {  // the first tokens' tiles run into the window's
    s.t_lo = 0;
    s.n_near = 0;
  }
  s.n = s.n_near + (s.hi + kTile - 1) / kTile - s.t_lo;
  return s;
}

// The batch's work is the list of its units (tile of columns, head), request by request, each of its token tiles.
// The list is cut into equal ranges, one per workgroup: lengths differ between requests, and few units leave
// places empty (one request of 8 heads on 4000 tokens: 17 us by ranges, 42 by units).
struct Work {
  int32_t first, k, len;      // the request
  int32_t tiles, n;           // column tiles; token tiles of a unit (those of all its rows)
  __device__ int64_t units(const AttendArgs& a) const { return (int64_t)tiles * a.cache.n_heads; }
};
__device__ __forceinline__ Work work_of(const AttendArgs& a, int32_t i, int32_t columns) {
  Work w;
  w.tiles = w.n = 0;
  w.len = a.cache.len[i];
  const Request r = request_at(a.cu, i, a.n_d);
  w.first = r.first;
  w.k = r.k;
  if (r.index < 0) return w;
  w.tiles = (int32_t)(((uint32_t)(r.k + 1) * a.G + columns - 1) / (uint32_t)columns);
  w.n = !len_fits(w.len, r.k) ? 1 : span_of(w.len, 0, r.k, a.window, a.sinks).n;
  return w;
}
struct Stream {
  int32_t per;                   // requests per lane
  Work own;                      // of the lane's first
  int64_t before, units_before;  // items, and units, before the lane's requests
  int64_t total;                 // items of the batch
  int64_t length;                // of a range
};
__device__ __forceinline__ Stream stream_of(const AttendArgs& a, int32_t columns) {
  const int lane = threadIdx.x & (kWave - 1);
  Stream s;
  s.per = (a.B + kWave - 1) / kWave;
  s.own.first = s.own.k = s.own.len = s.own.tiles = s.own.n = 0;
  uint64_t items = 0, units = 0;
  for (int32_t k = 0; k < s.per; ++k) {
    const int32_t i = lane * s.per + k;
    if (i >= a.B) break;
    const Work w = work_of(a, i, columns);
    if (k == 0) s.own = w;
    items += (uint64_t)(w.units(a) * w.n);
    units += (uint64_t)w.units(a);
  }
  const uint64_t inc = wave_inclusive_scan(items);
  s.before = (int64_t)(inc - items);
  s.units_before = (int64_t)(wave_inclusive_scan(units) - units);
  s.total = (int64_t)lane_value(inc, kWave - 1);
  s.length = (s.total + a.ranges - 1) / a.ranges;
  return s;
}
// The work of request i: from the lanes where they hold one request each.
__device__ __forceinline__ Work work_at(const AttendArgs& a, const Stream& s, int32_t i, int32_t columns) {
  if (s.per > 1) return work_of(a, i, columns);
  Work w;
  w.first = lane_value(s.own.first, i);
  w.k = lane_value(s.own.k, i);
  w.len = lane_value(s.own.len, i);
  w.tiles = lane_value(s.own.tiles, i);
  w.n = lane_value(s.own.n, i);
  return w;
}
__device__ __forceinline__ Request request_with(const Work& w, int32_t i) {
  Request r;
  r.index = i;
  r.first = w.first;
  r.k = w.k;
  r.row0 = (int64_t)w.first + i;
  return r;
}

__device__ __forceinline__ float both_max16_32(float v) {
  float x, y;
  wave_detail::both<16>(v, x, y);
  v = fmaxf(x, y);
  wave_detail::both<32>(v, x, y);
  return fmaxf(x, y);
}
__device__ __forceinline__ float both_sum16_32(float v) {
  float x, y;
  wave_detail::both<16>(v, x, y);
  v = x + y;
  wave_detail::both<32>(v, x, y);
  return x + y;
}

// Which rows of a tree a row sees: bit t of rows for row t < 64, last for row 64.
struct TreeSight {
  uint64_t rows;
  bool last;
};

template <class E, int D, int QB, int kWaves>
struct Shape {
  static constexpr int kColumns = 16 * QB;
  static constexpr bool kBf16 = E::kBytes == 2;
  static constexpr int kValueStride = D * 2 + 32;  // bytes; rows 8 banks apart for the transposing reads
  static constexpr int kValueBytes = kBf16 ? kWaves * kTile * kValueStride : 0;
  static constexpr int kMergeStride = D + 4;
  static constexpr int kMergeBytes = kWaves / 2 * kColumns * kMergeStride * 4;
  static constexpr int kBytes = kValueBytes > kMergeBytes ? kValueBytes : kMergeBytes;
};

template <class E, int D, int QB, int kWaves>
struct Scratch {
  using S = Shape<E, D, QB, kWaves>;
  __align__(16) char smem[S::kBytes];
  float m_s[kWaves][S::kColumns], l_s[kWaves][S::kColumns];
  int32_t odd_s[kWaves];
  int32_t parent_s[kWave], depth_s[kMaxNodes + 1];
  uint64_t sight_s[kMaxNodes + 1];
  int32_t last_s[kMaxNodes + 1];
};

// Values that are not finite, in a tile that not every column sees whole: a column that does not see such a token has
// the weight 0 for it, and 0 times NaN is NaN.  The tiles' products take 0 in their place, and where there were
// some, a pass behind the unit adds them to the results of the columns that do see them (an infinity or NaN times a
// positive weight is itself).
__device__ __forceinline__ bool not_finite(u32x4 v) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 top = {0, 0};
#pragma unroll
  for (int w = 0; w < 4; ++w) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, v[w] & 0x7fff7fffu));
  return top.x >= 0x7f80 || top.y >= 0x7f80;
}
__device__ __forceinline__ u32x4 finite_of(u32x4 v) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if ((v[w] & 0x7f80u) == 0x7f80u) v[w] &= 0xffff0000u;
    if ((v[w] & 0x7f800000u) == 0x7f800000u) v[w] &= 0xffffu;
  }
  return v;
}
// One wave, for its columns and the tiles of [lo, hi) that are not all_see(start): add(column, d, value).
template <class E, int D, int kTokens, class Start, class AllSee, class Sees, class Add>
__device__ __forceinline__ void add_not_finite(const AttendArgs& a, int32_t i, int32_t head, int32_t lo, int32_t hi,
                                               int32_t columns, Start start, AllSee all_see, Sees sees, Add add) {
  const int lane = threadIdx.x & (kWave - 1);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");  // the results are there
  for (int32_t n = lo; n < hi; ++n) {
    if (all_see(start(n))) continue;
    for (int32_t s = start(n); s < start(n) + kTokens; ++s) {
      const int32_t page = a.cache.page(i, s);
      if (page < 0) continue;
      const char* const row = a.cache.values + a.cache.row(page, head, s) * (D * E::kBytes);
#pragma unroll 1
      for (int d = lane; d < D; d += kWave) {
        const float v = E::at(row, d);
        const bool bad = !(v - v == 0.0f);
        if (!__any(bad)) continue;
        for (int32_t c = 0; c < columns; ++c)
          if (sees(c, s) && bad) add(c, d, v);
      }
    }
  }
}
template <class E>
__device__ __forceinline__ void add_to(char* out, int d, float v) {
  if constexpr (E::kBytes == 2) {
    __bf16* const p = reinterpret_cast<__bf16*>(out) + d;
    *p = (__bf16)((float)*p + v);
  } else {
    reinterpret_cast<float*>(out)[d] += v;
  }
}

// One unit (a tile of a request's columns, one key/value head), or of its token tiles [w_lo, w_hi) when
// pos_all (then the tiles are those of all of the request's rows).  slot: where the sums go that another
// workgroup's are joined with; -1: the unit is whole and its result is written.
//
// kWholePages: pages hold 16 slots or more, so 16 tokens lie in one page and its address is a scalar; smaller
// pages take an address per token.
//
// The waves of a workgroup take every fourth tile of 32 tokens, keys and values loaded a tile ahead, and join their sums
// at the end.  Bound by the reads of the cache: 64 requests of K in 0..8 on 4096 to 8192 tokens (window 4096, 8 heads of
// 128, bf16) 232 us, 4.6 TB/s of 1.08 GB (a large copy reaches 4.9), with the second tile of requests of more than 32 columns read again.  Few units
// are bound by what a compute unit loads (1000 tokens of a head, 512 KB, in about 8 us; 8 waves instead of 4 take as long).
template <class E, int D, int QB, int kWaves, bool kWholePages>
__device__ __forceinline__ void attend_unit(const AttendArgs& a, Scratch<E, D, QB, kWaves>& sh, const TileOf& at,
                                            int32_t len, int32_t head, bool pos_all, int32_t w_lo, int32_t w_hi, int64_t slot) {
  using S = Shape<E, D, QB, kWaves>;
  constexpr bool kBf16 = S::kBf16;
  constexpr int kSteps = kBf16 ? D / 32 : D / 16;  // 16-byte pieces of a key row per lane
  constexpr int kDB = D / 16;                       // blocks of 16 output values
  char* const smem = sh.smem;
  auto& m_s = sh.m_s;
  auto& l_s = sh.l_s;
  auto& parent_s = sh.parent_s;
  auto& depth_s = sh.depth_s;
  auto& sight_s = sh.sight_s;
  auto& last_s = sh.last_s;

  const int t = threadIdx.x, lane = t & (kWave - 1), col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int32_t i = at.r.index, K = at.r.k;
  const int32_t columns = (K + 1) * a.G;
  const int32_t c_last = at.c0 + S::kColumns < columns ? at.c0 + S::kColumns - 1 : columns - 1;
  const int32_t j_lo = (uint32_t)at.c0 / (uint32_t)a.G, j_hi = (uint32_t)c_last / (uint32_t)a.G;  // rows of this tile
  bool ok = len_fits(len, K);
  if (a.parents && ok) {
    ok = tree_depths(a.parents, at.r, parent_s, depth_s);
    if (ok) {
      if (t <= K) {
        uint64_t rows = a.window == 0 || depth_s[t] < a.window || len < a.sinks;
        bool last = false;
        for (int32_t n = t - 1; n >= 0; n = parent_s[n]) {
          if (!(a.window == 0 || depth_s[t] - depth_s[n + 1] < a.window || len + n + 1 < a.sinks)) continue;
          if (n < 63)
            rows |= 2ull << n;
          else
            last = true;
        }
        sight_s[t] = rows;
        last_s[t] = last;
      }
      __syncthreads();
    }
  }

  // this lane's columns: their rows, positions and queries
  int32_t pos[QB];
  int32_t jrow[QB];
  bool live[QB];
  TreeSight sight[QB];
  u32x4 q[QB][kSteps];
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    const int32_t c = at.c0 + 16 * b + col;
    live[b] = ok && c < columns;
    jrow[b] = live[b] ? (uint32_t)c / (uint32_t)a.G : 0;
    pos[b] = len + (a.parents && live[b] ? depth_s[jrow[b]] : jrow[b]);
    sight[b].rows = a.parents && live[b] ? sight_s[jrow[b]] : 0;
    sight[b].last = a.parents && live[b] ? last_s[jrow[b]] != 0 : false;
    const int32_t h = head * a.G + (c - jrow[b] * a.G);
    const char* src = a.queries + ((at.r.row0 + jrow[b]) * a.query_stride + h * D) * E::kBytes + 16 * g;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      u32x4 z;
      z.x = z.y = z.z = z.w = 0;
      if (live[b]) z = *reinterpret_cast<const u32x4*>(src + 64 * s) ^ a.flip;
      q[b][s] = z;
    }
  }

  // the tiles are those of the rows, or of all the request's rows; what this tile's rows see of them is the same
  const int32_t tail_lo = a.parents ? 0 : j_lo, tail_hi = a.parents ? K : j_hi;
  const Span own = span_of(len, tail_lo, tail_hi, a.window, a.sinks);
  const Span span = pos_all ? span_of(len, 0, K, a.window, a.sinks) : own;
  const int32_t lo = own.lo, hi = own.hi, near_end = own.near_end, n_near = span.n_near, t_lo = span.t_lo;
  if (!pos_all) {
    w_lo = 0;
    w_hi = span.n;
  }
  if (!ok) w_hi = w_lo;
  const int32_t far = len + tail_hi;  // the largest position
  auto start = [&](int32_t n) { return (n < n_near ? n : n - n_near + t_lo) * kTile; };
  auto held = [&](int32_t s) { return (s >= lo && s < hi) || s < near_end; };

  f32x4 acc[QB][kDB];
  float m[QB], l[QB];
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    m[b] = -__builtin_inff();
    l[b] = 0.0f;
#pragma unroll
    for (int d = 0; d < kDB; ++d) acc[b][d] = f32x4{0, 0, 0, 0};
  }

  // every row of the tile's columns sees every token from s0 on that is in a page
  auto all_see = [&](int32_t s0) {
    return s0 + kTile <= (a.parents ? len : len + j_lo + 1) &&
           (a.window == 0 || s0 > far - a.window || s0 + kTile <= a.sinks);
  };
  bool odd = false;

  char* const v_lds = smem + wave * kTile * S::kValueStride;
  u32x4 kreg[2][kSteps];
  u32x4 vreg[kBf16 ? D / 16 : 1];
  float vf[kBf16 ? 1 : 8][kDB];
  // The table's entry of token lane & 31 as it is, checked when it is used: a check would wait for it, and for
  // the keys and values asked for before it.
  const int32_t* const table = a.cache.table + (int64_t)i * a.cache.max_pages;
  auto entry_at = [&](int32_t n) -> int32_t {
    const int32_t s = start(n) + (lane & (kTile - 1)), k = s >> a.cache.page_log2;
    return n < w_hi && (kWholePages || held(s)) && k < a.cache.max_pages ? table[k] : -1;
  };
  auto page_of = [&](int32_t entry) { return entry >= 0 && entry < a.cache.n_pages ? entry : -1; };
  constexpr int kLine = D * E::kBytes;
  // the lane's byte offsets within 16 tokens' rows
  const uint32_t k_off = col * kLine + 16 * g;
  constexpr int kLanes = D / 8, kRows = kWave / kLanes;  // lanes of a bf16 value row, rows of one load
  const uint32_t v_off = (lane / kLanes) * kLine + (lane % kLanes) * 16;
  // Keys and values of a tile are asked for separately, each as soon as the registers of the tile before are free.
  auto load_keys = [&](int32_t n, int32_t page) {
    const int32_t s0 = start(n);
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      const char* src;
      if constexpr (kWholePages) {
        const int32_t p = lane_value(page, 16 * blk);
        src = a.cache.keys + a.cache.row(p < 0 ? 0 : p, head, s0 + 16 * blk) * kLine + k_off;
      } else {
        const int32_t p = __shfl(page, 16 * blk + col);
        src = a.cache.keys + a.cache.row(p < 0 ? 0 : p, head, s0 + 16 * blk + col) * kLine + 16 * g;
      }
#pragma unroll
      for (int s = 0; s < kSteps; ++s) kreg[blk][s] = *reinterpret_cast<const u32x4*>(src + 64 * s);
    }
  };
  auto load_values = [&](int32_t n, int32_t page) {
    const int32_t s0 = start(n);
    if constexpr (kBf16) {
      if constexpr (kWholePages) {
#pragma unroll
        for (int blk = 0; blk < 2; ++blk) {
          const int32_t p = lane_value(page, 16 * blk);
          const char* vs = a.cache.values + a.cache.row(p < 0 ? 0 : p, head, s0 + 16 * blk) * kLine + v_off;
#pragma unroll
          for (int x = 0; x < D / 32; ++x)
            vreg[blk * (D / 32) + x] = *reinterpret_cast<const u32x4*>(vs + x * kRows * kLine);
        }
      } else {
#pragma unroll
        for (int x = 0; x < D / 16; ++x) {
          const int k = x * kRows + lane / kLanes;
          const int32_t p = __shfl(page, k);
          vreg[x] = *reinterpret_cast<const u32x4*>(a.cache.values +
                                                    a.cache.row(p < 0 ? 0 : p, head, s0 + k) * kLine +
                                                    (lane % kLanes) * 16);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int k = 16 * (e >> 2) + 4 * g + (e & 3);
        const int32_t p = __shfl(page, k);
        const char* src = a.cache.values + a.cache.row(p < 0 ? 0 : p, head, s0 + k) * kLine + col * 4;
#pragma unroll
        for (int d = 0; d < kDB; ++d) vf[e][d] = *reinterpret_cast<const float*>(src + d * 64);
      }
    }
  };

  int32_t n = w_lo + wave;
  // the pages of two tiles ahead: a page read behind a tile's loads would wait for them
  int32_t page = page_of(entry_at(n)), entry_1 = entry_at(n + kWaves);
  if (n < w_hi) {
    load_keys(n, page);
    load_values(n, page);
  }
  for (; n < w_hi; n += kWaves) {
    const int32_t s0 = start(n);
    const int32_t page_1 = page_of(entry_1);
    entry_1 = entry_at(n + 2 * kWaves);
    // a value no row sees is 0: what lies there may be NaN
    const uint32_t there = (uint32_t)__ballot(page >= 0 && held(s0 + (lane & (kTile - 1))));  // bit k: token s0 + k
    const bool paged = there == ~0u;
    const bool more = n + kWaves < w_hi;
    f32x4 sc[QB][2];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        sc[b][blk] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          if constexpr (kBf16) {
            sc[b][blk] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kreg[blk][s]),
                                                                  __builtin_bit_cast(bf16x8, q[b][s]), sc[b][blk], 0, 0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sc[b][blk] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(kreg[blk][s][e]),
                                                                __uint_as_float(q[b][s][e]), sc[b][blk], 0, 0, 0);
          }
        }
      }
    }
    if (more) load_keys(n + kWaves, page_1);
    if constexpr (kBf16) {
      if (!paged) {
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          if (!((there >> (x * kRows + lane / kLanes)) & 1)) vreg[x].x = vreg[x].y = vreg[x].z = vreg[x].w = 0;
      }
      if (!all_see(s0)) {
        bool bad = false;
#pragma unroll
        for (int x = 0; x < D / 16; ++x) bad |= not_finite(vreg[x]);
        if (__any(bad)) {
          odd = true;
#pragma unroll
          for (int x = 0; x < D / 16; ++x) vreg[x] = finite_of(vreg[x]);
        }
      }
#pragma unroll
      for (int x = 0; x < D / 16; ++x)
        *reinterpret_cast<u32x4*>(v_lds + (x * kRows + lane / kLanes) * S::kValueStride + (lane % kLanes) * 16) = vreg[x];
      if (more) load_values(n + kWaves, page_1);
    }

    const bool whole = paged && all_see(s0);  // no masks
    bf16x8 pb[QB];
    float pf[QB][8];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      if (!whole) {
        // bit k: the column sees token s0 + k
        auto below = [&](int32_t s) { return s - s0 >= kTile ? ~0u : (s > s0 ? (1u << (s - s0)) - 1 : 0u); };
        uint32_t see = a.window ? ~below(pos[b] - a.window + 1) | below(a.sinks) : ~0u;
        if (!a.parents) {
          see &= below(pos[b] + 1);
        } else {  // the cached slots, then the row's own path
          const int32_t d = len - s0;  // the tile's token of row 0
          see &= below(len);
          if (d < kTile)
            see |= d >= 0 ? (uint32_t)(sight[b].rows << d)
                          : (d > -64 ? (uint32_t)(sight[b].rows >> -d) : 0u) |
                                (sight[b].last && -d > 32 && -d <= 64 ? 1u << (64 + d) : 0u);
        }
        see = live[b] ? (see & there) >> (4 * g) : 0u;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (!((see >> (16 * (e >> 2) + (e & 3))) & 1)) sc[b][e >> 2][e & 3] = -__builtin_inff();
      }
      const f32x4 y = sc[b][0], z = sc[b][1];
      float top = fmaxf(fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3])), fmaxf(fmaxf(z[0], z[1]), fmaxf(z[2], z[3])));
      top = both_max16_32(top) * a.scale2;
      // The frame follows the maximum only when a weight would pass 2^8: the sums have room for that, and they
      // are not rescaled for each small step up.
      if (__any(top > m[b] + 8.0f)) {
        const float next = fmaxf(m[b], top);
        const float keep = next == -__builtin_inff() ? 1.0f : fast_exp2(m[b] - next);
        m[b] = next;
        l[b] *= keep;
#pragma unroll
        for (int d = 0; d < kDB; ++d) acc[b][d] *= keep;
      }
      const float frame = m[b] == -__builtin_inff() ? 0.0f : m[b];
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float p = fast_exp2(fmaf(sc[b][e >> 2][e & 3], a.scale2, -frame));
        sum += p;
        if constexpr (kBf16)
          pb[b][e] = (__bf16)p;
        else
          pf[b][e] = p;
      }
      l[b] += sum;
    }
    if constexpr (kBf16) {
      __builtin_amdgcn_wave_barrier();
      // lane (g, col) supplies 8 bytes of token 4 g + col / 4; the read hands it four tokens of its column
      const char* src = v_lds + (4 * g + (col >> 2)) * S::kValueStride + (col & 3) * 8;
#pragma unroll
      for (int d = 0; d < kDB; ++d) {
        typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
        const bf16x4 v0 = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(src + d * 32));
        const bf16x4 v1 = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(src + d * 32 + 16 * S::kValueStride));
        const bf16x8 v = __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7);
#pragma unroll
        for (int b = 0; b < QB; ++b)
          acc[b][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, pb[b], acc[b][d], 0, 0, 0);
      }
      __builtin_amdgcn_wave_barrier();
    } else {
      if (!paged) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool held_e = (there >> (16 * (e >> 2) + 4 * g + (e & 3))) & 1;
#pragma unroll
          for (int d = 0; d < kDB; ++d) vf[e][d] = held_e ? vf[e][d] : 0.0f;
        }
      }
      if (!all_see(s0)) {
        float none = 0.0f;  // stays 0 over finite values
#pragma unroll
        for (int e = 0; e < 8; ++e)
#pragma unroll
          for (int d = 0; d < kDB; ++d) none = fmaf(vf[e][d], 0.0f, none);
        if (__any(!(none == 0.0f))) {
          odd = true;
#pragma unroll
          for (int e = 0; e < 8; ++e)
#pragma unroll
            for (int d = 0; d < kDB; ++d) vf[e][d] = vf[e][d] - vf[e][d] == 0.0f ? vf[e][d] : 0.0f;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int d = 0; d < kDB; ++d)
#pragma unroll
          for (int b = 0; b < QB; ++b)
            acc[b][d] = __builtin_amdgcn_mfma_f32_16x16x4f32(vf[e][d], pf[b][e], acc[b][d], 0, 0, 0);
      if (more) load_values(n + kWaves, page_1);
    }
    page = page_1;
  }

  // the four waves' sums in one frame
  __syncthreads();
  odd = __any(odd);
  if (lane == 0) sh.odd_s[wave] = odd;
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    l[b] = both_sum16_32(l[b]);
    if (g == 0) {
      m_s[wave][16 * b + col] = m[b];
      l_s[wave][16 * b + col] = l[b];
    }
  }
  __syncthreads();
  float* const merge = reinterpret_cast<float*>(smem);
  float top[QB], sum[QB];
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    const int c = 16 * b + col;
    top[b] = m_s[0][c];
    for (int w = 1; w < kWaves; ++w) top[b] = fmaxf(top[b], m_s[w][c]);
    const float frame = top[b] == -__builtin_inff() ? 0.0f : top[b];
    sum[b] = 0.0f;
    for (int w = 0; w < kWaves; ++w) sum[b] += l_s[w][c] * fast_exp2(m_s[w][c] - frame);
    const float fade = fast_exp2(m[b] - frame);
#pragma unroll
    for (int d = 0; d < kDB; ++d) acc[b][d] *= fade;
  }
#pragma unroll
  for (int half = kWaves / 2; half > 0; half /= 2) {
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int b = 0; b < QB; ++b)
#pragma unroll
        for (int d = 0; d < kDB; ++d)
          *reinterpret_cast<f32x4*>(merge + ((wave - half) * S::kColumns + 16 * b + col) * S::kMergeStride + 16 * d +
                                    4 * g) = acc[b][d];
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int b = 0; b < QB; ++b)
#pragma unroll
        for (int d = 0; d < kDB; ++d)
          acc[b][d] += *reinterpret_cast<const f32x4*>(merge + (wave * S::kColumns + 16 * b + col) * S::kMergeStride +
                                                       16 * d + 4 * g);
    }
    __syncthreads();
  }
  if (wave != 0) return;
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    const int32_t c = at.c0 + 16 * b + col;
    if (c >= columns) continue;
    const int32_t j = (uint32_t)c / (uint32_t)a.G;
    if (slot >= 0) {
      const int64_t u = slot * S::kColumns + 16 * b + col;
      if (g == 0) {
        a.stats[2 * u] = top[b];
        a.stats[2 * u + 1] = sum[b];
      }
#pragma unroll
      for (int d = 0; d < kDB; ++d) *reinterpret_cast<f32x4*>(a.part + u * D + 16 * d + 4 * g) = acc[b][d];
    } else {
      const int32_t h = head * a.G + (c - j * a.G);
      const float inv = sum[b] > 0.0f ? 1.0f / sum[b] : 0.0f;
      char* dst = a.out + ((at.r.row0 + j) * a.n_q + h) * (D * E::kBytes) + 4 * g * E::kBytes;
#pragma unroll
      for (int d = 0; d < kDB; ++d) {
        const f32x4 o = acc[b][d] * inv;
        if constexpr (kBf16) {
          bf16x4 w;
          for (int e = 0; e < 4; ++e) w[e] = (__bf16)o[e];
          *reinterpret_cast<bf16x4*>(dst + d * 32) = w;
        } else {
          *reinterpret_cast<f32x4*>(dst + d * 64) = o;
        }
      }
    }
  }
  for (int w = 1; w < kWaves; ++w) odd |= sh.odd_s[w] != 0;
  if (odd) {
    auto row_of = [&](int32_t c) { return (int32_t)((uint32_t)(at.c0 + c) / (uint32_t)a.G); };
    add_not_finite<E, D, kTile>(
        a, i, head, w_lo, w_hi, c_last - at.c0 + 1, start, all_see,
        [&](int32_t c, int32_t s) {
          const int32_t j = row_of(c), pos_c = len + (a.parents ? depth_s[j] : j);
          if (a.parents && s >= len) {
            const int32_t r = s - len;
            return r < 64 ? ((sight_s[j] >> r) & 1) != 0 : r == 64 && last_s[j] != 0;
          }
          return s <= pos_c && (a.window == 0 || s > pos_c - a.window || s < a.sinks);
        },
        [&](int32_t c, int d, float v) {
          const int32_t j = row_of(c), h = head * a.G + (at.c0 + c - j * a.G);
          if (slot >= 0)
            a.part[(slot * S::kColumns + c) * D + d] += v;
          else
            add_to<E>(a.out + ((at.r.row0 + j) * a.n_q + h) * (D * E::kBytes), d, v);
        });
  }
}

// Two waves per SIMD hide each other's loads; sums of 64 columns, or of 256 values, take the registers of both.
template <class E, int D, int QB>
constexpr int kMinWaves = E::kBytes == 4 ? (D <= 128 ? 2 : 1) : (D * QB <= 256 ? 2 : 1);

// A workgroup per unit.
template <class E, int D, int QB, int kWaves, bool kWholePages>
__global__ __launch_bounds__(kWaves* kWave, (kMinWaves<E, D, QB>)) void attend_units(AttendArgs a) {
  __shared__ Scratch<E, D, QB, kWaves> sh;
  const int64_t block = unit_of_block(blockIdx.x, gridDim.x);
  const TileOf at = tile_of<16 * QB>(a, block / a.cache.n_heads);
  if (at.r.index < 0) return;
  attend_unit<E, D, QB, kWaves, kWholePages>(a, sh, at, a.cache.len[at.r.index], (int32_t)(block % a.cache.n_heads),
                                             false, 0, 0, -1);
}

// A workgroup per range of the batch's work.
constexpr int kStreamWaves = 4;
template <class E, int D, int QB>
__global__ __launch_bounds__(kStreamWaves* kWave, (kMinWaves<E, D, QB>)) void attend_ranges(AttendArgs a) {
  constexpr int kColumns = 16 * QB;
  __shared__ Scratch<E, D, QB, kStreamWaves> sh;
  const Stream s = stream_of(a, kColumns);
  const int64_t range = unit_of_block(blockIdx.x, gridDim.x);
  const int64_t end = (range + 1) * s.length < s.total ? (range + 1) * s.length : s.total;
  int64_t p = range * s.length;
  if (p >= end) return;
  // the request of p, then on from one to the next
  const int who = 63 - __builtin_clzll(__ballot(s.before <= p));
  int32_t i = who * s.per;
  int64_t base = (int64_t)lane_value((uint64_t)s.before, who);
  while (p < end && i < a.B) {
    const Work w = work_at(a, s, i, kColumns);
    const int64_t items = w.units(a) * w.n;
    if (p >= base + items) {
      base += items;
      ++i;
      continue;
    }
    const uint32_t unit = (uint32_t)((p - base) / w.n);
    const int32_t q_lo = (int32_t)(p - base - (int64_t)unit * w.n);
    const int32_t q_hi = q_lo + (end - p) < w.n ? (int32_t)(q_lo + (end - p)) : w.n;
    TileOf at;
    at.r = request_with(w, i);
    at.c0 = (int32_t)(unit / (uint32_t)a.cache.n_heads) * kColumns;
    const bool first = q_lo == 0, whole = first && q_hi == w.n;
    attend_unit<E, D, QB, kStreamWaves, true>(a, sh, at, w.len, (int32_t)(unit % (uint32_t)a.cache.n_heads), true,
                                              q_lo, q_hi,
                                              whole ? -1 : 2 * range + (first ? 1 : 0));
    p += q_hi - q_lo;
    __syncthreads();
  }
}

// Joins the pieces of the units that ranges cut.  A workgroup takes kJoin columns of a unit, or, where a
// unit is cut into many pieces (few units, long caches), one column whose pieces its waves share.  Lane k of
// D / 4 holds four values of a column; the wave's other lanes hold the same of further pieces.
constexpr int kJoinWaves = 4;
constexpr int kJoin = 8;

template <class E, int D, int QB, bool kMany>
__global__ __launch_bounds__(kJoinWaves* kWave) void join(AttendArgs a) {
  constexpr int kColumns = 16 * QB, kLanes = D / 4, kRows = kWave / kLanes;  // pieces a wave reads at once
  __shared__ float o_s[kJoinWaves][D], stat_s[kJoinWaves][2];
  const int t = threadIdx.x, lane = t & (kWave - 1), k = lane % kLanes;
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const Stream s = stream_of(a, kColumns);
  const int64_t u = blockIdx.x;
  const int who = 63 - __builtin_clzll(__ballot(s.units_before <= u));
  int64_t begin = (int64_t)lane_value((uint64_t)s.before, who);
  int64_t unit = u - (int64_t)lane_value((uint64_t)s.units_before, who);
  int32_t i = who * s.per;
  Work w;
  for (;; ++i) {
    if (i >= a.B) return;
    w = work_at(a, s, i, kColumns);
    if (unit < w.units(a)) break;
    unit -= w.units(a);
    begin += w.units(a) * w.n;
  }
  begin += unit * w.n;
  const int64_t r_lo = begin / s.length;
  const int32_t pieces = (int32_t)((begin + w.n - 1) / s.length - r_lo) + 1;
  if (pieces == 1) return;
  const Request r = request_with(w, i);
  const int32_t head = (uint32_t)unit % (uint32_t)a.cache.n_heads;
  const int32_t c0 = (int32_t)((uint32_t)unit / (uint32_t)a.cache.n_heads) * kColumns, columns = (r.k + 1) * a.G;
  // the piece with the unit's first tile is its range's second, the others their ranges' first
  auto at = [&](int32_t piece) { return (2 * (r_lo + piece) + (piece == 0 ? 1 : 0)) * kColumns; };
  const int x_lo = blockIdx.y * (kMany ? 1 : kJoin), x_hi = x_lo + (kMany ? 1 : kJoin);
  for (int x = x_lo + (kMany ? 0 : wave); x < x_hi; x += kMany ? 1 : kJoinWaves) {
    const int32_t c = c0 + x;
    if (c >= columns) break;
    // this wave's pieces: all of them, or every kJoinWaves-th 64
    float top = -__builtin_inff(), sum = 0.0f;
    f32x4 o = f32x4{0, 0, 0, 0};
    for (int32_t p0 = kMany ? wave * kWave : 0; p0 < pieces; p0 += kMany ? kJoinWaves * kWave : kWave) {
      const int32_t p = p0 + lane;
      float m = -__builtin_inff(), l = 0.0f;
      if (p < pieces) {
        m = a.stats[2 * (at(p) + x)];
        l = a.stats[2 * (at(p) + x) + 1];
      }
      const float next = fmaxf(top, wave_max(m)), frame = next == -__builtin_inff() ? 0.0f : next;
      const float fade = fast_exp2(top - frame), scale = fast_exp2(m - frame);
      top = next;
      sum = sum * fade + wave_sum(l * scale);
      o *= fade;
      const int32_t n = pieces - p0 < kWave ? pieces - p0 : kWave;
#pragma unroll 4
      for (int32_t q = 0; q < n; q += kRows) {
        const int32_t mine = q + lane / kLanes;
        const float f = __shfl(scale, mine & (kWave - 1));
        if (mine < n) o += *reinterpret_cast<const f32x4*>(a.part + (at(p0 + mine) + x) * D + 4 * k) * f;
      }
    }
    if constexpr (kRows > 1) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
#pragma unroll
        for (int step = kLanes; step < kWave; step *= 2) o[e] += __shfl_xor(o[e], step);
      }
    }
    if constexpr (kMany) {
      if (lane < kLanes) *reinterpret_cast<f32x4*>(&o_s[wave][4 * k]) = o;
      if (lane == 0) {
        stat_s[wave][0] = top;
        stat_s[wave][1] = sum;
      }
      __syncthreads();
      if (wave != 0) return;
      top = -__builtin_inff();
      for (int v = 0; v < kJoinWaves; ++v) top = fmaxf(top, stat_s[v][0]);
      const float frame = top == -__builtin_inff() ? 0.0f : top;
      sum = 0.0f;
      o = f32x4{0, 0, 0, 0};
      for (int v = 0; v < kJoinWaves; ++v) {
        const float f = fast_exp2(stat_s[v][0] - frame);
        sum += stat_s[v][1] * f;
        o += *reinterpret_cast<const f32x4*>(&o_s[v][4 * k]) * f;
      }
    }
    if (lane >= kLanes) continue;
    o *= sum > 0.0f ? 1.0f / sum : 0.0f;
    const int32_t j = (uint32_t)c / (uint32_t)a.G, h = head * a.G + (c - j * a.G);
    char* dst = a.out + ((r.row0 + j) * a.n_q + h) * (D * E::kBytes) + k * 4 * E::kBytes;
    if constexpr (E::kBytes == 2) {
      bf16x4 v;
      for (int e = 0; e < 4; ++e) v[e] = (__bf16)o[e];
      *reinterpret_cast<bf16x4*>(dst) = v;
    } else {
      *reinterpret_cast<f32x4*>(dst) = o;
    }
  }
}

// Many rows per request (prompts), bf16, linear: products bound the call (16 x 2501 rows on 4000 tokens 970 to 1024 TF/s, near
// a large library product; under a window of 1024 650 TF/s, where the 8 to 10 us in which a workgroup finds its pages,
// loads its queries and stores its results weigh, and tiles at the window's ends are cut).  A workgroup takes 128 columns, a
// wave 32 of them, and the waves share the keys and values of 64 tokens through shared memory, where direct loads
// put the next 64 meanwhile.  Matrix instructions of 32 x 32 x 16; per tile and wave 32 of them (1024
// cycles at D = 128) against 32 KiB of shared-memory reads.  The scores of the next tile are computed between the
// exponentials of this one, whose cycles they fill: without, two waves per SIMD wait for each other (954 TF/s at
// the same shape).
//
// A row of a tile keeps its 16-byte pieces in the order p ^ 2 (token mod 8) (for D = 64, of 8 pieces, p ^ 2 (token
// / 2 mod 4)): the 32 rows that a key read takes, and the 8 that a transposing value read takes, then lie in
// different banks.  A direct load writes its lanes' 16 bytes in lane order, so the permutation is in the addresses
// that the lanes read from.
typedef float f32x16 __attribute__((ext_vector_type(16)));
constexpr int kRowsWaves = 4;
constexpr int kRowsTile = 64;
constexpr int kRowsColumns = 32 * kRowsWaves;

template <int D>
__device__ __forceinline__ int piece_of(int token, int p) {
  return D == 128 ? p ^ (2 * (token & 7)) : p ^ (2 * ((token >> 1) & 3));
}

// 16 bytes per lane from base + off to to + 16 lane, past the registers.  As a buffer load: a load by flat address that
// writes shared memory counts as a flat one, and while one is in flight every wait for a read of shared memory is a
// wait for all of them.
__device__ __forceinline__ void direct_load(const char* base, int32_t bytes, uint32_t off, char* to) {
  constexpr int kRaw = 0x27000;  // last word of the buffer's description: bytes, no stride
  __builtin_amdgcn_raw_ptr_buffer_load_lds(__builtin_amdgcn_make_buffer_rsrc((void*)base, 0, bytes, kRaw),
                                           (__attribute__((address_space(3))) void*)to, 16, off, 0, 0, 0);
}

template <int D>
__global__ __launch_bounds__(kRowsWaves* kWave, 2) void attend_rows(AttendArgs a) {
  constexpr int kLine = D * 2, kPieces = D / 8, kSteps = D / 16, kDB = D / 32;
  constexpr int kLoadRows = kWave / kPieces;       // rows of one direct load
  constexpr int kLoads = 16 / kLoadRows;           // of a wave's 16 rows
  constexpr int kKeys = 6;                         // keys' operands in flight
  // arrays of their own: reads of one tile do not wait for the loads into the other
  __shared__ __align__(16) char k_0[kRowsTile * kLine], k_1[kRowsTile * kLine];
  __shared__ __align__(16) char v_0[kRowsTile * kLine], v_1[kRowsTile * kLine];
  const int t = threadIdx.x, lane = t & (kWave - 1), col = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  // head by head, the last tiles (of the longest rows) first
  const uint32_t unit = (uint32_t)unit_of_block(blockIdx.x, gridDim.x), tiles = (uint32_t)a.tiles;
  const int32_t head = (int32_t)(unit / tiles);
  const int64_t tile_no = tiles - 1 - (unit - head * tiles);
  // one value in all lanes: kept in scalar registers
  auto all = [](int32_t x) { return __builtin_amdgcn_readfirstlane(x); };
  // tile_of, with the lengths loaded beside the offsets, 64 requests at a time: a workgroup has nothing to do until
  // its pages are known, so each load behind another counts
  TileOf at;
  int32_t len;
  {
    const int32_t i0 =
        a.B <= kWave ? 0 : find_last(a.B, tile_no, [&](int32_t q) { return first_tile(a.cu, q, a.G, kRowsColumns); });
    const bool in = i0 >= 0 && i0 + lane < a.B;
    const int32_t mine = in ? i0 + lane : a.B - 1;
    const int32_t lo = a.cu[mine], hi = a.cu[mine + 1], n = a.cache.len[mine];
    const int64_t first = (uint32_t)(lo + mine) * (uint32_t)a.G / (uint32_t)kRowsColumns + mine;  // first_tile
    const uint64_t who = __ballot(in && first <= tile_no);
    const int src = who && a.B <= kWave ? 63 - __builtin_clzll(who) : 0;
    int32_t begin = lane_value(lo, src), behind = lane_value(hi, src);
    int64_t tile_0 = (int64_t)lane_value((uint64_t)first, src);
    at.r.index = i0 + src;
    len = lane_value(n, src);
    if (__builtin_expect(!who || (who & (who + 1)) || begin < 0 || behind < begin || behind > a.n_d, 0)) {
      at.r.index = tile_among<kRowsColumns>(a, tile_no);  // some offsets are not valid
      if (at.r.index < 0) return;
      begin = all(a.cu[at.r.index]);
      behind = all(a.cu[at.r.index + 1]);
      tile_0 = all((int32_t)first_tile(a.cu, at.r.index, a.G, kRowsColumns));
      len = all(a.cache.len[at.r.index]);
    }
    at.r.first = begin;
    at.r.k = behind - begin;
    at.r.row0 = (int64_t)begin + at.r.index;
    const int64_t c0 = (tile_no - tile_0) * kRowsColumns;
    if (c0 >= (int64_t)(at.r.k + 1) * a.G) return;
    at.c0 = (int32_t)c0;
  }
  const int32_t i = at.r.index;
  const bool ok = len_fits(len, at.r.k);
  const int32_t columns = (at.r.k + 1) * a.G;
  const int32_t c_end = at.c0 + kRowsColumns < columns ? at.c0 + kRowsColumns : columns;
  Span span = span_of(len, (uint32_t)at.c0 / (uint32_t)a.G, (uint32_t)(c_end - 1) / (uint32_t)a.G, a.window, a.sinks);
  span.lo = all(span.lo);
  span.hi = all(span.hi);
  span.near_end = all(span.near_end);
  // tiles of 64 tokens over [0, near_end) and [lo, hi)
  int32_t t_lo = span.lo / kRowsTile, n_near = (span.near_end + kRowsTile - 1) / kRowsTile;
  if (t_lo <= n_near) t_lo = n_near = 0;
  const int32_t n_tiles = ok ? n_near + (span.hi + kRowsTile - 1) / kRowsTile - t_lo : 0;
  auto start = [&](int32_t n) { return (n < n_near ? n : n - n_near + t_lo) * kRowsTile; };

  // the wave's columns
  const int32_t c = at.c0 + 32 * wave + col;
  const bool live = c < columns;
  const int32_t j = (uint32_t)(live ? c : columns - 1) / (uint32_t)a.G;
  const int32_t h = head * a.G + (live ? c - j * a.G : 0);
  const int32_t pos = len + j;
  const int32_t pos_lo = lane_value(pos, 0), pos_hi = lane_value(pos, 31);  // ascending over the columns

  // Rows 16 wave .. of a tile are the wave's to load: one page.
  uint32_t off[kLoads];
#pragma unroll
  for (int x = 0; x < kLoads; ++x) {
    const int row = x * kLoadRows + lane / kPieces;
    off[x] = row * kLine + piece_of<D>(row, lane % kPieces) * 16;
  }
  // The table's entry as it is, checked when it is used: a check would wait for it, and for the direct loads before it.
  const int32_t* const table = a.cache.table + (int64_t)i * a.cache.max_pages;
  auto entry_at = [&](int32_t n) {
    const int32_t k = (start(n) + 16 * wave) >> a.cache.page_log2;
    return n < n_tiles && k < a.cache.max_pages ? table[k] : -1;
  };
  auto page_of = [&](int32_t entry) {
    const int32_t p = __builtin_amdgcn_readfirstlane(entry);
    return p >= 0 && p < a.cache.n_pages ? p : -1;
  };
  auto load = [&](const char* from, int32_t n, int32_t page, char* to) {
    const int64_t at_row = a.cache.row(page < 0 ? 0 : page, head, start(n) + 16 * wave) * kLine;
    from += ((int64_t)all((int32_t)(at_row >> 32)) << 32) | (uint32_t)all((int32_t)at_row);
    to += 16 * wave * kLine;
#pragma unroll
    for (int x = 0; x < kLoads; ++x) direct_load(from, 16 * kLine, off[x], to + x * 1024);
  };

  const int32_t entry_0 = entry_at(0), entry_1 = entry_at(1);
  int32_t entry_2 = entry_at(2);
  // The wave's queries and results pass through shared memory, where they change between a column per lane and whole
  // lines (16-byte pieces of 32 columns took 2 to 3 us of a workgroup's time each way): one array holds the
  // first halves of its 32 columns, another the second halves, each in the place of the wave's 16 rows of a tile.
  constexpr int kHalf = kPieces / 2;                // pieces of half a column
  constexpr int kQLoads = 32 * kHalf / kWave;
  auto half_piece = [](int column, int p) { return 16 * (column * kHalf + (p ^ (column & (kHalf - 1)))); };
  auto column_of = [&](int x) { return x * (kWave / kHalf) + lane / kHalf; };
  auto from_lane = [](int64_t v, int src) {
    return ((int64_t)__shfl((int32_t)(v >> 32), src) << 32) | (uint32_t)__shfl((int32_t)v, src);
  };
  {
    typedef __attribute__((address_space(3))) void* Lds;
    typedef const __attribute__((address_space(1))) void* Global;
    const int64_t q_at = ((at.r.row0 + j) * a.query_stride + (int64_t)h * D) * 2;
#pragma unroll
    for (int x = 0; x < kQLoads; ++x) {
      const int column = column_of(x);
      const char* const src = a.queries + from_lane(q_at, column) + 16 * ((lane % kHalf) ^ (column & (kHalf - 1)));
      __builtin_amdgcn_global_load_lds((Global)src, (Lds)(k_1 + 16 * wave * kLine + x * 1024), 16, 0, 0);
      __builtin_amdgcn_global_load_lds((Global)(src + 16 * kHalf), (Lds)(v_1 + 16 * wave * kLine + x * 1024), 16, 0, 0);
    }
  }
  int32_t page = page_of(entry_0), page_1 = page_of(entry_1);
  if (n_tiles > 0) {
    load(a.cache.keys, 0, page, k_0);
    load(a.cache.values, 0, page, v_0);
  }
  bf16x8 q[kSteps];

  f32x16 acc[kDB];
#pragma unroll
  for (int d = 0; d < kDB; ++d)
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[d][e] = 0.0f;
  float m = -__builtin_inff(), l = 0.0f;
  __shared__ __align__(16) int32_t page_s[2][kRowsWaves];
  __shared__ int32_t odd_s;
  if (t == 0) odd_s = 0;
  const int32_t first_pos = len + (int32_t)((uint32_t)at.c0 / (uint32_t)a.G);
  const int32_t last_pos = len + (int32_t)((uint32_t)(c_end - 1) / (uint32_t)a.G);
  auto all_see = [&](int32_t s0) {
    return s0 + kRowsTile <= first_pos + 1 && (a.window == 0 || s0 > last_pos - a.window || s0 + kRowsTile <= a.sinks);
  };

  typedef f32x16 Scores[2];  // element e of a block: token 8 (e / 4) + 4 half + e mod 4
  const f32x16 none16 = {};
  auto key = [&](const char* k_s, int blk, int s) {
    const int token = 32 * blk + col;
    return *reinterpret_cast<const bf16x8*>(k_s + token * kLine + piece_of<D>(token, 2 * s + half) * 16);
  };
  // values of step s: tokens 16 s + 4 half + 0 .. 3 and 8 further; a 16-lane group reads 4 tokens x 16 values
  auto value = [&](char* v_s, int s, bf16x4 (&v)[kDB][2]) {
    typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
    const int g = (lane >> 4) & 1, in = lane & 15, token = 16 * s + 4 * half + (in >> 2);
#pragma unroll
    for (int d = 0; d < kDB; ++d) {
      const int pc = 4 * d + 2 * g + ((in >> 1) & 1);
      char* const r0 = v_s + token * kLine + piece_of<D>(token, pc) * 16 + (in & 1) * 8;
      char* const r1 = v_s + (token + 8) * kLine + piece_of<D>(token + 8, pc) * 16 + (in & 1) * 8;
      v[d][0] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)r0);
      v[d][1] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)r1);
    }
  };
  const int32_t near = a.window ? pos - a.window : -1;  // slots above it are seen, and the first `sinks`

  // Tile n's softmax and product with its values, the next tile's scores under the softmax (behind the last tile those
  // of what its buffer holds, which nothing uses).
  auto tile = [&](int32_t n, Scores& sc, Scores& ahead, char* k_s, char* v_s, char* k_next, char* v_next) {
    const int32_t s0 = start(n);
    // a value no row sees is 0: what lies there may be NaN
    const int32_t first = s0 + 16 * wave;
    const bool held = page >= 0 && (first + 16 <= span.near_end || (first >= span.lo && first + 16 <= span.hi));
    if (!held) {
      __builtin_amdgcn_s_waitcnt(0);
      const int row = lane >> 2;  // 4 lanes of a row
      const int32_t s = first + row;
      if (page < 0 || !(s < span.near_end || (s >= span.lo && s < span.hi))) {
        u32x4 z;
        z.x = z.y = z.z = z.w = 0;
        char* const to = v_s + (16 * wave + row) * kLine;
#pragma unroll
        for (int x = 0; x < kPieces / 4; ++x) *reinterpret_cast<u32x4*>(to + ((lane & 3) + 4 * x) * 16) = z;
      }
    }
    if (lane == 0) page_s[n & 1][wave] = page;
    __builtin_amdgcn_s_waitcnt(0x0f70);  // this wave's direct loads
    if (!all_see(s0)) {
      u32x4* const mine = reinterpret_cast<u32x4*>(v_s + 16 * wave * kLine) + lane;
      bool bad = false;
#pragma unroll
      for (int x = 0; x < kLoads; ++x) bad |= not_finite(mine[64 * x]);
      if (__any(bad)) {
        for (int x = 0; x < kLoads; ++x) mine[64 * x] = finite_of(mine[64 * x]);
        odd_s = 1;
      }
    }
    __syncthreads();  // its values and the next keys are there, and every wave is done with the other buffers
    const int4 pages = *reinterpret_cast<const int4*>(page_s[n & 1]);
    bf16x8 kf[kKeys];
#pragma unroll
    for (int f = 0; f < kKeys; ++f) kf[f] = key(k_s, f / kSteps, f % kSteps);
    page = page_1;
    page_1 = page_of(entry_2);
    if (n + 1 < n_tiles) load(a.cache.values, n + 1, page, v_next);
    if (n + 2 < n_tiles) load(a.cache.keys, n + 2, page_1, k_next);
    entry_2 = entry_at(n + 3);
    bool whole = s0 + kRowsTile <= pos_lo + 1 && (a.window == 0 || s0 > pos_hi - a.window || s0 + kRowsTile <= a.sinks);
    const int missing = pages.x | pages.y | pages.z | pages.w;  // negative: one of the four pages is none
    whole = whole && missing >= 0;
    if (!whole) {
      // the tile's tokens that the column sees, a bit each
      auto below = [&](int32_t x) { return x - s0 >= 64 ? ~0ull : (x > s0 ? (1ull << (x - s0)) - 1 : 0ull); };
      uint64_t see = below(pos + 1) & (~below(near + 1) | below(a.sinks));
      see &= (pages.x < 0 ? 0 : 0xffffull) | (pages.y < 0 ? 0 : 0xffffull << 16) | (pages.z < 0 ? 0 : 0xffffull << 32) |
             (pages.w < 0 ? 0 : 0xffffull << 48);
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const uint32_t hide = (uint32_t)~see >> (4 * half);
        see >>= 32;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          sc[blk][e] = hide & (1u << (8 * (e >> 2) + (e & 3))) ? -__builtin_inff() : sc[blk][e];
        }
      }
    }
    float top = sc[0][0];
#pragma unroll
    for (int blk = 0; blk < 2; ++blk)
#pragma unroll
      for (int e = 0; e < 16; ++e) top = fmaxf(top, sc[blk][e]);
    {
      float x, y;
      wave_detail::both<32>(top, x, y);
      top = fmaxf(x, y) * a.scale2;
    }
    // The frame follows the maximum only when a weight would pass 2^8: the sums have room for that, and 64 of them
    // are not rescaled for each small step up.
    if (__any(top > m + 8.0f)) {
      const float next = fmaxf(m, top);
      const float fade = fast_exp2(m - next);  // 0 from -inf; a column that saw nothing yet keeps -inf
      const float keep = next == -__builtin_inff() ? 1.0f : fade;
      m = next;
      l *= keep;
#pragma unroll
      for (int d = 0; d < kDB; ++d) acc[d] *= keep;
    }
    const float frame = m == -__builtin_inff() ? 0.0f : m;
    float sum = 0.0f;
    bf16x8 p[4];
    auto weigh = [&](int blk, int e) {
      const float x = fast_exp2(fmaf(sc[blk][e], a.scale2, -frame));
      sum += x;
      p[2 * blk + (e >> 3)][e & 7] = (__bf16)x;
    };
    // In the order written: a product of the next scores, then the weights that fill its cycles; operands are read
    // a block or a step ahead.
    bf16x4 vf[2][kDB][2];
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int f = 0; f < 2 * kSteps; ++f) {
      const int blk = f / kSteps, s = f % kSteps;
      ahead[blk] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[f % kKeys], q[s], s == 0 ? none16 : ahead[blk], 0, 0, 0);
      if (f + kKeys < 2 * kSteps) kf[f % kKeys] = key(k_s, (f + kKeys) / kSteps, (f + kKeys) % kSteps);
      if (f == 2 * kSteps - 4) value(v_s, 0, vf[0]);
#pragma unroll
      for (int e = 0; e < 16 / kSteps; ++e) weigh(blk, 16 / kSteps * s + e);
      __builtin_amdgcn_sched_barrier(0);
    }
    l += sum;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
#pragma unroll
      for (int d = 0; d < kDB; ++d) {
        acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
            __builtin_shufflevector(vf[s & 1][d][0], vf[s & 1][d][1], 0, 1, 2, 3, 4, 5, 6, 7), p[s], acc[d], 0, 0, 0);
        if (d == 0 && s < 3) {  // the next step's, under the rest of this one
          __builtin_amdgcn_sched_barrier(0);
          value(v_s, s + 1, vf[(s + 1) & 1]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
  };
  __builtin_amdgcn_s_waitcnt(0x0f70);  // the direct loads, of a request without tiles too: its zeros take their place
  if (n_tiles > 0) {
    Scores sc_0, sc_1;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const char* const from = (s < kSteps / 2 ? k_1 : v_1) + 16 * wave * kLine;
      q[s] = __builtin_bit_cast(
          bf16x8, *reinterpret_cast<const u32x4*>(from + half_piece(col, (2 * s) % kHalf + half)) ^ a.flip);
    }
    __syncthreads();
    if (n_tiles > 1) load(a.cache.keys, 1, page_1, k_1);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      sc_0[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key(k_0, 0, s), q[s], s == 0 ? none16 : sc_0[0], 0, 0, 0);
      sc_0[1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key(k_0, 1, s), q[s], s == 0 ? none16 : sc_0[1], 0, 0, 0);
    }
    for (int32_t n = 0; n < n_tiles; n += 2) {
      tile(n, sc_0, sc_1, k_1, v_0, k_0, v_1);
      if (n + 1 < n_tiles) tile(n + 1, sc_1, sc_0, k_0, v_1, k_1, v_0);
    }
  }
  {
    float x, y;
    wave_detail::both<32>(l, x, y);
    l = x + y;
  }
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  const int64_t out_at = ((at.r.row0 + j) * a.n_q + h) * (int64_t)kLine;
  // the buffers that the last tile's successors would have taken are free
  auto store = [&](char* first, char* second) {
    first += 16 * wave * kLine;
    second += 16 * wave * kLine;
#pragma unroll
    for (int d = 0; d < kDB; ++d)
#pragma unroll
      for (int e = 0; e < 16; e += 4) {
        bf16x4 w;
#pragma unroll
        for (int x = 0; x < 4; ++x) w[x] = (__bf16)(acc[d][e + x] * inv);
        const int piece = 4 * d + e / 4;
        *reinterpret_cast<bf16x4*>((d < kDB / 2 ? first : second) + half_piece(col, piece % kHalf) + 8 * half) = w;
      }
#pragma unroll
    for (int x = 0; x < kQLoads; ++x) {
      const int column = column_of(x);
      char* const dst = a.out + from_lane(out_at, column) + 16 * (lane % kHalf);
      const u32x4 lo = *reinterpret_cast<const u32x4*>(first + half_piece(column, lane % kHalf));
      const u32x4 hi = *reinterpret_cast<const u32x4*>(second + half_piece(column, lane % kHalf));
      if (at.c0 + 32 * wave + column >= columns) continue;
      *reinterpret_cast<u32x4*>(dst) = lo;
      *reinterpret_cast<u32x4*>(dst + 16 * kHalf) = hi;
    }
  };
  if (n_tiles & 1)
    store(k_0, v_1);
  else
    store(k_1, v_0);
  if (n_tiles > 0 && odd_s) {
    const int32_t c_lo = at.c0 + 32 * wave;
    auto row_of = [&](int32_t x) { return (int32_t)((uint32_t)(c_lo + x) / (uint32_t)a.G); };
    add_not_finite<Bf16, D, kRowsTile>(
        a, i, head, 0, n_tiles, c_end - c_lo < 32 ? c_end - c_lo : 32, start, all_see,
        [&](int32_t x, int32_t s) {
          const int32_t at_pos = len + row_of(x);
          return s <= at_pos && (a.window == 0 || s > at_pos - a.window || s < a.sinks);
        },
        [&](int32_t x, int d, float v) {
          const int32_t row = row_of(x), q_head = head * a.G + (c_lo + x - row * a.G);
          add_to<Bf16>(a.out + ((at.r.row0 + row) * a.n_q + q_head) * kLine, d, v);
        });
  }
}

enum Mode { kUnits, kRanges, kSmallPages, kRows };

// The rules, by what the host knows: the batch's mean rows, and for its lengths the page table's width (under a window, the
// window).  A table wider than the lengths need takes short caches to ranges: 16 requests of 500 tokens without a
// window 14.3 us there for 11.3 by units, 64 of them 27.6 for 24.0.  Times of 8 heads, D = 128, bf16, for one side and the other.
//
// attend_rows from this many columns of a request (its rows times the heads of a group) and this many workgroups on: 64
// requests of 96 columns on 4000 tokens 258 us for 552, 16 of 128 on 1000 29 for 36, of 64 on 4000 260 for
// 227; one request of 512 on 4000 (32 workgroups) 87 for 55.
constexpr int64_t kManyColumns = 96, kManyWorkgroups = 128;

// Ranges for units of more token tiles than this: one request on 1000 tokens 14 us either way, on 4000 17 for 42 by
// units; 16 requests (128 units) 52 for 50.  With this many units, of more than twice that: 16 trees of binary32 on 1045
// tokens 54 us by ranges, 25 by units.
constexpr int64_t kShort = 32, kSomeUnits = 64;

// Units, however long, from this many on: their rounds are even enough (256 requests on 1000 tokens 200 us for 224
// by ranges).
constexpr int64_t kManyUnits = 2048;

// Units of 16 columns up to which they are not paired (4 requests of 64 columns on 1000 tokens 16.3 us for 19.4 in
// pairs; 16 of 32 columns, 256 units, 25.4 for 20.2).  Binary32 units never are (16 of 52 columns 25 us for 35.5): the
// binary32 matrix instructions set their time, which a pair doubles.  Ranges are in pairs: they read the cache
// again for each column tile (16 of 48 columns on 4000 tokens 126 us for 58).
constexpr int64_t kFewUnits = 128;

// Workgroups at once: two per compute unit.
constexpr int64_t kPlaces = 512;

struct Plan {
  int qb;
  Mode mode;
  int32_t ranges;
  int32_t pieces;  // of a unit, about
  int64_t tiles;
  size_t part_bytes, bytes;
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
  const bool pairs = mean > 16 && !(c->dtype == SDV_FP32 && c->head_dim > 64);
  const bool split = tokens > (units_of(16) < kSomeUnits ? kShort : 2 * kShort) && B <= 512 &&
                     rows <= 64 * (int64_t)B && units_of(32) < kManyUnits;
  p.mode = c->page_size < 16 ? kSmallPages : (split ? kRanges : kUnits);
  if (pairs && (p.mode == kRanges || (c->dtype == SDV_BF16 && units_of(16) > kFewUnits))) p.qb = 2;
  p.tiles = rows * G / (16 * p.qb) + B;
  if (p.mode == kRanges) {
    const int64_t units = units_of(16 * p.qb), groups = (units * tokens + kStreamWaves - 1) / kStreamWaves;
    p.ranges = (int32_t)(groups < kPlaces ? groups : kPlaces);
    p.pieces = (int32_t)((p.ranges + units - 1) / units) + 1;
    const size_t n = (size_t)2 * p.ranges * 16 * p.qb;
    p.part_bytes = up256(n * c->head_dim * 4);
    p.bytes = p.part_bytes + up256(n * 8);
  }
  return p;
}

template <class E, int D, int QB>
int launch(const AttendArgs& a, const Plan& p, hipStream_t s) {
  const dim3 units((unsigned)(a.tiles * a.cache.n_heads)), threads(kStreamWaves * kWave);
  if (p.mode == kSmallPages) {
    hipLaunchKernelGGL((attend_units<E, D, QB, kStreamWaves, false>), units, threads, 0, s, a);
  } else if (p.mode == kUnits) {
    hipLaunchKernelGGL((attend_units<E, D, QB, kStreamWaves, true>), units, threads, 0, s, a);
  } else {
    hipLaunchKernelGGL((attend_ranges<E, D, QB>), dim3((unsigned)a.ranges), threads, 0, s, a);
    if (p.pieces > 16)
      hipLaunchKernelGGL((join<E, D, QB, true>), dim3(units.x, 16 * QB), dim3(kJoinWaves * kWave), 0, s, a);
    else
      hipLaunchKernelGGL((join<E, D, QB, false>), dim3(units.x, 16 * QB / kJoin), dim3(kJoinWaves * kWave), 0, s, a);
  }
  return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
}

template <class E, int D>
int launch_columns(const AttendArgs& a, const Plan& p, hipStream_t s) {
  if constexpr (E::kBytes == 2 && D <= 128) {
    if (p.mode == kRows) {
      hipLaunchKernelGGL((attend_rows<D>), dim3((unsigned)(a.tiles * a.cache.n_heads)), dim3(kRowsWaves * kWave), 0, s, a);
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

}  // namespace attend_impl

extern "C" size_t sdv_attend_workspace_bytes(const sdv_cache* cache, int32_t B, int64_t n_draft_rows,
                                             int32_t n_q_heads, int32_t window, int32_t sinks) {
  using namespace attend_impl;
  if (!cache || B < 1 || n_draft_rows < 0 || cache->n_kv_heads < 1 || cache->max_pages < 1 || cache->page_size < 1 ||
      n_draft_rows + B > INT32_MAX || check(cache, B, n_draft_rows, n_q_heads, window, sinks) != SDV_OK)
    return 0;
  return plan_of(cache, B, n_draft_rows, n_q_heads, window, sinks, true).bytes;  // without a tree: that or less
}

extern "C" int sdv_attend(const sdv_cache* cache, int32_t B, int64_t n_draft_rows, const int32_t* ragged_offsets,
                          const int32_t* parents, const void* queries, int64_t query_stride, int32_t n_q_heads,
                          float scale, int32_t window, int32_t sinks, void* out, void* workspace,
                          size_t workspace_bytes, void* stream) {
  using namespace attend_impl;
  int rc = check_cache(cache, B, n_draft_rows, ragged_offsets);
  if (rc != SDV_OK) return rc;
  rc = check(cache, B, n_draft_rows, n_q_heads, window, sinks);
  if (rc != SDV_OK) return rc;
  const int64_t per = cache->dtype == SDV_BF16 ? 8 : 4;
  if (!queries || !out || out == queries || !aligned16(queries) || !aligned16(out) || query_stride % per ||
      query_stride < (int64_t)n_q_heads * cache->head_dim || !(scale - scale == 0.0f))
    return SDV_ERR_INVALID_ARG;
  if (query_stride > ((int64_t)1 << 31)) return SDV_ERR_LIMIT;
  const Plan p = plan_of(cache, B, n_draft_rows, n_q_heads, window, sinks, parents != nullptr);
  static_assert(kStreamWaves == kRowsWaves && kStreamWaves == kJoinWaves, "one bound for every launch");
  if (too_many(p.tiles * cache->n_kv_heads, kStreamWaves * kWave)) return SDV_ERR_LIMIT;
  if (p.bytes > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < p.bytes)) return SDV_ERR_WORKSPACE;
  AttendArgs a;
  a.cache = view_of(cache);
  a.B = B;
  a.n_q = n_q_heads;
  a.G = n_q_heads / cache->n_kv_heads;
  a.ranges = p.ranges;
  a.window = window;
  a.sinks = sinks;
  a.n_d = n_draft_rows;
  a.query_stride = query_stride;
  a.tiles = p.tiles;
  a.scale2 = fmaxf(fabsf(scale) * 1.4426950408889634f, 0x1p-126f);
  a.flip = scale < 0 ? (cache->dtype == SDV_BF16 ? 0x80008000u : 0x80000000u) : 0u;
  a.cu = ragged_offsets;
  a.parents = parents;
  a.queries = static_cast<const char*>(queries);
  a.out = static_cast<char*>(out);
  a.part = static_cast<float*>(workspace);
  a.stats = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.part_bytes);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return cache->dtype == SDV_BF16 ? launch_dim<Bf16>(a, cache->head_dim, p, s)
                                  : launch_dim<F32>(a, cache->head_dim, p, s);
}
