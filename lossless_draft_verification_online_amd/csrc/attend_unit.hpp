// Units of attention over the paged cache: a tile of a request's columns on one key/value head, whole or in
// ranges of its tokens that a second launch joins.  Shared by the calls over caches of the rows' type and in 8 bits.
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
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "cache8_view.hpp"

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
  // a cache in 8 bits: bytes b of the scales 2^(b - 127), [pages][heads][page_size >> block_log2]
  const uint8_t* key_scales;
  const uint8_t* value_scales;
  int32_t block_log2;
  bool many;           // cuts are told by unit
  struct Cut* cuts;    // [ranges][heads], or [units][heads] and one more with the number of units
};
// A unit that ranges cut, as its first range tells the join.
struct Cut {
  int32_t pieces, first_range, row0, k, head, c0, pad[2];  // pieces 0 or 1: it is whole, or the range begins none
};

// A cache in 8 bits holds e4m3 codes with a power of two as the scale of a block of tokens and head.  A code times its
// scale is a bf16 number without rounding (4 significant bits), so the products are those of bf16 caches, of
// operands converted in registers.  Queries and probabilities of binary32 rows go into them as three bf16 numbers
// whose sum they are: three products of the bf16 rate for eight of the binary32 instructions'.
struct Codes8 {
  static constexpr int kBytes = 1;
  // What is finite adds nothing where this is used; a code of seven set bits is no number.
  __device__ static __forceinline__ float at(const void* row, int64_t v) {
    return (static_cast<const uint8_t*>(row)[v] & 0x7f) == 0x7f ? __builtin_nanf("") : 0.0f;
  }
};

// 8 codes (two words) times their scale.
__device__ __forceinline__ bf16x8 bf16_of_codes(uint32_t lo, uint32_t hi, float scale) {
  const auto a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
  const auto b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
  const auto c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
  const auto d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
  bf16x8 v;
  v[0] = a[0], v[1] = a[1], v[2] = b[0], v[3] = b[1], v[4] = c[0], v[5] = c[1], v[6] = d[0], v[7] = d[1];
  return v;
}

// Codes that are no numbers, in a word of four.
__device__ __forceinline__ uint32_t nan_codes(uint32_t v) { return ((v & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }

// x as three bf16 numbers, cut and not rounded: 3 times 8 bits are its 24.  One that is not finite is the first.
__device__ __forceinline__ void three_of(float x, __bf16& a, __bf16& b, __bf16& c) {
  const float h = __uint_as_float(__float_as_uint(x) & 0xffff0000u);
  const float r = x - h;  // exact; NaN where x is infinite
  const float m = __uint_as_float(__float_as_uint(r) & 0xffff0000u);
  const bool finite = r == r;
  a = (__bf16)(finite ? h : x);
  b = (__bf16)(finite ? m : 0.0f);
  c = (__bf16)(finite ? r - m : 0.0f);
}

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

// tile_of, and the request's cached length: the lengths are loaded beside the offsets, where one wave holds those of all requests, since
// a workgroup has nothing to do until its pages are known.
template <int kColumns>
__device__ __forceinline__ TileOf tile_and_length(const AttendArgs& a, int64_t tile, int32_t& len) {
  if (a.B > kWave) {
    const TileOf t = tile_of<kColumns>(a, tile);
    len = t.r.index >= 0 ? a.cache.len[t.r.index] : -1;
    return t;
  }
  const int lane = threadIdx.x & (kWave - 1);
  const bool in = lane < a.B;
  const int32_t mine = in ? lane : a.B - 1;
  const int32_t lo = a.cu[mine], hi = a.cu[mine + 1], n = a.cache.len[mine];
  const int64_t first = (uint32_t)(lo + mine) * (uint32_t)a.G / (uint32_t)kColumns + mine;  // first_tile
  const uint64_t who = __ballot(in && first <= tile);
  const int src = who ? 63 - __builtin_clzll(who) : 0;
  Request r;
  r.index = src;
  r.first = lane_value(lo, src);
  r.k = lane_value(hi, src) - r.first;
  r.row0 = (int64_t)r.first + src;
  len = lane_value(n, src);
  if (__builtin_expect(!who || (who & (who + 1)) || r.first < 0 || r.k < 0 || (int64_t)r.first + r.k > a.n_d, 0)) {
    r = request_at(a.cu, tile_among<kColumns>(a, tile), a.n_d);  // some offsets are not valid
    len = r.index >= 0 ? a.cache.len[r.index] : -1;
  }
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
  __device__ __forceinline__ int32_t start(int32_t n) const { return (n < n_near ? n : n - n_near + t_lo) * kTile; }
  __device__ __forceinline__ bool held(int32_t s) const { return (s >= lo && s < hi) || s < near_end; }
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

// The entry of the table for token lane & 31 of tile n, below `end`.
template <bool kWholePages>
__device__ __forceinline__ int32_t table_entry(const AttendArgs& a, int32_t i, const Span& own, const Span& span, int32_t n,
                                               int32_t end) {
  const int32_t s = span.start(n) + (int32_t)(threadIdx.x & (kTile - 1)), k = s >> a.cache.page_log2;
  return n < end && (kWholePages || own.held(s)) && k < a.cache.max_pages ? a.cache.table[(int64_t)i * a.cache.max_pages + k] : -1;
}

// The batch's work is the list of its units (tile of columns, head), request by request, each of its token tiles.
// The list is cut into equal ranges, one per workgroup (8 bits: one per workgroup and head, so that the heads
// of a page, which lie next to each other, are read at about one time: 64 requests of K in 0 .. 8 137 us for 145): lengths differ
// between requests, and few units leave places empty (one request of 8 heads on 4000 tokens: 17 us by ranges, 42 by units).
struct Work {
  int32_t first, k, len;      // the request
  int32_t tiles, n;           // column tiles; token tiles of a unit (those of all its rows)
  // of the list: those of 8 bits are cut alike for every head
  template <bool k8>
  __device__ int64_t units(const AttendArgs& a) const { return k8 ? tiles : (int64_t)tiles * a.cache.n_heads; }
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
  int64_t total, units;          // items, and units, of the batch
  int64_t length;                // of a range
};
// A unit costs more than its tiles: its pages are found, its queries loaded and its waves joined.  For caches in 8 bits it
// counts as that many tiles more, or a range of many short units would end long after the others (64 requests of 4096 visible
// tokens and one that is empty: 190 us without, 148 with).
template <bool k8>
constexpr int kUnitCost = k8 ? 12 : 0;

template <bool k8>
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
    items += (uint64_t)(w.units<k8>(a) * (w.n + kUnitCost<k8>));
    units += (uint64_t)w.units<k8>(a);
  }
  const uint64_t inc = wave_inclusive_scan(items);
  s.before = (int64_t)(inc - items);
  const uint64_t inc_units = wave_inclusive_scan(units);
  s.units_before = (int64_t)(inc_units - units);
  s.units = (int64_t)lane_value(inc_units, kWave - 1);
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

template <class E, int D, int QB, int kWaves, bool k8>
struct Shape {
  static constexpr int kColumns = 16 * QB;
  static constexpr bool kBf16 = E::kBytes == 2 || k8;  // of the products
  static constexpr int kValueStride = D * 2 + 32;  // bytes; rows 8 banks apart for the transposing reads
  static constexpr int kValueBytes = kBf16 ? kWaves * kTile * kValueStride : 0;
  static constexpr int kMergeStride = D + 4;
  static constexpr int kMergeBytes = kWaves / 2 * kColumns * kMergeStride * 4;
  static constexpr int kBytes = kValueBytes > kMergeBytes ? kValueBytes : kMergeBytes;
};

template <class E, int D, int QB, int kWaves, bool k8>
struct Scratch {
  using S = Shape<E, D, QB, kWaves, k8>;
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
template <class C>
__device__ __forceinline__ bool not_finite(u32x4 v) {
  if constexpr (C::kBytes == 1) return (nan_codes(v.x) | nan_codes(v.y) | nan_codes(v.z) | nan_codes(v.w)) != 0;
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  u16x2 top = {0, 0};
#pragma unroll
  for (int w = 0; w < 4; ++w) top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, v[w] & 0x7fff7fffu));
  return top.x >= 0x7f80 || top.y >= 0x7f80;
}
template <class C>
__device__ __forceinline__ u32x4 finite_of(u32x4 v) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if constexpr (C::kBytes == 1) {
      v[w] &= ~((nan_codes(v[w]) >> 7) * 255u);
      continue;
    }
    if ((v[w] & 0x7f80u) == 0x7f80u) v[w] &= 0xffff0000u;
    if ((v[w] & 0x7f800000u) == 0x7f800000u) v[w] &= 0xffffu;
  }
  return v;
}
// One wave, for its columns and the tiles of [lo, hi) that are not all_see(start): add(column, d, value).
template <class C, int D, int kTokens, class Start, class AllSee, class Sees, class Add>
__device__ __forceinline__ void add_not_finite(const AttendArgs& a, int32_t i, int32_t head, int32_t lo, int32_t hi,
                                               int32_t columns, Start start, AllSee all_see, Sees sees, Add add) {
  const int lane = threadIdx.x & (kWave - 1);
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");  // the results are there
  for (int32_t n = lo; n < hi; ++n) {
    if (all_see(start(n))) continue;
    for (int32_t s = start(n); s < start(n) + kTokens; ++s) {
      const int32_t page = a.cache.page(i, s);
      if (page < 0) continue;
      const char* const row = a.cache.values + a.cache.row(page, head, s) * (D * C::kBytes);
#pragma unroll 1
      for (int d = lane; d < D; d += kWave) {
        const float v = C::at(row, d);
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
//
// 8 bits: a code times its scale is a bf16 number, converted in registers (keys) or on the way to shared memory (values).  The
// same 64 requests 119 us, 4.5 TB/s of 0.53 GB, and 6.2 for the join; three of 200 000 tokens in all 76 us, 5.4 TB/s.  Binary32
// rows take three bf16 products for one (16 trees 14.0 us, of a binary32 cache 24.8).
//
// Weights of bf16 rows go into the second product as bf16 numbers, off by 2^-8 at most each, as a result's own rounding is; as
// three terms they would take its time three times.  Errors against 64 bits, of results that are rounded from 32 bits in
// brackets: the 64 requests 0.0019 (0.0016) of the results' size, one row on 1000 tokens 0.0020 (0.0017), prompts 0.0023 (0.0017).
template <class E, int D, int QB, int kWaves, bool kWholePages, bool k8>
__device__ __forceinline__ void attend_unit(const AttendArgs& a, Scratch<E, D, QB, kWaves, k8>& sh, const TileOf& at,
                                            int32_t len, int32_t head, bool pos_all, int32_t w_lo, int32_t w_hi, int64_t slot) {
  using S = Shape<E, D, QB, kWaves, k8>;
  using C = typename std::conditional<k8, Codes8, E>::type;  // what the cache holds
  constexpr bool kBf16 = S::kBf16;
  constexpr int kSteps = k8 ? D / 64 : (kBf16 ? D / 32 : D / 16);  // 16-byte pieces of a key row per lane
  constexpr int kTerms = k8 && E::kBytes == 4 ? 3 : 1;             // of a query, or a probability
  constexpr int kQ = k8 ? D / 32 : kSteps;                         // pieces of a query's operands
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
  // Everything waits for the first pages: 8 bits ask for them before the queries (16 requests of one row on up to 4096 tokens
  // 35.7 us for 37.1 behind them; caches of the rows' type as they were).
  [[maybe_unused]] int32_t first_0 = -1, first_1 = -1;
  if constexpr (k8) {
    const int32_t tail_lo = a.parents ? 0 : j_lo, tail_hi = a.parents ? K : j_hi;
    const Span own = span_of(len, tail_lo, tail_hi, a.window, a.sinks);
    const Span span = pos_all ? span_of(len, 0, K, a.window, a.sinks) : own;
    const int32_t first = (pos_all ? w_lo : 0) + wave, end = !ok ? 0 : (pos_all ? w_hi : span.n);
    first_0 = table_entry<kWholePages>(a, i, own, span, first, end);
    first_1 = table_entry<kWholePages>(a, i, own, span, first + kWaves, end);
    __builtin_amdgcn_sched_barrier(0);
  }
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
  u32x4 q[QB][kTerms][kQ];
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    const int32_t c = at.c0 + 16 * b + col;
    live[b] = ok && c < columns;
    jrow[b] = live[b] ? (uint32_t)c / (uint32_t)a.G : 0;
    pos[b] = len + (a.parents && live[b] ? depth_s[jrow[b]] : jrow[b]);
    sight[b].rows = a.parents && live[b] ? sight_s[jrow[b]] : 0;
    sight[b].last = a.parents && live[b] ? last_s[jrow[b]] != 0 : false;
    const int32_t h = head * a.G + (c - jrow[b] * a.G);
    const char* src = a.queries + ((at.r.row0 + jrow[b]) * a.query_stride + h * D) * E::kBytes;
    if constexpr (!k8) src += 16 * g;
#pragma unroll
    for (int s = 0; s < kQ; ++s) {
      u32x4 z;
      z.x = z.y = z.z = z.w = 0;
      if constexpr (!k8) {
        if (live[b]) z = *reinterpret_cast<const u32x4*>(src + 64 * s) ^ a.flip;
        q[b][0][s] = z;
      } else {  // the 8 values that lie opposite to half s % 2 of a lane's 16 codes
        const char* const from = src + (64 * (s / 2) + 16 * g + 8 * (s % 2)) * E::kBytes;
        if (live[b]) z = *reinterpret_cast<const u32x4*>(from) ^ a.flip;
        if constexpr (kTerms == 1) {
          q[b][0][s] = z;
        } else {
          u32x4 y;
          y.x = y.y = y.z = y.w = 0;
          if (live[b]) y = *reinterpret_cast<const u32x4*>(from + 16) ^ a.flip;
          bf16x8 term[3];
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            __bf16 t0, t1, t2;
            three_of(__uint_as_float(e < 4 ? z[e & 3] : y[e & 3]), t0, t1, t2);
            term[0][e] = t0;
            term[1][e] = t1;
            term[2][e] = t2;
          }
#pragma unroll
          for (int x = 0; x < 3; ++x) q[b][x][s] = __builtin_bit_cast(u32x4, term[x]);
        }
      }
    }
  }

  // The tiles are those of the rows, or of all the request's rows; what this tile's rows see of them is the same.  (Found here and
  // not before the queries, and written out: units of 256 values keep 28 registers in memory, and 32 otherwise, of the
  // first keys among them, which wait for their load: 512 requests of one row on 4000 tokens 1492 us for 1807.)
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
  constexpr int kLine = D * C::kBytes;
  constexpr int kLoads = kLine / 32;  // 16-byte pieces per lane of a tile's values
  u32x4 vreg[kBf16 ? kLoads : 1];
  uint32_t byte_1 = 0;  // the next tile's scale of token lane & 31: of its keys, in the upper half of its values
  float scale = 0.0f;
  float vf[kBf16 ? 1 : 8][kDB];
  // The table's entry of token lane & 31 as it is, checked when it is used: a check would wait for it, and for
  // the keys and values asked for before it.
  const int32_t* const table = a.cache.table + (int64_t)i * a.cache.max_pages;
  auto entry_at = [&](int32_t n) -> int32_t {
    const int32_t s = start(n) + (lane & (kTile - 1)), k = s >> a.cache.page_log2;
    return n < w_hi && (kWholePages || held(s)) && k < a.cache.max_pages ? table[k] : -1;
  };
  auto page_of = [&](int32_t entry) { return entry >= 0 && entry < a.cache.n_pages ? entry : -1; };
  // the lane's byte offsets within 16 tokens' rows
  const uint32_t k_off = col * kLine + 16 * g;
  constexpr int kLanes = kLine / 16, kRows = kWave / kLanes;  // lanes of a value row, rows of one load
  const uint32_t v_off = (lane / kLanes) * kLine + (lane % kLanes) * 16;
  auto load_scales = [&](int32_t n, int32_t page) {
    const int32_t s = start(n) + (lane & (kTile - 1)), in = s & ((1 << a.cache.page_log2) - 1);
    const uint8_t* const from = lane < kTile ? a.key_scales : a.value_scales;
    byte_1 = from[(((int64_t)(page < 0 ? 0 : page) * a.cache.n_heads + head) << (a.cache.page_log2 - a.block_log2)) +
                  (in >> a.block_log2)];
  };
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
          for (int x = 0; x < kLoads / 2; ++x)
            vreg[blk * (kLoads / 2) + x] = *reinterpret_cast<const u32x4*>(vs + x * kRows * kLine);
        }
      } else {
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
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
  int32_t page = page_of(k8 ? first_0 : entry_at(n)), entry_1 = k8 ? first_1 : entry_at(n + kWaves);
  if (n < w_hi) {
    if constexpr (k8) load_scales(n, page);
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
    if constexpr (k8) {
      scale = scale_of(byte_1);
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        const float by = __shfl(scale, 16 * blk + col);
#pragma unroll
        for (int b = 0; b < QB; ++b) sc[b][blk] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < kQ; ++s) {
          const bf16x8 k = bf16_of_codes(kreg[blk][s / 2][2 * (s % 2)], kreg[blk][s / 2][2 * (s % 2) + 1], by);
#pragma unroll
          for (int b = 0; b < QB; ++b)
#pragma unroll
            for (int x = kTerms - 1; x >= 0; --x)
              sc[b][blk] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, __builtin_bit_cast(bf16x8, q[b][x][s]), sc[b][blk],
                                                                    0, 0, 0);
        }
      }
      if (more) load_scales(n + kWaves, page_1);
    }
#pragma unroll
    for (int b = 0; b < QB && !k8; ++b) {
#pragma unroll
      for (int blk = 0; blk < 2; ++blk) {
        sc[b][blk] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          if constexpr (kBf16) {
            sc[b][blk] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, kreg[blk][s]),
                                                                  __builtin_bit_cast(bf16x8, q[b][0][s]), sc[b][blk], 0, 0, 0);
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              sc[b][blk] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(kreg[blk][s][e]),
                                                                __uint_as_float(q[b][0][s][e]), sc[b][blk], 0, 0, 0);
          }
        }
      }
    }
    if (more) load_keys(n + kWaves, page_1);
    if constexpr (kBf16) {
      if (!paged) {
#pragma unroll
        for (int x = 0; x < kLoads; ++x)
          if (!((there >> (x * kRows + lane / kLanes)) & 1)) vreg[x].x = vreg[x].y = vreg[x].z = vreg[x].w = 0;
      }
      if (!all_see(s0)) {
        bool bad = false;
#pragma unroll
        for (int x = 0; x < kLoads; ++x) bad |= not_finite<C>(vreg[x]);
        if (__any(bad)) {
          odd = true;
#pragma unroll
          for (int x = 0; x < kLoads; ++x) vreg[x] = finite_of<C>(vreg[x]);
        }
      }
#pragma unroll
      for (int x = 0; x < kLoads; ++x) {
        char* const to = v_lds + (x * kRows + lane / kLanes) * S::kValueStride + (lane % kLanes) * (16 * 2 / C::kBytes);
        if constexpr (k8) {
          const float by = __shfl(scale, kTile + x * kRows + lane / kLanes);
          *reinterpret_cast<bf16x8*>(to) = bf16_of_codes(vreg[x].x, vreg[x].y, by);
          *reinterpret_cast<bf16x8*>(to + 16) = bf16_of_codes(vreg[x].z, vreg[x].w, by);
        } else {
          *reinterpret_cast<u32x4*>(to) = vreg[x];
        }
      }
      if (more) load_values(n + kWaves, page_1);
    }

    const bool whole = paged && all_see(s0);  // no masks
    bf16x8 pb[QB][kTerms];
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
        if constexpr (kTerms == 3) {
          __bf16 t0, t1, t2;
          three_of(p, t0, t1, t2);
          pb[b][0][e] = t0;
          pb[b][1][e] = t1;
          pb[b][2][e] = t2;
        } else if constexpr (kBf16) {
          pb[b][0][e] = (__bf16)p;
        } else {
          pf[b][e] = p;
        }
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
#pragma unroll
          for (int x = kTerms - 1; x >= 0; --x)
            acc[b][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, pb[b][x], acc[b][d], 0, 0, 0);
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
        if constexpr (E::kBytes == 2) {
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
    add_not_finite<C, D, kTile>(
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

// Two waves per SIMD hide each other's loads; sums of 64 columns, or of 256 values, take the registers of both.  (Of 256 bf16
// values two waves keep registers in memory: units 28, ranges 55, ranges over 8 bits 27.)
template <class E, int D, int QB>
constexpr int kMinWaves = E::kBytes == 4 ? (D <= 128 ? 2 : 1) : (D * QB <= 256 ? 2 : 1);

// A workgroup per unit.
template <class E, int D, int QB, int kWaves, bool kWholePages, bool k8>
__global__ __launch_bounds__(kWaves* kWave, (kMinWaves<E, D, QB>)) void attend_units(AttendArgs a) {
  __shared__ Scratch<E, D, QB, kWaves, k8> sh;
  const int64_t block = unit_of_block(blockIdx.x, gridDim.x);
  TileOf at;
  int32_t len = 0;
  if constexpr (k8)
    at = tile_and_length<16 * QB>(a, block / a.cache.n_heads, len);
  else
    at = tile_of<16 * QB>(a, block / a.cache.n_heads);
  if (at.r.index < 0) return;
  attend_unit<E, D, QB, kWaves, kWholePages, k8>(a, sh, at, k8 ? len : a.cache.len[at.r.index],
                                                 (int32_t)(block % a.cache.n_heads), false, 0, 0, -1);
}

// A workgroup per range of the batch's work.
constexpr int kStreamWaves = 4;
template <class E, int D, int QB, bool k8>
__global__ __launch_bounds__(kStreamWaves* kWave, (kMinWaves<E, D, QB>)) void attend_ranges(AttendArgs a) {
  constexpr int kColumns = 16 * QB, kCost = kUnitCost<k8>;
  __shared__ Scratch<E, D, QB, kStreamWaves, k8> sh;
  const Stream s = stream_of<k8>(a, kColumns);
  const int64_t block = unit_of_block(blockIdx.x, gridDim.x);
  const int64_t range = k8 ? (uint32_t)block / (uint32_t)a.cache.n_heads : block;
  const int32_t own_head = k8 ? (int32_t)(block - range * a.cache.n_heads) : 0;
  const int64_t end = (range + 1) * s.length < s.total ? (range + 1) * s.length : s.total;
  int64_t p = range * s.length;
  Cut cut = {};
  if constexpr (k8) {
    // requests that do not lie in their order can have more units than there is room for
    if (a.many && block == 0 && threadIdx.x == 0)
      a.cuts[a.tiles * a.cache.n_heads].pieces = (int32_t)(s.units < a.tiles ? s.units : a.tiles);
    if (p >= end && !a.many && threadIdx.x == 0) a.cuts[block] = cut;
  }
  if (p >= end) return;
  // the request of p, then on from one to the next
  const int who = 63 - __builtin_clzll(__ballot(s.before <= p));
  int32_t i = who * s.per;
  int64_t base = (int64_t)lane_value((uint64_t)s.before, who);
  int64_t units = k8 ? (int64_t)lane_value((uint64_t)s.units_before, who) : 0;  // before the request
  while (p < end && i < a.B) {
    const Work w = work_at(a, s, i, kColumns);
    const int32_t span = w.n + kCost;
    const int64_t items = w.units<k8>(a) * span;
    if (p >= base + items) {
      base += items;
      if constexpr (k8) units += w.units<k8>(a);
      ++i;
      continue;
    }
    const uint32_t unit = (uint32_t)((p - base) / span);
    int32_t q_lo = (int32_t)(p - base - (int64_t)unit * span);
    int32_t q_hi = q_lo + (end - p) < span ? (int32_t)(q_lo + (end - p)) : span;
    p += q_hi - q_lo;
    if constexpr (kCost > 0) {  // the cost comes before the tiles
      q_lo = q_lo > kCost ? q_lo - kCost : 0;
      q_hi -= kCost;
      if (q_hi <= 0) continue;
    }
    TileOf at;
    at.r = request_with(w, i);
    const int32_t head = k8 ? own_head : (int32_t)(unit % (uint32_t)a.cache.n_heads);
    at.c0 = (int32_t)(k8 ? unit : unit / (uint32_t)a.cache.n_heads) * kColumns;
    const bool first = q_lo == 0, whole = first && q_hi == w.n;
    if constexpr (k8) {
      if (first) {
        const int64_t begin = base + (int64_t)unit * span + kCost;
        cut.pieces = whole ? 1 : (int32_t)((uint64_t)(begin + w.n - 1) / (uint64_t)s.length - range) + 1;
        cut.first_range = (int32_t)range;
        cut.row0 = w.first + i;
        cut.k = w.k;
        cut.head = head;
        cut.c0 = at.c0;
        if (a.many && threadIdx.x == 0 && units + unit < a.tiles) a.cuts[(units + unit) * a.cache.n_heads + head] = cut;
      }
    }
    attend_unit<E, D, QB, kStreamWaves, true, k8>(a, sh, at, w.len, head, true, q_lo, q_hi,
                                                  whole ? -1 : 2 * block + (first ? 1 : 0));
    __syncthreads();
  }
  if constexpr (k8) {
    if (!a.many && threadIdx.x == 0) a.cuts[block] = cut;  // the last unit that it begins: no other is cut
  }
}

// Joins the pieces of the units that ranges cut.  A workgroup takes kJoin columns of a unit, or, where a
// unit is cut into many pieces (few units, long caches), one column whose pieces its waves share.  Lane k of
// D / 4 holds four values of a column; the wave's other lanes hold the same of further pieces.
constexpr int kJoinWaves = 4;
constexpr int kJoin = 8;

template <class E, int D, int QB, bool kMany, bool k8>
__global__ __launch_bounds__(kJoinWaves* kWave) void join(AttendArgs a) {
  constexpr int kColumns = 16 * QB, kLanes = D / 4, kRows = kWave / kLanes;  // pieces a wave reads at once
  __shared__ float o_s[kJoinWaves][D], stat_s[kJoinWaves][2];
  const int t = threadIdx.x, lane = t & (kWave - 1), k = lane % kLanes;
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int64_t u = blockIdx.x;
  int64_t r_lo, row0;
  int32_t pieces, head, c0, columns;
  if constexpr (k8) {
    const Cut cut = a.cuts[u];
    if (kMany && u >= (int64_t)a.cuts[gridDim.x].pieces * a.cache.n_heads) return;
    if (cut.pieces <= 1) return;
    r_lo = cut.first_range;
    pieces = cut.pieces;
    row0 = cut.row0;
    head = cut.head;
    c0 = cut.c0;
    columns = (cut.k + 1) * a.G;
  } else {
    const Stream s = stream_of<false>(a, kColumns);
    const int who = 63 - __builtin_clzll(__ballot(s.units_before <= u));
    int64_t begin = (int64_t)lane_value((uint64_t)s.before, who);
    int64_t unit = u - (int64_t)lane_value((uint64_t)s.units_before, who);
    int32_t i = who * s.per;
    Work w;
    for (;; ++i) {
      if (i >= a.B) return;
      w = work_at(a, s, i, kColumns);
      if (unit < w.units<false>(a)) break;
      unit -= w.units<false>(a);
      begin += w.units<false>(a) * w.n;
    }
    begin += unit * w.n;
    r_lo = begin / s.length;
    pieces = (int32_t)((begin + w.n - 1) / s.length - r_lo) + 1;
    if (pieces == 1) return;
    const Request r = request_with(w, i);
    row0 = r.row0;
    head = (uint32_t)unit % (uint32_t)a.cache.n_heads;
    c0 = (int32_t)((uint32_t)unit / (uint32_t)a.cache.n_heads) * kColumns;
    columns = (r.k + 1) * a.G;
  }
  // the piece with the unit's first tile is its range's second, the others their ranges' first
  auto at = [&](int32_t piece) {
    const int64_t range = k8 ? (r_lo + piece) * a.cache.n_heads + head : r_lo + piece;
    return (2 * range + (piece == 0 ? 1 : 0)) * kColumns;
  };
  const int x_lo = blockIdx.y * (kMany ? 1 : kJoin), x_hi = x_lo + (kMany ? 1 : kJoin);
  for (int x = x_lo + (kMany ? 0 : wave); x < x_hi; x += kMany ? 1 : kJoinWaves) {
    const int32_t c = c0 + x;
    if (c >= columns) break;
    // this wave's pieces: all of them, or every kJoinWaves-th 64
    float top = -__builtin_inff(), sum = 0.0f;
    f32x4 o = f32x4{0, 0, 0, 0};
    const int32_t share = k8 && kMany ? (pieces + kJoinWaves - 1) / kJoinWaves : kWave;  // 8 bits: in equal parts
    const int32_t p_end = k8 && kMany ? (wave * share + share < pieces ? wave * share + share : pieces) : pieces;
    for (int32_t p0 = kMany ? wave * share : 0; p0 < p_end; p0 += kMany && !k8 ? kJoinWaves * kWave : kWave) {
      const int32_t p = p0 + lane;
      float m = -__builtin_inff(), l = 0.0f;
      if (p < p_end) {
        m = a.stats[2 * (at(p) + x)];
        l = a.stats[2 * (at(p) + x) + 1];
      }
      const float next = fmaxf(top, wave_max(m)), frame = next == -__builtin_inff() ? 0.0f : next;
      const float fade = fast_exp2(top - frame), scale = fast_exp2(m - frame);
      top = next;
      sum = sum * fade + wave_sum(l * scale);
      o *= fade;
      const int32_t n = p_end - p0 < kWave ? p_end - p0 : kWave;
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
    char* dst = a.out + ((row0 + j) * a.n_q + h) * (D * E::kBytes) + k * 4 * E::kBytes;
    if constexpr (E::kBytes == 2) {
      bf16x4 v;
      for (int e = 0; e < 4; ++e) v[e] = (__bf16)o[e];
      *reinterpret_cast<bf16x4*>(dst) = v;
    } else {
      *reinterpret_cast<f32x4*>(dst) = o;
    }
  }
}

}  // namespace attend_impl
