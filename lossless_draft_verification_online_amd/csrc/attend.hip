// Attention of a ragged batch's rows over the paged cache, with a sliding window and first tokens
// that stay visible: sdv_attend.  Short calls and long caches run by the units of attend_unit.hpp; prompts
// by attend_rows, below.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "attend_unit.hpp"

namespace attend_impl {

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
      for (int x = 0; x < kLoads; ++x) bad |= not_finite<Bf16>(mine[64 * x]);
      if (__any(bad)) {
        for (int x = 0; x < kLoads; ++x) mine[64 * x] = finite_of<Bf16>(mine[64 * x]);
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
    hipLaunchKernelGGL((attend_units<E, D, QB, kStreamWaves, false, false>), units, threads, 0, s, a);
  } else if (p.mode == kUnits) {
    hipLaunchKernelGGL((attend_units<E, D, QB, kStreamWaves, true, false>), units, threads, 0, s, a);
  } else {
    hipLaunchKernelGGL((attend_ranges<E, D, QB, false>), dim3((unsigned)a.ranges), threads, 0, s, a);
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
