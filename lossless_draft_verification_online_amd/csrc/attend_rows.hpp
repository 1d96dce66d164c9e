// Attention of many rows per request (prompts) over the paged cache: a workgroup per tile of 128 columns and head.
#pragma once

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
// 8 bits: a wave turns the codes of its 16 rows into bf16 numbers in their place before the barrier, so that the products read
// what they read of a bf16 cache.  Those conversions are the difference: 16 x 2501 rows on 4000 tokens 874 to 884 TF/s, under a
// window of 1024 550.  Among the exponentials, or behind the products, they took longer (registers, and waits for the loads).
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

template <int D, bool k8>
__global__ __launch_bounds__(kRowsWaves* kWave, 2) void attend_rows(AttendArgs a) {
  using C = typename std::conditional<k8, Codes8, Bf16>::type;  // what the cache holds
  constexpr int kCacheLine = D * C::kBytes, kCachePieces = kCacheLine / 16;
  constexpr int kLine = D * 2, kPieces = D / 8, kSteps = D / 16, kDB = D / 32;
  constexpr int kLoadRows = kWave / kCachePieces;  // rows of one direct load
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
    const int row = x * kLoadRows + lane / kCachePieces;
    off[x] = row * kCacheLine + (k8 ? lane % kCachePieces : piece_of<D>(row, lane % kCachePieces)) * 16;
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
    const int64_t at_row = a.cache.row(page < 0 ? 0 : page, head, start(n) + 16 * wave) * kCacheLine;
    from += ((int64_t)all((int32_t)(at_row >> 32)) << 32) | (uint32_t)all((int32_t)at_row);
    to += 16 * wave * kLine;
#pragma unroll
    for (int x = 0; x < kLoads; ++x) direct_load(from, 16 * kCacheLine, off[x], to + x * 1024);
  };
  // 8 bits: lanes 0 .. 15 take the bytes of the scales of the wave's rows of keys, lanes 16 .. 31 of values
  uint32_t byte = 0;
  auto load_scales = [&](int32_t n_keys, int32_t page_keys, int32_t n_values, int32_t page_values) {
    const bool keys = lane < 16;
    const int32_t page_here = keys ? page_keys : page_values;
    const int32_t s = start(keys ? n_keys : n_values) + 16 * wave + (lane & 15), in = s & ((1 << a.cache.page_log2) - 1);
    const uint8_t* const from_scales = keys ? a.key_scales : a.value_scales;
    byte = from_scales[(((int64_t)(page_here < 0 ? 0 : page_here) * a.cache.n_heads + head)
                        << (a.cache.page_log2 - a.block_log2)) +
                       (in >> a.block_log2)];
  };
  // The codes of the wave's rows, where direct loads put them at the front of the rows' place, and their bf16 values
  // in that place: both are the wave's own until the barrier.
  // A lane's codes go to pieces p and p + 1 of its row, neighbours in the permuted order too (p is even, and so is what it is
  // combined with); its rows are a multiple of 8 apart: one address serves all.
  const int codes_off = 16 * wave * kLine + lane * 16;
  const int wide_row = lane / kCachePieces;
  const int wide_off = (16 * wave + wide_row) * kLine + piece_of<D>(wide_row, 2 * (lane % kCachePieces)) * 16;
  auto codes_at = [&](const char* to, u32x4 (&v)[kLoads]) {
#pragma unroll
    for (int x = 0; x < kLoads; ++x) v[x] = *reinterpret_cast<const u32x4*>(to + codes_off + x * 1024);
  };
  auto widen = [&](const u32x4 (&v)[kLoads], float scale, int lane_0, char* to) {
#pragma unroll
    for (int x = 0; x < kLoads; ++x) {
      const float by = __int_as_float(
          __builtin_amdgcn_ds_bpermute(4 * wide_row + 4 * (lane_0 + x * kLoadRows), __float_as_int(scale)));
      char* const dst = to + wide_off + x * kLoadRows * kLine;
      *reinterpret_cast<bf16x8*>(dst) = bf16_of_codes(v[x].x, v[x].y, by);
      *reinterpret_cast<bf16x8*>(dst + 16) = bf16_of_codes(v[x].z, v[x].w, by);
    }
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
    if constexpr (k8) load_scales(0, page, 0, page);
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
  // 8 bits: a row's pieces differ in the bits above 2^5 (keys) or 2^6 (values), which the permutation flips: a step's address is
  // made of one by an exclusive or.  `here` keeps the compiler from holding all of them, for which there are no registers (what is
  // spilled and loaded again waits for the direct loads).
  const int key_off = col * kLine + piece_of<D>(col, half) * 16;
  const int value_token = 4 * half + ((lane & 15) >> 2);
  const int value_off = value_token * kLine + piece_of<D>(value_token, 2 * ((lane >> 4) & 1) + ((lane >> 1) & 1)) * 16 + (lane & 1) * 8;
  int key_here = 0, value_here = 0;
  auto key = [&](const char* k_s, int blk, int s) {
    if constexpr (k8) return *reinterpret_cast<const bf16x8*>(k_s + (key_here ^ (32 * s)) + 32 * blk * kLine);
    const int token = 32 * blk + col;
    return *reinterpret_cast<const bf16x8*>(k_s + token * kLine + piece_of<D>(token, 2 * s + half) * 16);
  };
  // values of step s: tokens 16 s + 4 half + 0 .. 3 and 8 further; a 16-lane group reads 4 tokens x 16 values
  auto value = [&](char* v_s, int s, bf16x4 (&v)[kDB][2]) {
    typedef __attribute__((address_space(3))) bf16x4 lds_bf16x4;
    const int g = (lane >> 4) & 1, in = lane & 15, token = 16 * s + 4 * half + (in >> 2);
#pragma unroll
    for (int d = 0; d < kDB; ++d) {
      if constexpr (k8) {
        char* const r = v_s + (value_here ^ (64 * d)) + 16 * s * kLine;
        v[d][0] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)r);
        v[d][1] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_bf16x4*)(r + 8 * kLine));
        continue;
      }
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
    if constexpr (k8) {
      key_here = key_off;
      value_here = value_off;
      asm volatile("" : "+v"(key_here), "+v"(value_here));
    }
    // a value no row sees is 0: what lies there may be NaN
    const int32_t first = s0 + 16 * wave;
    const bool held = page >= 0 && (first + 16 <= span.near_end || (first >= span.lo && first + 16 <= span.hi));
    if constexpr (k8) {
      if (lane == 0) page_s[n & 1][wave] = page;
      __builtin_amdgcn_s_waitcnt(0x0f70);  // this wave's direct loads
      u32x4 kv[kLoads], vv[kLoads];
      codes_at(k_s, kv);
      codes_at(v_s, vv);
      if (!held) {
#pragma unroll
        for (int x = 0; x < kLoads; ++x) {
          const int32_t s = first + x * kLoadRows + lane / kCachePieces;
          if (page < 0 || !(s < span.near_end || (s >= span.lo && s < span.hi))) vv[x].x = vv[x].y = vv[x].z = vv[x].w = 0;
        }
      }
      if (!all_see(s0)) {
        bool bad = false;
#pragma unroll
        for (int x = 0; x < kLoads; ++x) bad |= not_finite<C>(vv[x]);
        if (__any(bad)) {
          for (int x = 0; x < kLoads; ++x) vv[x] = finite_of<C>(vv[x]);
          odd_s = 1;
        }
      }
      const float scale = scale_of(byte);
      widen(kv, scale, 0, k_s);
      widen(vv, scale, 16, v_s);
    } else {
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
        for (int x = 0; x < kLoads; ++x) bad |= not_finite<C>(mine[64 * x]);
        if (__any(bad)) {
          for (int x = 0; x < kLoads; ++x) mine[64 * x] = finite_of<C>(mine[64 * x]);
          odd_s = 1;
        }
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
    if constexpr (k8) load_scales(n + 2, page_1, n + 1, page);
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
    // weights in 8 bits for the product with the values, as in attend_unit; their sum is of 32
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
    key_here = key_off;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const char* const from = (s < kSteps / 2 ? k_1 : v_1) + 16 * wave * kLine;
      q[s] = __builtin_bit_cast(
          bf16x8, *reinterpret_cast<const u32x4*>(from + half_piece(col, (2 * s) % kHalf + half)) ^ a.flip);
    }
    if constexpr (k8) {
      u32x4 kv[kLoads];
      codes_at(k_0, kv);
      widen(kv, scale_of(byte), 0, k_0);
      load_scales(1, page_1, 0, page);
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
    add_not_finite<C, D, kRowsTile>(
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

}  // namespace attend_impl
