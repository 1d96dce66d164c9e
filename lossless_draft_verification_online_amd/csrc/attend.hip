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

#include "cache_view.hpp"

namespace attend_impl {

using namespace sdv;

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
constexpr int kTile = 32;  // tokens a wave takes at a time

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

struct AttendArgs {
  CacheView cache;
  int32_t B, n_q, G, splits, window, sinks;
  int64_t n_d, query_stride, tiles;
  float scale2;  // scale * log2(e)
  const int32_t* cu;
  const int32_t* parents;
  const char* queries;
  char* out;
  float* part;   // [unit][column][D] sums of a split, in the frame of its maxima
  float* stats;  // [unit][column][2] maximum and sum of weights
};

// First tile number of request i: its columns take at most ceil((K + 1) G / columns) tiles from there.
__device__ __forceinline__ int64_t first_tile(const int32_t* cu, int32_t i, int32_t G, int32_t columns) {
  return ((int64_t)cu[i] + i) * G / columns + i;
}

struct TileOf {
  Request r;
  int64_t c0;  // its first column within the request
};

template <int kColumns>
__device__ __forceinline__ TileOf tile_of(const AttendArgs& a, int64_t tile) {
  TileOf t;
  const int32_t i =
      find_last(a.B, tile, [&](int32_t q) { return first_tile(a.cu, q, a.G, kColumns); });
  t.r = request_at(a.cu, i, a.n_d);
  t.c0 = 0;
  if (t.r.index < 0) return t;
  t.c0 = (tile - first_tile(a.cu, i, a.G, kColumns)) * kColumns;
  if (t.c0 >= ((int64_t)t.r.k + 1) * a.G) t.r.index = -1;
  return t;
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

// Which rows of a tree a row sees: bit n of nodes for node n's slot, root for row 0's.
struct TreeSight {
  uint64_t nodes;
  bool root;
};

template <class E, int D, int QB>
struct Shape {
  static constexpr int kColumns = 16 * QB;
  static constexpr bool kBf16 = E::kBytes == 2;
  static constexpr int kValueStride = D * 2 + 32;  // bytes; rows 8 banks apart for the transposing reads
  static constexpr int kValueBytes = kBf16 ? kWaves * kTile * kValueStride : 0;
  static constexpr int kMergeStride = D + 4;
  static constexpr int kMergeBytes = 2 * kColumns * kMergeStride * 4;
  static constexpr int kBytes = kValueBytes > kMergeBytes ? kValueBytes : kMergeBytes;
};

template <class E, int D, int QB>
__global__ __launch_bounds__(kThreads) void attend(AttendArgs a) {
  using S = Shape<E, D, QB>;
  constexpr bool kBf16 = S::kBf16;
  constexpr int kSteps = kBf16 ? D / 32 : D / 16;  // 16-byte pieces of a key row per lane
  constexpr int kDB = D / 16;                       // blocks of 16 output values
  __shared__ __align__(16) char smem[S::kBytes];
  __shared__ float m_s[kWaves][S::kColumns], l_s[kWaves][S::kColumns];
  __shared__ int32_t parent_s[kWave], depth_s[kMaxNodes + 1];
  __shared__ uint64_t sight_s[kMaxNodes + 1];
  __shared__ int32_t root_s[kMaxNodes + 1];

  const int t = threadIdx.x, lane = t & (kWave - 1), col = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int32_t head = (int32_t)(blockIdx.x % a.cache.n_heads);
  const int64_t rest = blockIdx.x / a.cache.n_heads;
  const int32_t split = (int32_t)(rest % a.splits);
  const int64_t tile = rest / a.splits;
  const TileOf at = tile_of<S::kColumns>(a, tile);
  if (at.r.index < 0) return;
  const int32_t i = at.r.index, K = at.r.k;
  const int64_t len = a.cache.len[i];
  const int64_t columns = ((int64_t)K + 1) * a.G;
  const int64_t c_last = at.c0 + S::kColumns < columns ? at.c0 + S::kColumns - 1 : columns - 1;
  const int64_t j_lo = at.c0 / a.G, j_hi = c_last / a.G;  // rows of this tile
  bool ok = len >= 0;
  if (a.parents && ok) {
    ok = tree_depths(a.parents, at.r, parent_s, depth_s);
    if (ok) {
      if (t <= K) {
        uint64_t nodes = 0;
        for (int32_t n = t - 1; n >= 0; n = parent_s[n])
          if (a.window == 0 || depth_s[t] - depth_s[n + 1] < a.window || len + n + 1 < a.sinks) nodes |= 1ull << n;
        sight_s[t] = nodes;
        root_s[t] = a.window == 0 || depth_s[t] < a.window || len < a.sinks;
      }
      __syncthreads();
    }
  }

  // this lane's columns: their rows, positions and queries
  int64_t pos[QB];
  int32_t jrow[QB];
  bool live[QB];
  TreeSight sight[QB];
  u32x4 q[QB][kSteps];
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    const int64_t c = at.c0 + 16 * b + col;
    live[b] = ok && c < columns;
    jrow[b] = live[b] ? (int32_t)(c / a.G) : 0;
    pos[b] = len + (a.parents && live[b] ? depth_s[jrow[b]] : jrow[b]);
    sight[b].nodes = a.parents && live[b] ? sight_s[jrow[b]] : 0;
    sight[b].root = a.parents && live[b] ? root_s[jrow[b]] != 0 : false;
    const int64_t h = (int64_t)head * a.G + (c - (int64_t)jrow[b] * a.G);
    const char* src = a.queries + ((at.r.row0 + jrow[b]) * a.query_stride + h * D) * E::kBytes + 16 * g;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      u32x4 z;
      z.x = z.y = z.z = z.w = 0;
      if (live[b]) z = *reinterpret_cast<const u32x4*>(src + 64 * s);
      q[b][s] = z;
    }
  }

  // The slots that any row of the tile sees: [0, near_end) and [lo, hi).
  const int64_t tail_lo = a.parents ? 0 : j_lo, tail_hi = a.parents ? K : j_hi;
  const int64_t hi = len + tail_hi + 1;
  const int64_t lo = a.window && len + tail_lo - a.window + 1 > 0 ? len + tail_lo - a.window + 1 : 0;
  const int64_t near_end = lo < a.sinks ? lo : a.sinks;
  int64_t t_lo = lo / kTile, n_near = (near_end + kTile - 1) / kTile;
  if (t_lo <= n_near) {  // the first tokens' tiles run into the window's
    t_lo = 0;
    n_near = 0;
  }
  const int64_t n_tiles = ok ? n_near + (hi + kTile - 1) / kTile - t_lo : 0;
  const int64_t w_lo = n_tiles * split / a.splits, w_hi = n_tiles * (split + 1) / a.splits;
  const int64_t far = len + tail_hi;  // the largest position
  auto start = [&](int64_t n) { return (n < n_near ? n : n - n_near + t_lo) * kTile; };
  auto held = [&](int64_t s) { return (s >= lo && s < hi) || s < near_end; };

  f32x4 acc[QB][kDB];
  float m[QB], l[QB];
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    m[b] = -__builtin_inff();
    l[b] = 0.0f;
#pragma unroll
    for (int d = 0; d < kDB; ++d) acc[b][d] = f32x4{0, 0, 0, 0};
  }

  char* const v_lds = smem + wave * kTile * S::kValueStride;
  u32x4 kreg[2][kSteps];
  u32x4 vreg[kBf16 ? D / 16 : 1];
  auto page_at = [&](int64_t n) -> int32_t {  // of token lane & 31
    const int64_t s = start(n) + (lane & (kTile - 1));
    return n < w_hi && held(s) ? a.cache.page(i, s) : -1;
  };
  auto load = [&](int64_t n, int32_t page) {
    const int64_t s0 = start(n);
#pragma unroll
    for (int blk = 0; blk < 2; ++blk) {
      const int k = 16 * blk + col;
      const int32_t p = __shfl(page, k);
      const char* src = a.cache.keys + a.cache.row(p < 0 ? 0 : p, head, s0 + k) * (D * E::kBytes) + 16 * g;
#pragma unroll
      for (int s = 0; s < kSteps; ++s) kreg[blk][s] = *reinterpret_cast<const u32x4*>(src + 64 * s);
    }
    if constexpr (kBf16) {
      constexpr int kLanes = D / 8, kRows = kWave / kLanes;  // lanes of a value row, rows of one load
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        const int k = x * kRows + lane / kLanes;
        const int32_t p = __shfl(page, k);
        const u32x4 v = *reinterpret_cast<const u32x4*>(
            a.cache.values + a.cache.row(p < 0 ? 0 : p, head, s0 + k) * (D * 2) + (lane % kLanes) * 16);
        vreg[x] = v;
      }
    }
  };

  int64_t n = w_lo + wave;
  int32_t page = page_at(n);
  if (n < w_hi) load(n, page);
  for (; n < w_hi; n += kWaves) {
    const int64_t s0 = start(n);
    const int32_t page_next = page_at(n + kWaves);
    // a value no row sees is 0: what lies there may be NaN
    const bool paged = __all(page >= 0);
    if constexpr (kBf16) {
      constexpr int kLanes = D / 8, kRows = kWave / kLanes;
#pragma unroll
      for (int x = 0; x < D / 16; ++x) {
        const int k = x * kRows + lane / kLanes;
        u32x4 v = vreg[x];
        if (!paged && __shfl(page, k) < 0) v.x = v.y = v.z = v.w = 0;
        *reinterpret_cast<u32x4*>(v_lds + k * S::kValueStride + (lane % kLanes) * 16) = v;
      }
    }
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
    const int32_t page_now = page;
    page = page_next;
    if (n + kWaves < w_hi) load(n + kWaves, page);

    // every row sees every token of the tile: no masks
    const bool whole = paged && s0 + kTile <= (a.parents ? len : len + j_lo + 1) &&
                       (a.window == 0 || s0 > far - a.window || s0 + kTile <= a.sinks);
    bf16x8 pb[QB];
    float pf[QB][8];
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = sc[b][e >> 2][e & 3] * a.scale2;
      if (!whole) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int k = 16 * (e >> 2) + 4 * g + (e & 3);
          const int64_t s = s0 + k;
          const bool there = __shfl(page_now, k) >= 0;  // by every lane: before the tests that part them
          const bool near = a.window == 0 || pos[b] - s < a.window || s < a.sinks;
          const int64_t node = s - len;  // row index behind the cached slots
          bool see;
          if (node < 0)
            see = near;
          else if (!a.parents)
            see = near && node <= jrow[b];
          else
            see = node == 0 ? sight[b].root : (node <= K && ((sight[b].nodes >> ((node - 1) & 63)) & 1));
          if (!see || !live[b] || !there) x[e] = -__builtin_inff();
        }
      }
      float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
      top = both_max16_32(top);
      const float m_new = fmaxf(m[b], top);
      const float frame = m_new == -__builtin_inff() ? 0.0f : m_new;
      const float fade = fast_exp2(m[b] - frame);
      m[b] = m_new;
      float sum = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float p = fast_exp2(x[e] - frame);
        sum += p;
        if constexpr (kBf16)
          pb[b][e] = (__bf16)p;
        else
          pf[b][e] = p;
      }
      l[b] = l[b] * fade + sum;
      if (!__all(fade == 1.0f)) {
#pragma unroll
        for (int d = 0; d < kDB; ++d) acc[b][d] *= fade;
      }
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
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int k = 16 * (e >> 2) + 4 * g + (e & 3);
        const int32_t p = __shfl(page_now, k);
        const char* src = a.cache.values + a.cache.row(p < 0 ? 0 : p, head, s0 + k) * (D * 4) + col * 4;
#pragma unroll
        for (int d = 0; d < kDB; ++d) {
          float v = *reinterpret_cast<const float*>(src + d * 64);
          if (p < 0) v = 0.0f;
#pragma unroll
          for (int b = 0; b < QB; ++b)
            acc[b][d] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, pf[b][e], acc[b][d], 0, 0, 0);
        }
      }
    }
  }

  // the four waves' sums in one frame
  __syncthreads();
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
  const int64_t unit = (tile * a.cache.n_heads + head) * a.splits + split;
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    const int64_t c = at.c0 + 16 * b + col;
    if (c >= columns) continue;
    const int64_t j = c / a.G;
    if (a.splits > 1) {
      const int64_t u = unit * S::kColumns + 16 * b + col;
      if (g == 0) {
        a.stats[2 * u] = top[b];
        a.stats[2 * u + 1] = sum[b];
      }
      if (sum[b] > 0.0f) {
#pragma unroll
        for (int d = 0; d < kDB; ++d) *reinterpret_cast<f32x4*>(a.part + u * D + 16 * d + 4 * g) = acc[b][d];
      }
    } else {
      const int64_t h = (int64_t)head * a.G + (c - j * a.G);
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
}

// Joins the splits of a tile's columns: D / 4 lanes per column.
template <class E, int D, int QB>
__global__ __launch_bounds__(kThreads) void join(AttendArgs a) {
  constexpr int kColumns = 16 * QB, kLanes = D / 4, kPer = kThreads / kLanes;
  const int t = threadIdx.x;
  const int32_t head = (int32_t)(blockIdx.x % a.cache.n_heads);
  const int64_t tile = blockIdx.x / a.cache.n_heads;
  const TileOf at = tile_of<kColumns>(a, tile);
  if (at.r.index < 0) return;
  const int64_t columns = ((int64_t)at.r.k + 1) * a.G;
  const int64_t unit = (tile * a.cache.n_heads + head) * a.splits;
  for (int x = t / kLanes; x < kColumns; x += kPer) {
    const int64_t c = at.c0 + x;
    if (c >= columns) break;
    float top = -__builtin_inff();
    for (int s = 0; s < a.splits; ++s) top = fmaxf(top, a.stats[2 * ((unit + s) * kColumns + x)]);
    f32x4 o = f32x4{0, 0, 0, 0};
    float sum = 0.0f;
    for (int s = 0; s < a.splits; ++s) {
      const int64_t u = (unit + s) * kColumns + x;
      const float w = a.stats[2 * u + 1];
      if (!(w > 0.0f)) continue;
      const float fade = fast_exp2(a.stats[2 * u] - top);
      sum += w * fade;
      o += *reinterpret_cast<const f32x4*>(a.part + u * D + (t % kLanes) * 4) * fade;
    }
    o *= sum > 0.0f ? 1.0f / sum : 0.0f;
    const int64_t j = c / a.G, h = (int64_t)head * a.G + (c - j * a.G);
    char* dst = a.out + ((at.r.row0 + j) * a.n_q + h) * (D * E::kBytes) + (t % kLanes) * 4 * E::kBytes;
    if constexpr (E::kBytes == 2) {
      bf16x4 w;
      for (int e = 0; e < 4; ++e) w[e] = (__bf16)o[e];
      *reinterpret_cast<bf16x4*>(dst) = w;
    } else {
      *reinterpret_cast<f32x4*>(dst) = o;
    }
  }
}

struct Plan {
  int qb;
  int32_t splits;
  int64_t tiles;
  size_t part_bytes, bytes;
};

inline size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

inline Plan plan_of(const sdv_cache* c, int32_t B, int64_t n_d, int32_t n_q, int32_t window, int32_t sinks) {
  const int64_t G = n_q / c->n_kv_heads, rows = n_d + B, mean = (rows * G + B - 1) / B;
  Plan p;
  p.qb = mean <= 16 ? 1 : 2;
  if (mean > 48 && c->dtype == SDV_BF16 && c->head_dim <= 128) p.qb = 4;
  const int64_t columns = 16 * p.qb;
  p.tiles = rows * G / columns + B;
  // splits: enough workgroups to fill the card, each with two tiles per wave
  const int64_t busy = (rows * G / columns > B ? rows * G / columns : B) * c->n_kv_heads;
  int64_t seen = (int64_t)c->max_pages * c->page_size;
  if (window && (int64_t)window + sinks + rows / B < seen) seen = (int64_t)window + sinks + rows / B;
  int64_t splits = (1024 + busy - 1) / busy;
  const int64_t most = seen / (kWaves * kTile * 2);
  if (splits > most) splits = most;
  if (splits > 64) splits = 64;
  p.splits = splits < 1 ? 1 : (int32_t)splits;
  p.part_bytes = p.bytes = 0;
  if (p.splits > 1) {
    const int64_t units = p.tiles * c->n_kv_heads * p.splits * columns;
    p.part_bytes = up256((size_t)units * c->head_dim * 4);
    p.bytes = p.part_bytes + up256((size_t)units * 8);
  }
  return p;
}

template <class E, int D, int QB>
int launch(const AttendArgs& a, hipStream_t s) {
  const int64_t grid = a.tiles * a.cache.n_heads;
  hipLaunchKernelGGL((attend<E, D, QB>), dim3((unsigned)(grid * a.splits)), dim3(kThreads), 0, s, a);
  if (a.splits > 1) hipLaunchKernelGGL((join<E, D, QB>), dim3((unsigned)grid), dim3(kThreads), 0, s, a);
  return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
}

template <class E, int D>
int launch_columns(const AttendArgs& a, int qb, hipStream_t s) {
  if (qb == 1) return launch<E, D, 1>(a, s);
  if constexpr (E::kBytes == 2 && D <= 128) {
    if (qb == 4) return launch<E, D, 4>(a, s);
  }
  return launch<E, D, 2>(a, s);
}

template <class E>
int launch_dim(const AttendArgs& a, int32_t D, int qb, hipStream_t s) {
  return D == 64 ? launch_columns<E, 64>(a, qb, s)
                 : (D == 128 ? launch_columns<E, 128>(a, qb, s) : launch_columns<E, 256>(a, qb, s));
}

inline int check(const sdv_cache* c, int32_t B, int64_t n_d, int32_t n_q, int32_t window, int32_t sinks) {
  if (n_q < 1 || n_q % c->n_kv_heads || window < 0 || sinks < 0) return SDV_ERR_INVALID_ARG;
  if (n_q > 1024) return SDV_ERR_LIMIT;
  const Plan p = plan_of(c, B, n_d, n_q, window, sinks);
  return p.tiles * c->n_kv_heads * p.splits > INT32_MAX ? SDV_ERR_LIMIT : SDV_OK;
}

}  // namespace attend_impl

extern "C" size_t sdv_attend_workspace_bytes(const sdv_cache* cache, int32_t B, int64_t n_draft_rows,
                                             int32_t n_q_heads, int32_t window, int32_t sinks) {
  using namespace attend_impl;
  if (!cache || B < 1 || n_draft_rows < 0 || cache->n_kv_heads < 1 || cache->max_pages < 1 || cache->page_size < 1 ||
      n_draft_rows + B > INT32_MAX || check(cache, B, n_draft_rows, n_q_heads, window, sinks) != SDV_OK)
    return 0;
  return plan_of(cache, B, n_draft_rows, n_q_heads, window, sinks).bytes;
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
  if (!queries || !out || !aligned16(queries) || !aligned16(out) || query_stride % per ||
      query_stride < (int64_t)n_q_heads * cache->head_dim || !(scale - scale == 0.0f))
    return SDV_ERR_INVALID_ARG;
  if (query_stride > ((int64_t)1 << 31)) return SDV_ERR_LIMIT;
  const Plan p = plan_of(cache, B, n_draft_rows, n_q_heads, window, sinks);
  if (p.bytes > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < p.bytes)) return SDV_ERR_WORKSPACE;
  AttendArgs a;
  a.cache = view_of(cache);
  a.B = B;
  a.n_q = n_q_heads;
  a.G = n_q_heads / cache->n_kv_heads;
  a.splits = p.splits;
  a.window = window;
  a.sinks = sinks;
  a.n_d = n_draft_rows;
  a.query_stride = query_stride;
  a.tiles = p.tiles;
  a.scale2 = scale * 1.4426950408889634f;
  a.cu = ragged_offsets;
  a.parents = parents;
  a.queries = static_cast<const char*>(queries);
  a.out = static_cast<char*>(out);
  a.part = static_cast<float*>(workspace);
  a.stats = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.part_bytes);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  return cache->dtype == SDV_BF16 ? launch_dim<Bf16>(a, cache->head_dim, p.qb, s)
                                  : launch_dim<F32>(a, cache->head_dim, p.qb, s);
}
