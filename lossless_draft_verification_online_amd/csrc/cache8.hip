// The paged cache in 8 bits: sdv_kv_append8 turns the batch's keys and values into e4m3 codes under a power-of-two scale for
// each block of tokens and head, and sdv_kv_settle8 moves a verified tree's accepted path in them.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cache8_view.hpp"

namespace cache8_impl {

using namespace sdv;

constexpr int kThreads = 256, kWaves = kThreads / kWave;

struct Append8Args {
  Cache8View view;
  int32_t B, D, rotary, n_q;
  int32_t parts;      // workgroups of a block of tokens
  int64_t units;      // workgroups that write the cache; the rows' queries follow
  int64_t n_d, key_stride, value_stride, query_stride;
  const int32_t* cu;
  const int32_t* parents;
  const char* keys;
  const char* values;
  const float* inv_freq;
  const char* queries;
  char* queries_out;
};

// 8 values of a row as binary32.
template <class E>
__device__ __forceinline__ void load8(const char* src, float (&f)[8]) {
  if constexpr (E::kBytes == 2) {
    Bf16::unpack(*reinterpret_cast<const u32x4*>(src), f);
  } else {
    const u32x4 x = *reinterpret_cast<const u32x4*>(src), y = *reinterpret_cast<const u32x4*>(src + 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      f[e] = __uint_as_float(x[e]);
      f[4 + e] = __uint_as_float(y[e]);
    }
  }
}

// Values 8 at .. 8 at + 7 of a head, rotated: c and s are the position's cosines and sines.  o: half of |a| + |b| of a value's pair.
template <class E, bool kInterleaved>
__device__ __forceinline__ void load_rotated(const char* head, int at, int rotary, const float* c, const float* s,
                                             float (&f)[8], float (&o)[8]) {
  load8<E>(head + at * 8 * E::kBytes, f);
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.0f;
  if (at * 8 >= rotary) return;
  if constexpr (kInterleaved) {
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const float cs = c[at * 4 + e / 2], sn = s[at * 4 + e / 2], a = f[e], b = f[e + 1];
      f[e] = a * cs - b * sn;
      f[e + 1] = b * cs + a * sn;
      o[e] = o[e + 1] = 0.5f * fabsf(a) + 0.5f * fabsf(b);
    }
  } else {
    const int half = rotary / 16;  // in pieces of 8
    const bool first = at < half;
    load8<E>(head + (first ? at + half : at - half) * 8 * E::kBytes, o);
    const int f0 = (first ? at : at - half) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float cs = c[f0 + e], sn = s[f0 + e], a = f[e];
      f[e] = first ? a * cs - o[e] * sn : a * cs + o[e] * sn;
      o[e] = 0.5f * fabsf(a) + 0.5f * fabsf(o[e]);
    }
  }
}

// Codes of two values, at most 448, in the lower half.
__device__ __forceinline__ uint32_t codes_of(float x, float y) {
  return __builtin_amdgcn_cvt_pk_fp8_f32(__builtin_amdgcn_fmed3f(x, -448.0f, 448.0f), __builtin_amdgcn_fmed3f(y, -448.0f, 448.0f),
                                         0, false) & 0xffffu;
}
__device__ __forceinline__ uint2 codes_of(const float (&f)[8]) {
  return make_uint2(codes_of(f[0], f[1]) | codes_of(f[2], f[3]) << 16, codes_of(f[4], f[5]) | codes_of(f[6], f[7]) << 16);
}

// Cosine and sine of an angle in turns, at most half a turn either way, to 2^-50: the series around the next quarter.  (The library's
// take the registers of four waves.)
__device__ __forceinline__ void cos_sin(double turns, double& c, double& s) {
  const double quarter = rint(4.0 * turns), y = (turns - 0.25 * quarter) * 6.283185307179586, z = y * y;  // |y| <= pi / 4
  double a = 1.0 / 6402373705728000.0, b = 1.0 / 121645100408832000.0;  // 1 / 18!, 1 / 19!
  constexpr double kCos[] = {1.0 / 20922789888000.0, 1.0 / 87178291200.0, 1.0 / 479001600.0, 1.0 / 3628800.0,
                             1.0 / 40320.0,          1.0 / 720.0,         1.0 / 24.0,        0.5,
                             1.0};
  constexpr double kSin[] = {1.0 / 355687428096000.0, 1.0 / 1307674368000.0, 1.0 / 6227020800.0, 1.0 / 39916800.0,
                             1.0 / 362880.0,          1.0 / 5040.0,          1.0 / 120.0,        1.0 / 6.0,
                             1.0};
#pragma unroll
  for (int k = 0; k < 9; ++k) {
    a = kCos[k] - z * a;
    b = kSin[k] - z * b;
  }
  b *= y;
  const int q = (int)quarter & 3;
  const double u = q & 1 ? b : a, v = q & 1 ? a : b;
  c = q == 1 || q == 2 ? -u : u;
  s = q >= 2 ? -v : v;
}

// The code of a value in binary64, at most 448.
__device__ __forceinline__ uint32_t code_of(double x) {
  // cut to binary32 with the lost bits in the last one: the next rounding sees on which side it lies
  float f = __double2float_rz(x);
  if ((double)f != x) f = __uint_as_float(__float_as_uint(f) | 1);
  return __builtin_amdgcn_cvt_pk_fp8_f32(__builtin_amdgcn_fmed3f(f, -448.0f, 448.0f), 0.0f, 0, false) & 255u;
}

// The largest finite magnitude of 8 values, as bits of binary32; odd where one is not finite.
template <class E>
__device__ __forceinline__ uint32_t top_bits(const char* src, bool& odd) {
  uint32_t top = 0;
  auto take = [&](uint32_t bits) {
    top = bits < 0x7f800000u && bits > top ? bits : top;
    odd |= bits >= 0x7f800000u;
  };
  const u32x4 x = *reinterpret_cast<const u32x4*>(src);
  if constexpr (E::kBytes == 2) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      take((x[w] << 16) & 0x7fffffffu);
      take(x[w] & 0x7fff0000u);
    }
  } else {
    const u32x4 y = *reinterpret_cast<const u32x4*>(src + 16);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      take(x[w] & 0x7fffffffu);
      take(y[w] & 0x7fffffffu);
    }
  }
  return top;
}
// The byte of the least scale with top <= limit * scale, limit 256 times the number of mantissa bits `mantissa`.
__device__ __forceinline__ int32_t least_byte(uint32_t top, uint32_t mantissa) {
  return scale_byte((int32_t)((top + (0x7fffffu - mantissa)) >> 23) - 8);
}
constexpr uint32_t kKeyLimit = 0x1e0000, kValueLimit = 0x600000;  // 316 = 256 * 1.234375, 448 = 256 * 1.75

__device__ __forceinline__ uint32_t wave_max_bits(uint32_t v) {
  return wave_detail::all_reduce(v, [](uint32_t a, uint32_t b) { return a > b ? a : b; });
}

// The first block of tokens of request i among all: its rows lie in at most (K + 1) / block + 2 from there.
__device__ __forceinline__ int64_t first_block(const int32_t* cu, int32_t i, int32_t block_log2) {
  return ((int64_t)((uint32_t)(cu[i] + i)) >> block_log2) + 2 * (int64_t)i;
}

constexpr int kTurns = 16;  // tokens whose angles are held at once

// A workgroup takes some of the keys' and values' heads of a block of tokens (a wave each), or one row's queries.
//
// A block's scale is the least power of two that its largest magnitude fits under, which one pass over its rows finds; the
// second, which turns and rounds them, finds them in a cache.  That a wave holds the whole block of a head makes the scale its
// own: no atomics, no second launch, and codes that were there are brought to a larger scale by the same wave.  The scale is
// that of the values as given, since a rotation is not needed to know it (316 sqrt(2) < 448).
//
// Many rows are bound by memory: 4 prompts of 4096 rows at most, 100 MB, 20.8 us, 4.8 TB/s (a large copy's rate).  Few are bound by
// the chain of offsets, length, page, and rows: 256 requests of K in 0 .. 8, 27 MB, 14.0 us (5.7 at a copy's rate); one 5.4.  Binary32
// rows: 194 MB of prompts 45 us (40.5 at a copy's rate), the 256 requests 17.6 (10.9), one 6.0.
//
// Eight waves per SIMD leave 64 registers, of which the rare binary64 path takes part: with pairs half a rotation apart bf16 rows keep
// 4 registers in memory and binary32 ones 10; with neighbours, none.
// Slower: rows held in registers between the passes (with the rotation's operands they leave fewer waves), several heads to a
// wave, the tables of angles in binary64 (in the place of the few values that need it computing their own), the list of
// units in shared memory.
template <class E, bool kInterleaved>
__global__ __launch_bounds__(kThreads, 8) void append8(Append8Args a) {
  __shared__ float cos_s[kTurns][128], sin_s[kTurns][128];
  __shared__ int32_t parent_s[kWave], depth_s[kMaxNodes + 1];
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const CacheView& cache = a.view.cache;
  const int half = a.rotary / 2, pieces = a.D / 8;
  const bool is_cache = blockIdx.x < a.units;

  Request r;
  int64_t slot0 = 0, n_rows = 1, j0 = 0;  // the block's first row, how many, its number in the request
  int32_t part = 0, len;
  if (is_cache) {
    const int64_t unit = (uint32_t)blockIdx.x / (uint32_t)a.parts;
    part = (int32_t)((uint32_t)blockIdx.x - (uint32_t)unit * (uint32_t)a.parts);
    const int32_t log2 = a.view.block_log2;
    // the unit's block of request q: its first row and their number, none if the request does not have it
    auto block_of = [&](const Request& q, int32_t n) {
      if (q.index < 0 || !len_fits(n, q.k)) return false;
      const int64_t b = (n >> log2) + unit - first_block(a.cu, q.index, log2);
      const int64_t lo = (b << log2) > n ? b << log2 : n, hi = (b + 1) << log2;
      if (b < (n >> log2) || lo > (int64_t)n + q.k) return false;
      slot0 = lo;
      j0 = lo - n;
      n_rows = (hi < (int64_t)n + q.k + 1 ? hi : (int64_t)n + q.k + 1) - lo;
      return true;
    };
    r = request_at(a.cu, find_last(a.B, unit, [&](int32_t i) { return first_block(a.cu, i, log2); }), a.n_d);
    if (__builtin_expect(r.index < 0, 0))  // some offsets are not valid: every request is looked at
      r = request_at(a.cu, find_among(a.B, [&](int32_t i) { return block_of(request_at(a.cu, i, a.n_d), cache.len[i]); }),
                     a.n_d);
    if (r.index < 0) return;
    len = cache.len[r.index];
    if (!block_of(r, len)) return;
  } else {
    const int64_t row = (int64_t)blockIdx.x - a.units;
    r = request_of_row(a.cu, a.B, a.n_d, row);
    j0 = row - r.row0;
    if (r.index < 0 || j0 > r.k) return;
    len = cache.len[r.index];
    if (!len_fits(len, r.k)) return;
  }
  if (a.parents && !tree_depths(a.parents, r, parent_s, depth_s)) return;

  // the angle of row j's pair f in turns, reduced in binary64: far positions keep their phase
  auto turns_of = [&](int64_t j, int f) {
    const double angle =
        (double)(len + (a.parents ? (int64_t)depth_s[j] : j)) * (double)a.inv_freq[f] * 0.15915494309189535;
    return angle - rint(angle);
  };
  // cosines and sines of `n` tokens from row j on
  auto turn = [&](int64_t j, int n) {
    for (int x = t; x < n * half; x += kThreads) {
      const int token = (uint32_t)x / (uint32_t)half, f = x - token * half;
      sincospif(2.0f * (float)turns_of(j + token, f), &sin_s[token][f], &cos_s[token][f]);
    }
    __syncthreads();
  };

  if (!is_cache) {
    turn(j0, 1);
    const int64_t row = r.row0 + j0;
    for (int x = t; x < a.n_q * pieces; x += kThreads) {
      const int h = x / pieces, at = x - h * pieces;
      float f[8], o[8];
      load_rotated<E, kInterleaved>(a.queries + (row * a.query_stride + (int64_t)h * a.D) * E::kBytes, at, a.rotary, cos_s[0],
                                    sin_s[0], f, o);
      char* const dst = a.queries_out + ((row * a.n_q + h) * a.D + at * 8) * E::kBytes;
      u32x4 v, w;
      if constexpr (E::kBytes == 2) {
        typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
        bf16x8 o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = (__bf16)f[e];
        v = __builtin_bit_cast(u32x4, o);
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = __float_as_uint(f[e]);
          w[e] = __float_as_uint(f[4 + e]);
        }
        *reinterpret_cast<u32x4*>(dst + 16) = w;
      }
      *reinterpret_cast<u32x4*>(dst) = v;
    }
    return;
  }

  const int32_t n_k = cache.n_heads, task = part * kWaves + wave;
  const bool works = task < 2 * n_k, is_key = task < n_k;
  const int32_t head = is_key ? task : task - n_k;
  const int32_t page = cache.page(r.index, slot0);
  if (page < 0) return;  // of all waves: a block lies in one page
  const char* const src = (is_key ? a.keys : a.values) +
                          ((r.row0 + j0) * (is_key ? a.key_stride : a.value_stride) + (int64_t)head * a.D) * E::kBytes;
  const int64_t stride = (is_key ? a.key_stride : a.value_stride) * E::kBytes;
  const int per = kWave / pieces;  // tokens that a wave takes at once
  const int token = lane / pieces, at = lane % pieces;
  char* const line = (is_key ? cache.keys : cache.values) + cache.row(page, works ? head : 0, slot0) * a.D;
  uint8_t* const scale = (is_key ? a.view.key_scales : a.view.value_scales) + a.view.scale_at(page, works ? head : 0, slot0);
  int32_t byte = 0;
  bool odd = false;
  if (works) {
    uint32_t top = 0;
    for (int x = token; x < n_rows; x += per) {
      const uint32_t v = top_bits<E>(src + x * stride + at * 8 * E::kBytes, odd);
      top = v > top ? v : top;
    }
    odd = __any(odd);
    byte = least_byte(wave_max_bits(top), is_key ? kKeyLimit : kValueLimit);
    const int64_t first = slot0 >> a.view.block_log2 << a.view.block_log2;
    if (first < len) {  // (then slot0 is len)
      const int32_t old = scale_byte(*scale);
      if (old >= byte) {
        byte = old;
      } else {
        const int held = (int)(len - first);
        char* const from = line - (int64_t)held * a.D;
        for (int x = lane; x < held * pieces; x += kWave) {
          uint2* const p = reinterpret_cast<uint2*>(from + x * 8);
          uint2 v = *p;
          v.x = shifted_codes(v.x, byte - old);
          v.y = shifted_codes(v.y, byte - old);
          *p = v;
        }
      }
    }
    if (lane == 0) *scale = (uint8_t)byte;
  }
  const float by = __uint_as_float((uint32_t)(254 - byte) << 23);  // 1 / scale
  const bool turns = part * kWaves < n_k && half > 0;              // some wave has keys
  for (int64_t x0 = 0; x0 < n_rows; x0 += kTurns) {
    const int n = n_rows - x0 < kTurns ? (int)(n_rows - x0) : kTurns;
    if (turns) turn(j0 + x0, n);
    if (works) {
      for (int x = token; x < n; x += per) {
        float f[8], o[8];
        const char* const from = src + (x0 + x) * stride;
        uint2 codes, differ = make_uint2(0, 0);
        if (is_key && half > 0) {
          load_rotated<E, kInterleaved>(from, at, a.rotary, cos_s[x], sin_s[x], f, o);
          // Off by less than 2^-21 (|a| + |b|): 2^-23.4 for the rounded angle, 2^-23 for its cosine and sine, and two roundings.
          // What lies so near to a border between two codes that binary32 does not tell its side (about one value in 15 000)
          // goes on in binary64.
          const float slack = 0x1.2p-20f * by;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            f[e] = fmaf(f[e], by, -o[e] * slack);
            o[e] = fmaf(o[e], 2.0f * slack, f[e]);
          }
          codes = codes_of(f);
          differ = codes_of(o);
          differ.x ^= codes.x;
          differ.y ^= codes.y;
        } else {
          load8<E>(from + at * 8 * E::kBytes, f);
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] *= by;
          codes = codes_of(f);
        }
        if (odd) differ = make_uint2(~0u, ~0u);
        if (__builtin_expect((differ.x | differ.y) != 0, 0)) {
          uint64_t word = codes.x | (uint64_t)codes.y << 32, again = differ.x | (uint64_t)differ.y << 32;
          while (again) {
            const int e = (__ffsll((unsigned long long)again) - 1) / 8, i = at * 8 + e;
            again &= ~((uint64_t)255 << (8 * e));
            const float p = E::at(from, i);
            float q = 0.0f;
            double v = p;
            if (is_key && i < a.rotary) {
              const bool one = kInterleaved ? i % 2 == 0 : i < half;
              q = E::at(from, kInterleaved ? i ^ 1 : (one ? i + half : i - half));
              double c, s;
              cos_sin(turns_of(j0 + x0 + x, kInterleaved ? i / 2 : (one ? i : i - half)), c, s);
              v = one ? p * c - q * s : p * c + q * s;
            }
            const uint64_t code = p - p == 0.0f && q - q == 0.0f ? code_of(v * (double)by) : 0x7fu;
            word = (word & ~((uint64_t)255 << (8 * e))) | code << (8 * e);
          }
          codes = make_uint2((uint32_t)word, (uint32_t)(word >> 32));
        }
        *reinterpret_cast<uint2*>(line + (x0 + x) * a.D + at * 8) = codes;
      }
    }
    if (turns) __syncthreads();
  }
}

struct Settle8Args {
  Cache8View view;
  int64_t n_d, layer_bytes, layer_scales;
  const int32_t* cu;
  const int32_t* accepted_len;
  const int32_t* accepted_nodes;
  int32_t* new_len;
};

// One wave per request and (layer, keys or values, head): all accepted tokens' codes are read before any is written, and the
// scales of the blocks that they come from before those of the blocks that they go to.  Bound by the chain of offsets and lengths,
// nodes, pages, scales and rows: 64 trees in four layers 5.0 us, one in one layer 3.3 (by workgroups of four waves, of which most
// had nothing to move, 9.4 and 4.2).
template <int D>
__global__ __launch_bounds__(kWave) void settle8(Settle8Args a) {
  constexpr int kVecs = D / 16, kRows = kWave / kVecs, kGroups = kMaxNodes / kRows;  // of 16 bytes; rows that the wave moves at once
  __shared__ int64_t from_s[kMaxNodes], to_s[kMaxNodes];
  __shared__ int32_t shift_s[kMaxNodes], most_s[kMaxNodes];
  const CacheView& cache = a.view.cache;
  const int t = threadIdx.x;
  const int32_t i = blockIdx.x;
  const int32_t head = blockIdx.y % cache.n_heads, rest = blockIdx.y / cache.n_heads;
  char* const base = ((rest & 1) ? cache.values : cache.keys) + (rest >> 1) * a.layer_bytes;
  uint8_t* const scales = ((rest & 1) ? a.view.value_scales : a.view.key_scales) + (rest >> 1) * a.layer_scales;
  const Request r = request_at(a.cu, i, a.n_d);
  const int32_t len = cache.len[i], acc = a.accepted_len[i];
  bool ok = r.index >= 0 && len_fits(len, r.k) && acc >= 0 && acc <= r.k && r.k <= kMaxNodes;
  int32_t node = t;
  if (ok && t < acc) node = a.accepted_nodes[r.first + t];
  const int32_t before = __shfl_up(node, 1);
  ok = ok && __ballot(t < acc && !(node > (t ? before : -1) && node < r.k)) == 0;
  if (t == 0 && blockIdx.y == 0) a.new_len[i] = ok ? len + 1 + acc : len;
  if (!ok || acc == 0) return;

  const int32_t log2 = a.view.block_log2, block_0 = (len + 1) >> log2;  // of blocks of the sequence
  const int32_t first = block_0 << log2;                                // first slot of the block that acceptance begins in
  const int64_t src = (int64_t)len + 1 + node, dst = (int64_t)len + 1 + t;
  const int32_t block = (int32_t)(dst >> log2) - block_0;
  most_s[t] = 0;
  int64_t from = -1, to = -1, scale_to = -1;
  int32_t byte = 0, old = 0;
  if (t < acc) {
    const int32_t sp = cache.page(i, src), dp = cache.page(i, dst);
    if (dp >= 0) {
      to = cache.row(dp, head, dst);
      from = sp >= 0 ? cache.row(sp, head, src) : to;  // without a page to come from it stays what is there
      scale_to = a.view.scale_at(dp, head, dst);
      byte = scale_byte(scales[sp >= 0 ? a.view.scale_at(sp, head, src) : scale_to]);
      if (t == 0 && first <= len) old = scale_byte(scales[scale_to]);  // the first block holds slots up to len
    }
  }
  __syncthreads();
  if (to >= 0) atomicMax(&most_s[block], byte > old ? byte : old);
  __syncthreads();
  const int32_t most = t < acc ? most_s[block] : 0;
  from_s[t] = from;
  to_s[t] = to;
  shift_s[t] = to >= 0 ? most - byte : 0;
  __syncthreads();
  const int k = t % kVecs, d0 = t / kVecs;
  u32x4 v[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    if (g * kRows >= acc) break;
    const int32_t d = g * kRows + d0;
    if (from_s[d] >= 0) v[g] = *reinterpret_cast<const u32x4*>(base + from_s[d] * D + k * 16);
  }
  __syncthreads();  // all are read
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    if (g * kRows >= acc) break;
    const int32_t d = g * kRows + d0;
    if (from_s[d] < 0) continue;
    const int32_t shift = shift_s[d];
    if (shift > 0) {
#pragma unroll
      for (int w = 0; w < 4; ++w) v[g][w] = shifted_codes(v[g][w], shift);
    }
    if (shift > 0 || from_s[d] != to_s[d]) *reinterpret_cast<u32x4*>(base + to_s[d] * D + k * 16) = v[g];
  }
  // what the first block held up to len
  const int32_t held = lane_value(old, 0), up = lane_value(most, 0) - held;
  if (held > 0 && up > 0) {
    char* const at = base + (to_s[0] - (len + 1 - first)) * D;
    for (int x = t; x < (len + 1 - first) * kVecs; x += kWave) {
      u32x4* const p = reinterpret_cast<u32x4*>(at + x * 16);
      u32x4 w = *p;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = shifted_codes(w[e], up);
      *p = w;
    }
  }
  // a block's scale, by its first token
  if (to >= 0 && (t == 0 || block != (int32_t)((dst - 1) >> log2) - block_0)) scales[scale_to] = (uint8_t)most;
}

}  // namespace cache8_impl

extern "C" int sdv_kv_append8(const sdv_cache8* cache, int32_t B, int64_t n_draft_rows, const int32_t* ragged_offsets,
                              const int32_t* parents, const void* keys, int64_t key_stride, const void* values,
                              int64_t value_stride, const float* inv_freq, int32_t rotary, int32_t interleaved,
                              const void* queries, int64_t query_stride, int32_t n_q_heads, void* queries_out,
                              void* stream) {
  using namespace cache8_impl;
  const int rc = check_cache8(cache, B, n_draft_rows, ragged_offsets);
  if (rc != SDV_OK) return rc;
  const sdv_cache& c = cache->cache;
  const int64_t per = c.dtype == SDV_BF16 ? 8 : 4, row = (int64_t)c.n_kv_heads * c.head_dim;
  if (!keys || !values || !aligned16(keys) || !aligned16(values) || key_stride < row || value_stride < row ||
      key_stride % per || value_stride % per || rotary < 0 || rotary > c.head_dim || rotary % 16 ||
      (rotary > 0) != (inv_freq != nullptr) || n_q_heads < 0 || (n_q_heads > 0) != (queries != nullptr) ||
      (n_q_heads > 0) != (queries_out != nullptr))
    return SDV_ERR_INVALID_ARG;
  const int64_t q_row = (int64_t)n_q_heads * c.head_dim;
  if (n_q_heads > 0 && (!aligned16(queries) || !aligned16(queries_out) || query_stride < q_row || query_stride % per ||
                        (queries == queries_out && query_stride != q_row)))
    return SDV_ERR_INVALID_ARG;
  Append8Args a;
  a.view = view_of(cache);
  a.parts = (2 * c.n_kv_heads + kWaves - 1) / kWaves;
  a.units = (((n_draft_rows + B) >> a.view.block_log2) + 2 * (int64_t)B) * a.parts;
  const int64_t groups = a.units + (n_q_heads > 0 ? n_draft_rows + B : 0);
  if (too_many(n_draft_rows + B, kThreads) || too_many(groups, kThreads) || n_q_heads > 1024 ||
      key_stride > ((int64_t)1 << 31) || value_stride > ((int64_t)1 << 31) || query_stride > ((int64_t)1 << 31))
    return SDV_ERR_LIMIT;
  a.B = B;
  a.D = c.head_dim;
  a.rotary = rotary;
  a.n_q = n_q_heads;
  a.n_d = n_draft_rows;
  a.key_stride = key_stride;
  a.value_stride = value_stride;
  a.query_stride = query_stride;
  a.cu = ragged_offsets;
  a.parents = parents;
  a.keys = static_cast<const char*>(keys);
  a.values = static_cast<const char*>(values);
  a.inv_freq = inv_freq;
  a.queries = static_cast<const char*>(queries);
  a.queries_out = static_cast<char*>(queries_out);
  const dim3 grid((unsigned)groups), threads(kThreads);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (c.dtype == SDV_BF16) {
    if (interleaved)
      hipLaunchKernelGGL((append8<Bf16, true>), grid, threads, 0, s, a);
    else
      hipLaunchKernelGGL((append8<Bf16, false>), grid, threads, 0, s, a);
  } else {
    if (interleaved)
      hipLaunchKernelGGL((append8<F32, true>), grid, threads, 0, s, a);
    else
      hipLaunchKernelGGL((append8<F32, false>), grid, threads, 0, s, a);
  }
  return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
}

extern "C" int sdv_kv_settle8(const sdv_cache8* cache, int32_t n_layers, int32_t B, int64_t n_draft_rows,
                              const int32_t* ragged_offsets, const int32_t* accepted_len, const int32_t* accepted_nodes,
                              int32_t* new_len, void* stream) {
  using namespace cache8_impl;
  const int rc = check_cache8(cache, B, n_draft_rows, ragged_offsets);
  if (rc != SDV_OK) return rc;
  const sdv_cache& c = cache->cache;
  if (n_layers < 1 || !accepted_len || (n_draft_rows > 0 && !accepted_nodes) || !new_len) return SDV_ERR_INVALID_ARG;
  if ((int64_t)n_layers * c.n_kv_heads * 2 > 65535 || too_many(B, kThreads)) return SDV_ERR_LIMIT;
  // every workgroup of a request reads these while one of them writes new_len
  const int64_t word = sizeof(int32_t), own = B * word;
  if (overlap(new_len, own, c.cache_len, own) || overlap(new_len, own, accepted_len, own) ||
      overlap(new_len, own, ragged_offsets, own + word) || overlap(new_len, own, accepted_nodes, n_draft_rows * word) ||
      overlap(new_len, own, c.page_table, own * c.max_pages))
    return SDV_ERR_INVALID_ARG;
  Settle8Args a;
  a.view = view_of(cache);
  a.n_d = n_draft_rows;
  a.layer_bytes = c.n_pages * c.n_kv_heads * (int64_t)c.page_size * c.head_dim;
  a.layer_scales = c.n_pages * c.n_kv_heads * (int64_t)(c.page_size / cache->block);
  a.cu = ragged_offsets;
  a.accepted_len = accepted_len;
  a.accepted_nodes = accepted_nodes;
  a.new_len = new_len;
  const dim3 grid((unsigned)B, (unsigned)(n_layers * c.n_kv_heads * 2)), threads(kWave);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (c.head_dim == 64)
    hipLaunchKernelGGL(settle8<64>, grid, threads, 0, s, a);
  else if (c.head_dim == 128)
    hipLaunchKernelGGL(settle8<128>, grid, threads, 0, s, a);
  else
    hipLaunchKernelGGL(settle8<256>, grid, threads, 0, s, a);
  return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
}
