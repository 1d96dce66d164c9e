// Drafting: one token per row from its logits under a sampling profile (temperature, top-k, top-p,
// min-p) and a given uniform, with the probability row it was drawn from (the q row that the
// verification takes as draft_probs).
//
// With z_max the row's largest logit, w_v = exp((z_v - z_max) / T).  Tokens rank by logit, equal
// logits by the smaller id.  Every truncation keeps a run of leading ranks, so the kept set is one
// cut: the order key of the last kept rank and the id of its last kept copy.  The token is
// min{v : C(v) > u S} over the kept weights in ascending id, S their sum.
//
// Which token a uniform lands on is decided by sums over up to V weights, and a border between two
// tokens of a flat row of 128256 is 8e-6 S wide: binary32 weights would put a few draws in a
// thousand on the neighbour.  Weights and sums are therefore binary64 (the weight to 2e-12), and
// every sum has a fixed order, so the token is that of the definition and the same on every run.
//
// Three passes: row_stats streams every row once (a wave per chunk of 64 lanes x kVpl vectors:
// maximum and sum), row_draw finishes each row in one workgroup (fold, cut, pick a chunk by prefix
// sums, search that chunk), and row_probs, when the probability rows are asked for, streams
// them out.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/sdv.h"
#include "sdv_device.hpp"

namespace sample_impl {

using namespace sdv;

constexpr int kStatsWaves = 4;
constexpr int kDrawThreads = 1024;
constexpr int kDrawWaves = kDrawThreads / kWave;
constexpr int kBins = 2048;

struct Record {  // one chunk of a row: sum of weights in the frame of its own maximum
  double s;
  float m;
  uint32_t eq;  // copies of the cut's key in the chunk (truncated rows)
};

struct RowState {  // what row_probs needs of a row
  double m, k2, inv_s;
  uint32_t key;   // kept: order key above this, or equal to it at an id of at most last
  int32_t last;
  int32_t token;  // kOneToken
  int32_t kind;
  int64_t slot;
};
enum Kind { kDistribution, kOneToken, kNothing, kSkipped };  // kNothing: a row of zeros

struct Args {
  const void* logits;
  int64_t n, stride, n_slots;
  int32_t V, C;
  double T;
  const float* temperature;
  const int32_t* top_k;
  const int32_t* top_p;
  const float* min_p;
  const double* uniform;
  const int32_t* slots;
  int32_t* tokens;
  float* prob;
  int32_t* kept;
  float* probs;
  Record* rec;
  RowState* state;
};

// A row as the 16-byte vectors of the aligned blocks that hold it: elements [lead, end) counted
// from base are the row's; what a block holds beside them is not read.
template <class E>
struct RowView {
  const char* base;
  int32_t lead, end;
  __device__ RowView(const Args& a, int64_t row) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.logits) + (uintptr_t)(row * a.stride * E::kBytes);
    lead = (int32_t)(p & 15) / E::kBytes;
    base = reinterpret_cast<const char*>(p & ~(uintptr_t)15);
    end = lead + a.V;
  }
  __device__ bool whole(int32_t e0, int32_t n) const { return e0 >= lead && (int64_t)e0 + n <= end; }
  __device__ u32x4 vec(int64_t j) const { return *reinterpret_cast<const u32x4*>(base + j * 16); }
  __device__ u32x4 vec_edge(int64_t j) const {  // a vector that may lie partly or wholly outside
    u32x4 v;
    v.x = v.y = v.z = v.w = E::kNegInfWord;
    const int64_t e0 = j * E::kPerVec;
    if (e0 + E::kPerVec <= lead || e0 >= end) return v;
    if (e0 >= lead && e0 + E::kPerVec <= end) return vec(j);
#pragma unroll
    for (int i = 0; i < E::kPerVec; ++i) {
      const int64_t e = e0 + i;
      if (e < lead || e >= end) continue;
      uint32_t* w = reinterpret_cast<uint32_t*>(&v);
      if constexpr (E::kBytes == 4) {
        w[i] = reinterpret_cast<const uint32_t*>(base)[e];
      } else {
        const uint32_t h = reinterpret_cast<const uint16_t*>(base)[e];
        const int sh = (i & 1) * 16;
        w[i >> 1] = (w[i >> 1] & ~(0xffffu << sh)) | (h << sh);
      }
    }
    return v;
  }
  // The chunk's vectors of this lane, lane-interleaved (vector c0 + 64 i + lane).
  template <int kVpl>
  __device__ void chunk(int32_t c, int lane, u32x4 (&v)[kVpl]) const {
    const int64_t j0 = (int64_t)c * (kVpl * kWave);
    if (j0 * E::kPerVec >= lead && (j0 + kVpl * kWave) * E::kPerVec <= end) {
#pragma unroll
      for (int i = 0; i < kVpl; ++i) v[i] = vec(j0 + i * kWave + lane);
    } else {
#pragma unroll
      for (int i = 0; i < kVpl; ++i) v[i] = vec_edge(j0 + i * kWave + lane);
    }
  }
};

// 2^t for t = (z - m) k2 <= 0: t = n + r with |r| <= 1/2 by adding 1.5 x 2^52, and 2^r = 1 + r q(r)
// with q the interpolation of (2^r - 1) / r at the eight Chebyshev nodes (relative error 2.1e-12).
// -inf and NaN logits take the lower bound of d, whose weight is 0.
struct Frame {
  double m, k2, d_min;
  __device__ Frame(double m_, double k2_) : m(m_), k2(k2_), d_min(-1100.0 / k2_) {}
  __device__ double weight(float z) const {
    constexpr double kMagic = 0x1.8p52;
    const double d = fmax((double)z - m, d_min);
    const double y = fma(d, k2, kMagic);
    const double r = fma(d, k2, kMagic - y);
    double q = 0x1.63b2d7967b894p-20;
    q = fma(q, r, 0x1.00c0e4e14e280p-16);
    q = fma(q, r, 0x1.4308c7183de44p-13);
    q = fma(q, r, 0x1.5d8775983512bp-10);
    q = fma(q, r, 0x1.3b2ab70ad2562p-7);
    q = fma(q, r, 0x1.c6b08da70cce3p-5);
    q = fma(q, r, 0x1.ebfbdff82a734p-3);
    q = fma(q, r, 0x1.62e42fef9cc69p-1);
    return __builtin_amdgcn_ldexp(fma(q, r, 1.0), __double2loint(y));
  }
};

// Unsigned order of the keys is the order of the logits; -0 shares +0's key, NaN shares -inf's.
__device__ __forceinline__ uint32_t order_key(float z) {
  uint32_t u = __float_as_uint(z);
  if ((u << 1) > 0xff000000u) u = 0xff800000u;
  if (u == 0x80000000u) u = 0;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key & 0x7fffffffu) : ~key);
}
// A key of a bf16 logit: the low 16 bits follow from the sign, so keys are compared without them.
template <class E>
__device__ __forceinline__ uint32_t row_key(float z) {
  const uint32_t k = order_key(z);
  return E::kBytes == 2 ? (k | 0xffffu) : k;
}
template <class E>
__device__ __forceinline__ float row_key_logit(uint32_t key) {
  if constexpr (E::kBytes == 2) key = (key & 0x80000000u) ? (key & 0xffff0000u) : key;
  return key_logit(key);
}

template <class E>
__device__ __forceinline__ const char* row_ptr_strided(const Args& a, int64_t row) {
  return static_cast<const char*>(a.logits) + row * a.stride * E::kBytes;
}

struct Profile {
  double T;
  int32_t k, p;
  float min_p;
  bool ok, greedy, cut, top_k, top_p;
};

__device__ __forceinline__ Profile profile_of(const Args& a, int64_t row) {
  Profile f;
  f.T = a.temperature ? (double)a.temperature[row] : a.T;
  f.k = a.top_k ? a.top_k[row] : 0;
  f.p = a.top_p ? a.top_p[row] : 1000;
  f.min_p = a.min_p ? a.min_p[row] : 0.0f;
  f.greedy = f.T == 0.0;
  f.ok = f.greedy || (f.T > 0.0 && f.T < __builtin_inf() && f.k >= 0 && f.p >= 0 && f.p <= 1000 && f.min_p >= 0.0f &&
                      f.min_p <= 1.0f);
  f.top_k = f.k > 0 && f.k < a.V;
  f.top_p = f.p < 1000;
  f.cut = !f.greedy && (f.top_k || f.top_p || f.min_p > 0.0f);
  return f;
}

__device__ __forceinline__ int64_t slot_of(const Args& a, int64_t row) {
  if (!a.slots) return row;
  const int32_t s = a.slots[row];
  return s >= 0 && s < a.n_slots ? s : -1;
}

constexpr double kLog2e = 0x1.71547652b82fep0;

template <class E, int kVpl>
__global__ __launch_bounds__(kStatsWaves* kWave) void row_stats(Args a) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t unit =
      (int64_t)blockIdx.x * kStatsWaves + __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
  if (unit >= a.n * a.C) return;
  const int64_t row = unit / a.C;
  const int32_t c = (int32_t)(unit - row * a.C);
  if (slot_of(a, row) < 0) return;
  const RowView<E> view(a, row);
  u32x4 v[kVpl];
  view.template chunk<kVpl>(c, lane, v);
  const Profile f = profile_of(a, row);
  float m = -__builtin_inff();
#pragma unroll
  for (int i = 0; i < kVpl; ++i) {
    float z[E::kPerVec];
    E::unpack(v[i], z);
#pragma unroll
    for (int e = 0; e < E::kPerVec; ++e) m = fmaxf(m, z[e]);
  }
  m = wave_max(m);
  double s = 0.0;
  if (f.ok && !f.greedy && !f.cut) {  // a cut row's sums wait for the cut
    const Frame frame(m, kLog2e / f.T);
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
      float z[E::kPerVec];
      E::unpack(v[i], z);
#pragma unroll
      for (int e = 0; e < E::kPerVec; ++e) s += frame.weight(z[e]);
    }
    s = wave_sum(s);
  }
  if (lane == 0) {
    Record r;
    r.s = s;
    r.m = m;
    r.eq = 0;
    a.rec[unit] = r;
  }
}

struct Shared {
  uint64_t hist[kBins];
  double wave_d[kDrawWaves];
  uint64_t wave_u[kDrawWaves];
  float wave_f[kDrawWaves];
  uint64_t found_before, found_at;
  double before;
  uint32_t found_bin, key;
  int32_t chunk, first, last, eq_last;
};

// Exclusive prefix over the workgroup's threads in thread order; total in every thread.
__device__ __forceinline__ double block_scan(double v, double* wave_d, double& total) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const double inc = wave_detail::inclusive_scan(v);
  __syncthreads();
  if (lane == kWave - 1) wave_d[wave] = inc;
  __syncthreads();
  double base = 0.0;
  total = 0.0;
  for (int w = 0; w < kDrawWaves; ++w) {
    if (w == wave) base = total;
    total += wave_d[w];
  }
  return base + (inc - v);
}
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* wave_u, uint64_t& total) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const uint64_t inc = wave_inclusive_scan(v);
  __syncthreads();
  if (lane == kWave - 1) wave_u[wave] = inc;
  __syncthreads();
  uint64_t base = 0;
  total = 0;
  for (int w = 0; w < kDrawWaves; ++w) {
    if (w == wave) base = total;
    total += wave_u[w];
  }
  return base + (inc - v);
}

// Every element of the row once, each chunk by one wave: f(z) for the row's own elements (padding
// arrives as -inf and must not count, so its place decides).
template <class E, int kVpl, class F>
__device__ __forceinline__ void each_element(const RowView<E>& view, int32_t C, F f) {
  const int lane = threadIdx.x & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
  for (int32_t c = wave; c < C; c += kDrawWaves) {
    u32x4 v[kVpl];
    view.template chunk<kVpl>(c, lane, v);
    const int64_t j0 = (int64_t)c * (kVpl * kWave) + lane;
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
      float z[E::kPerVec];
      E::unpack(v[i], z);
#pragma unroll
      for (int e = 0; e < E::kPerVec; ++e) {
        const int64_t at = (j0 + i * kWave) * E::kPerVec + e;
        if (at >= view.lead && at < view.end) f(z[e]);
      }
    }
  }
}

struct Selected {
  uint32_t key;
  uint64_t before, at, need;  // the sums above the key and at it, and the sum that was to be reached
};

// The largest key at which the running sum of value(z), from the largest key down, reaches
// need_of(total): one pass of the row per digit (11 + 5 bits of a bf16 key, 11 + 11 + 10 of a
// binary32 key) fills a histogram of the keys that share the digits found so far.  Sums are
// integers, so the order of the adds changes nothing.
template <class E, int kVpl, class Value, class Need>
__device__ Selected radix_select(const RowView<E>& view, int32_t C, Shared& sh, Value value, Need need_of) {
  constexpr int kLevels = E::kBytes == 2 ? 2 : 3;
  const int t = threadIdx.x;
  Selected r;
  r.key = 0;
  r.before = r.need = r.at = 0;
  for (int level = 0; level < kLevels; ++level) {
    const int shift = level == 0 ? 21 : (E::kBytes == 2 ? 16 : (level == 1 ? 10 : 0));
    const int width = level == 0 ? 11 : (E::kBytes == 2 ? 5 : (level == 1 ? 11 : 10));
    const int bins = 1 << width;
    __syncthreads();
    for (int b = t; b < kBins; b += kDrawThreads) sh.hist[b] = 0;
    __syncthreads();
    each_element<E, kVpl>(view, C, [&](float z) {
      const uint32_t key = order_key(z);
      if (level > 0 && ((key ^ r.key) >> (shift + width)) != 0) return;
      const uint64_t x = value(z);
      if (x)
        atomicAdd(reinterpret_cast<unsigned long long*>(&sh.hist[(key >> shift) & (bins - 1)]), (unsigned long long)x);
    });
    __syncthreads();
    // two bins per thread, from the top bin down
    const int hi = bins - 1 - 2 * t, lo = hi - 1;
    const uint64_t x = hi >= 0 ? sh.hist[hi] : 0, y = lo >= 0 ? sh.hist[lo] : 0;
    uint64_t total;
    const uint64_t pre = block_scan(x + y, sh.wave_u, total);
    if (level == 0) r.need = need_of(total);
    const uint64_t want = r.need - r.before;
    if (pre < want && pre + x >= want) {
      sh.found_bin = hi;
      sh.found_before = r.before + pre;
      sh.found_at = x;
    } else if (pre + x < want && pre + x + y >= want) {
      sh.found_bin = lo;
      sh.found_before = r.before + pre + x;
      sh.found_at = y;
    }
    __syncthreads();
    r.key |= sh.found_bin << shift;
    r.before = sh.found_before;
    r.at = sh.found_at;
  }
  if (E::kBytes == 2) r.key |= 0xffffu;
  return r;
}

template <class E, int kVpl>
__global__ __launch_bounds__(kDrawThreads) void row_draw(Args a) {
  __shared__ Shared sh;
  constexpr int kVecs = kVpl * kWave;  // vectors of a chunk
  constexpr int P = E::kPerVec;
  static_assert(kVecs <= kDrawThreads, "one vector of a chunk per thread");
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int64_t row = blockIdx.x;
  const int64_t slot = slot_of(a, row);
  RowState st;
  st.m = st.k2 = st.inv_s = 0.0;
  st.key = 0;
  st.last = 0x7fffffff;
  st.token = -1;
  st.kind = kSkipped;
  st.slot = slot;
  if (slot < 0) {
    if (a.probs && t == 0) a.state[row] = st;
    return;
  }
  const RowView<E> view(a, row);
  const Profile f = profile_of(a, row);
  Record* rec = a.rec + row * a.C;
  const int32_t C = a.C;

  float m = -__builtin_inff();
  for (int32_t c = t; c < C; c += kDrawThreads) m = fmaxf(m, rec[c].m);
  m = wave_max(m);
  if (lane == 0) sh.wave_f[wave] = m;
  if (t == 0) {
    sh.chunk = 0x7fffffff;
    sh.first = 0x7fffffff;
    sh.last = -1;
    sh.eq_last = 0x7fffffff;
  }
  __syncthreads();
  for (int w = 0; w < kDrawWaves; ++w) m = fmaxf(m, sh.wave_f[w]);

  const double u = f.greedy ? 0.0 : a.uniform[row];
  if (!f.ok || !(m > -__builtin_inff() && m < __builtin_inff()) || !(u >= 0.0 && u < 1.0)) {
    if (t == 0) {
      a.tokens[slot] = -1;
      a.prob[slot] = 0.0f;
      if (a.kept) a.kept[slot] = 0;
      st.kind = kNothing;
      if (a.probs) a.state[row] = st;
    }
    return;
  }

  if (f.greedy) {  // the first chunk that holds the maximum, then its first element
    for (int32_t c = t; c < C; c += kDrawThreads)
      if (rec[c].m == m) atomicMin(&sh.chunk, c);
    __syncthreads();
    const int64_t j = (int64_t)sh.chunk * kVecs + t;
    if (t < kVecs) {
      float z[P];
      E::unpack(view.vec_edge(j), z);
#pragma unroll
      for (int e = P - 1; e >= 0; --e)
        if (z[e] == m) atomicMin(&sh.first, (int32_t)(j * P + e - view.lead));
    }
    __syncthreads();
    if (t == 0) {
      a.tokens[slot] = sh.first;
      a.prob[slot] = 1.0f;
      if (a.kept) a.kept[slot] = 1;
      st.token = sh.first;
      st.kind = kOneToken;
      if (a.probs) a.state[row] = st;
    }
    return;
  }

  const Frame frame(m, kLog2e / f.T);
  uint32_t cut_key = 0;  // kept: keys above it, and its first cut_copies copies
  uint64_t cut_copies = ~0ull, k_copies_all = 0;
  if (f.top_k) {
    const uint64_t k = (uint64_t)f.k;
    const Selected r = radix_select<E, kVpl>(
        view, C, sh, [](float) { return (uint64_t)1; }, [k](uint64_t) { return k; });
    cut_key = r.key;
    cut_copies = k - r.before;
    k_copies_all = r.at;
  }
  if (f.top_p) {
    // Masses as integers, with room for V of them in 62 bits.  The copies of the top-k key behind
    // rank k count in the passes and are taken off the total; they rank last, so no prefix that
    // the smaller sum asks for reaches them.
    const int bits = 62 - (32 - __builtin_clz((unsigned)a.V));
    auto mass = [&](float z) { return (uint64_t)__builtin_rint(__builtin_amdgcn_ldexp(frame.weight(z), bits)); };
    const uint32_t k_key = cut_key;
    const uint64_t p = (uint64_t)f.p;
    const uint64_t over = f.top_k ? (k_copies_all - cut_copies) * mass(row_key_logit<E>(k_key)) : 0;
    const Selected r = radix_select<E, kVpl>(
        view, C, sh, [&](float z) { return row_key<E>(z) >= k_key ? mass(z) : (uint64_t)0; },
        [&](uint64_t total) {
          const uint64_t need = (uint64_t)(((unsigned __int128)(total - over) * p + 999) / 1000);
          return need ? need : (uint64_t)1;
        });
    const uint64_t one = mass(row_key_logit<E>(r.key));
    cut_key = r.key;
    cut_copies = (r.need - r.before + one - 1) / one;
  }
  if (f.min_p > 0.0f) {
    // the smallest key of weight min_p or more lies within rounding of z_max + T ln(min_p)
    if (wave == 0) {
      const float z0 = (float)((double)m + f.T * log((double)f.min_p));
      const int64_t step = E::kBytes == 2 ? 0x10000 : 1;
      const int64_t k = (int64_t)row_key<E>(z0) + (lane - 32) * step;
      const bool in = k >= 0 && k <= 0xffffffffll;
      const bool reach = in && frame.weight(row_key_logit<E>((uint32_t)k)) >= (double)f.min_p;
      const uint64_t who = __ballot(reach);
      if (who && lane == __ffsll((unsigned long long)who) - 1) sh.key = (uint32_t)k;
      if (!who && lane == 0) sh.key = row_key<E>(m);
    }
    __syncthreads();
    if (sh.key > cut_key) {
      cut_key = sh.key;
      cut_copies = ~0ull;
    }
  }

  int64_t n_kept = a.V;
  if (f.cut) {
    // each chunk's mass above the cut and its copies of the cut's key
    uint32_t above = 0;
    for (int32_t c = wave; c < C; c += kDrawWaves) {
      u32x4 v[kVpl];
      view.template chunk<kVpl>(c, lane, v);
      const int64_t j0 = (int64_t)c * kVecs + lane;
      double s = 0.0;
      uint32_t eq = 0;
#pragma unroll
      for (int i = 0; i < kVpl; ++i) {
        float z[P];
        E::unpack(v[i], z);
#pragma unroll
        for (int e = 0; e < P; ++e) {
          const int64_t at = (j0 + i * kWave) * P + e;
          const uint32_t key = row_key<E>(z[e]);
          if (key < cut_key || at < view.lead || at >= view.end) continue;
          if (key == cut_key) {
            ++eq;
          } else {
            ++above;
            s += frame.weight(z[e]);
          }
        }
      }
      s = wave_sum(s);
      eq = wave_sum_u32(eq);
      if (lane == 0) {
        rec[c].s = s;
        rec[c].eq = eq;
      }
    }
    uint64_t n_above;
    (void)block_scan((uint64_t)above, sh.wave_u, n_above);
    __syncthreads();
    // the kept copies, first chunk first
    const double one = frame.weight(row_key_logit<E>(cut_key));
    uint64_t seen = 0;
    for (int32_t c0 = 0; c0 < C; c0 += kDrawThreads) {
      const int32_t c = c0 + t;
      const uint64_t eq = c < C ? rec[c].eq : 0;
      uint64_t total;
      const uint64_t pre = seen + block_scan(eq, sh.wave_u, total);
      const uint64_t take = pre >= cut_copies ? 0 : (cut_copies - pre < eq ? cut_copies - pre : eq);
      if (c < C) rec[c].s += (double)take * one;
      if (take > 0 && take < eq) {  // the cut runs through this chunk's copies
        sh.chunk = c;
        sh.found_before = take;
      } else if (take == eq && eq > 0 && pre + eq == cut_copies) {  // or behind its last one
        sh.chunk = c;
        sh.found_before = take;
      }
      seen += total;
    }
    __syncthreads();
    n_kept = (int64_t)(n_above + (cut_copies < seen ? cut_copies : seen));
    if (cut_copies < seen) {
      const int64_t j = (int64_t)sh.chunk * kVecs + t;
      const uint64_t want = sh.found_before;
      uint64_t eq = 0;
      float z[P];
      E::unpack(view.vec_edge(t < kVecs ? j : 0), z);
      auto is = [&](int e) {
        const int64_t at = j * P + e;
        return t < kVecs && at >= view.lead && at < view.end && row_key<E>(z[e]) == cut_key;
      };
#pragma unroll
      for (int e = 0; e < P; ++e) eq += is(e);
      uint64_t total;
      uint64_t pre = block_scan(eq, sh.wave_u, total);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        if (!is(e)) continue;
        if (++pre == want) sh.eq_last = (int32_t)(j * P + e - view.lead);
      }
      __syncthreads();
    }
  }
  const int32_t eq_last = sh.eq_last;

  // S, and the chunk the uniform lands in
  auto mass_of = [&](int32_t c) {
    return c < C ? (f.cut ? rec[c].s : rec[c].s * frame.weight(rec[c].m)) : 0.0;
  };
  double S = 0.0;
  for (int32_t c0 = 0; c0 < C; c0 += kDrawThreads) {
    double total;
    (void)block_scan(mass_of(c0 + t), sh.wave_d, total);
    S += total;
  }
  const double target = u * S;
  if (t == 0) sh.chunk = 0x7fffffff;
  double carry = 0.0;
  for (int32_t c0 = 0; c0 < C; c0 += kDrawThreads) {
    double total;
    const double x = mass_of(c0 + t);
    const double pre = carry + block_scan(x, sh.wave_d, total);
    if (x > 0.0 && pre + x > target) atomicMin(&sh.chunk, c0 + t);
    if (x > 0.0) atomicMax(&sh.last, c0 + t);
    __syncthreads();
    if (sh.chunk == c0 + t) sh.before = pre;
    carry += total;
  }
  __syncthreads();
  // u S within rounding of S: the last chunk with a kept weight, and its last kept token
  const bool past = sh.chunk == 0x7fffffff;
  const int32_t chunk = past ? sh.last : sh.chunk;
  const double before = past ? 0.0 : sh.before;
  __syncthreads();
  if (t == 0) sh.last = -1;
  const int64_t j = (int64_t)chunk * kVecs + t;
  double w[P], sum = 0.0;
  {
    float z[P];
    E::unpack(view.vec_edge(t < kVecs ? j : 0), z);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const int64_t at = j * P + e;
      bool keep = t < kVecs && at >= view.lead && at < view.end;
      if (f.cut) {
        const uint32_t key = row_key<E>(z[e]);
        keep = keep && (key > cut_key || (key == cut_key && at - view.lead <= eq_last));
      }
      w[e] = keep ? frame.weight(z[e]) : 0.0;
      sum += w[e];
    }
  }
  double total;
  double run = before + block_scan(sum, sh.wave_d, total);
#pragma unroll
  for (int e = 0; e < P; ++e) {
    if (!(w[e] > 0.0)) continue;
    run += w[e];
    const int32_t id = (int32_t)(j * P + e - view.lead);
    if (!past && run > target) atomicMin(&sh.first, id);
    atomicMax(&sh.last, id);
  }
  __syncthreads();
  const int32_t y = sh.first != 0x7fffffff ? sh.first : sh.last;
#pragma unroll
  for (int e = 0; e < P; ++e) {
    if (t < kVecs && w[e] > 0.0 && (int32_t)(j * P + e - view.lead) == y) {
      a.tokens[slot] = y;
      a.prob[slot] = (float)(w[e] / S);
      if (a.kept) a.kept[slot] = (int32_t)n_kept;
    }
  }
  if (a.probs && t == 0) {
    st.m = (double)m;
    st.k2 = frame.k2;
    st.inv_s = 1.0 / S;
    st.key = cut_key;
    st.last = eq_last;
    st.kind = kDistribution;
    a.state[row] = st;
  }
}

constexpr int kProbThreads = 256;
constexpr int kProbTile = 2048;

template <class E>
__global__ __launch_bounds__(kProbThreads) void row_probs(Args a, int32_t tiles) {
  const int64_t row = blockIdx.x / tiles;
  const int32_t v0 = (int32_t)(blockIdx.x - row * tiles) * kProbTile;
  const RowState st = a.state[row];
  if (st.kind == kSkipped) return;
  float* out = a.probs + st.slot * a.V;
  const char* in = row_ptr_strided<E>(a, row);
  const float scale = (float)st.inv_s;
  for (int32_t v = v0 + threadIdx.x; v < v0 + kProbTile && v < a.V; v += kProbThreads) {
    float p = 0.0f;
    if (st.kind == kOneToken) {
      p = v == st.token ? 1.0f : 0.0f;
    } else if (st.kind == kDistribution) {
      const float z = E::at(in, v);
      const uint32_t key = row_key<E>(z);
      if (key > st.key || (key == st.key && v <= st.last)) {
        // the exponent in binary64, its fraction alone through the binary32 exponential
        const double d = fmax((double)z - st.m, -1100.0 / st.k2) * st.k2;
        const double n = __builtin_rint(d);
        p = __builtin_amdgcn_ldexpf(fast_exp2((float)(d - n)) * scale, (int)n);
      }
    }
    out[v] = p;
  }
}

// Units below which the chunks are a quarter as long, so that a small batch spreads over the card.
constexpr int64_t kFullUnits = 1024;

template <class E>
constexpr int32_t chunk_elems(int vpl) {
  return vpl * kWave * E::kPerVec;
}

struct Plan {
  int vpl;
  int32_t C;
  size_t rec_bytes, bytes;
};

inline size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Chunks of a row of V elements that may begin anywhere in its first 16-byte block.
inline Plan plan_of(int64_t n, int32_t V, int32_t dtype) {
  const int64_t per = dtype == SDV_BF16 ? 8 : 4, vecs = ((int64_t)V + 2 * per - 2) / per;
  Plan p;
  p.vpl = n * ((vecs + 16 * kWave - 1) / (16 * kWave)) >= kFullUnits ? 16 : 4;
  p.C = (int32_t)((vecs + p.vpl * kWave - 1) / (p.vpl * kWave));
  p.rec_bytes = up256((size_t)n * p.C * sizeof(Record));
  p.bytes = p.rec_bytes + up256((size_t)n * sizeof(RowState));
  return p;
}

template <class E, int kVpl>
int launch(const Args& a, hipStream_t stream) {
  const int64_t groups = (a.n * a.C + kStatsWaves - 1) / kStatsWaves;
  hipLaunchKernelGGL((row_stats<E, kVpl>), dim3((unsigned)groups), dim3(kStatsWaves * kWave), 0, stream, a);
  hipLaunchKernelGGL((row_draw<E, kVpl>), dim3((unsigned)a.n), dim3(kDrawThreads), 0, stream, a);
  if (a.probs) {
    const int32_t tiles = (int32_t)(((int64_t)a.V + kProbTile - 1) / kProbTile);
    hipLaunchKernelGGL((row_probs<E>), dim3((unsigned)(a.n * tiles)), dim3(kProbThreads), 0, stream, a, tiles);
  }
  return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
}

}  // namespace sample_impl

extern "C" size_t sdv_sample_workspace_bytes(int64_t n_rows, int32_t V, int32_t dtype) {
  using namespace sample_impl;
  if (n_rows < 1 || V < 1 || (dtype != SDV_BF16 && dtype != SDV_FP32)) return 0;
  return plan_of(n_rows, V, dtype).bytes;
}

extern "C" int sdv_sample(const void* logits, int64_t n_rows, int64_t row_stride, int32_t V, int32_t dtype,
                          double temperature, const double* uniform, const sdv_sample_options* options,
                          int32_t* tokens, float* prob, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace sample_impl;
  if (dtype != SDV_BF16 && dtype != SDV_FP32) return SDV_ERR_UNSUPPORTED;
  const uintptr_t size = dtype == SDV_BF16 ? 2 : 4;
  if (!logits || !uniform || !tokens || !prob || n_rows < 1 || V < 1 || row_stride < V ||
      reinterpret_cast<uintptr_t>(logits) % size)
    return SDV_ERR_INVALID_ARG;
  sdv_sample_options o = {};
  if (options) o = *options;
  if (!o.temperature && !(temperature >= 0.0 && temperature < __builtin_inf())) return SDV_ERR_INVALID_ARG;
  if (o.slots ? o.n_slots < 0 || o.n_slots > INT32_MAX : o.n_slots != 0) return SDV_ERR_INVALID_ARG;
  const Plan p = n_rows <= INT32_MAX ? plan_of(n_rows, V, dtype) : Plan();
  if (n_rows > INT32_MAX || V > INT32_MAX - 64 || row_stride > ((int64_t)1 << 40) ||
      n_rows * p.C > (int64_t)INT32_MAX || (o.probs && n_rows * (((int64_t)V + kProbTile - 1) / kProbTile) > INT32_MAX))
    return SDV_ERR_LIMIT;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < p.bytes) return SDV_ERR_WORKSPACE;
  Args a = {};
  a.logits = logits;
  a.n = n_rows;
  a.stride = row_stride;
  a.V = V;
  a.C = p.C;
  a.T = temperature;
  a.temperature = o.temperature;
  a.top_k = o.top_k;
  a.top_p = o.top_p_milli;
  a.min_p = o.min_p;
  a.uniform = uniform;
  a.slots = o.slots;
  a.n_slots = o.slots ? o.n_slots : n_rows;
  a.tokens = tokens;
  a.prob = prob;
  a.kept = o.kept_tokens;
  a.probs = o.probs;
  a.rec = static_cast<Record*>(workspace);
  a.state = reinterpret_cast<RowState*>(static_cast<char*>(workspace) + p.rec_bytes);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == SDV_BF16) return p.vpl == 16 ? launch<Bf16, 16>(a, s) : launch<Bf16, 4>(a, s);
  return p.vpl == 16 ? launch<F32, 16>(a, s) : launch<F32, 4>(a, s);
}
