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
// A row that fits a workgroup's shared memory takes one launch (row_whole).  A longer one takes two:
// row_stats streams every row once, a wave per chunk of 64 lanes x kVpl vectors (sum of weights,
// maximum), and row_draw finishes each row in one workgroup: fold, cut, pick a chunk by prefix
// sums, search that chunk.  row_probs, when the probability rows are asked for, streams them out.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "../../include/sdv.h"
#include "launch.hpp"
#include "sdv_device.hpp"

namespace sample_impl {

using namespace sdv;

constexpr int kStatsWaves = 4;
constexpr int kDrawThreads = 1024;
constexpr int kWindow = 4096;  // bins of the counts below the maximum

struct Record {  // one chunk of a row
  double s;      // sum of weights: absolute ones, 2^(z k2), or with far those in the frame of m
  float m;       // maximum (of far chunks, and in rows that are cut or take their argmax)
  uint32_t far;  // truncated rows: copies of the cut's key
};

struct RowState {  // what row_probs needs of a row
  double base, k2;
  float inv_s;    // 1 / S, S taken into [1/2, 1)
  int32_t exp_s;  // by 2^exp_s
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
  typedef const __attribute__((address_space(1))) u32x4* Vectors;
  typedef const __attribute__((address_space(1))) uint16_t* Halves;
  typedef const __attribute__((address_space(1))) uint32_t* Words;
  static constexpr int P = E::kPerVec;
  uintptr_t base;
  int32_t lead, end;
  int32_t whole_lo, whole_hi;  // vectors that lie within the row
  __device__ RowView(const Args& a, int64_t row) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a.logits) + (uintptr_t)(row * a.stride * E::kBytes);
    lead = (int32_t)(p & 15) / E::kBytes;
    base = p & ~(uintptr_t)15;
    end = lead + a.V;
    whole_lo = lead ? 1 : 0;
    whole_hi = end / P;
  }
  __device__ __forceinline__ u32x4 vec(int64_t j) const { return reinterpret_cast<Vectors>(base)[j]; }
  static __device__ __forceinline__ u32x4 nothing() {
    u32x4 v;
    v.x = v.y = v.z = v.w = E::kNegInfWord;
    return v;
  }
  // Vector j element by element: the row's own, -inf beside them.
  __device__ u32x4 part(int32_t j) const {
    u32x4 v = nothing();
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int32_t e = j * P + i;
      if (e < lead || e >= end) continue;
      if constexpr (E::kBytes == 4) {
        w[i] = reinterpret_cast<Words>(base)[e];
      } else {
        const uint32_t h = reinterpret_cast<Halves>(base)[e];
        const int sh = (i & 1) * 16;
        w[i >> 1] = (w[i >> 1] & ~(0xffffu << sh)) | (h << sh);
      }
    }
    v.x = w[0];
    v.y = w[1];
    v.z = w[2];
    v.w = w[3];
    return v;
  }
  // N vectors of a lane, j0 + i * step, any of which may lie partly or wholly outside: the whole ones by
  // vector loads; at most two of a row are parts, and those are put in their places.
  template <int N>
  __device__ __forceinline__ void edge(int32_t j0, int32_t step, u32x4 (&v)[N]) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int32_t j = j0 + i * step;
      v[i] = nothing();
      if (j >= whole_lo && j < whole_hi) v[i] = vec(j);
    }
    bool head = false, tail = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int32_t j = j0 + i * step;
      head = head || (j == 0 && whole_lo > 0);
      tail = tail || (j == whole_hi && j >= whole_lo);
    }
    if (head) {
      const u32x4 p = part(0);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (j0 + i * step == 0) v[i] = p;
    }
    if (tail) {
      const u32x4 p = part(whole_hi);
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (j0 + i * step == whole_hi) v[i] = p;
    }
  }
  __device__ __forceinline__ u32x4 one(int32_t j) const {
    u32x4 v[1];
    edge<1>(j, 1, v);
    return v[0];
  }
  __device__ __forceinline__ bool inside(int32_t j0, int32_t n) const { return j0 >= whole_lo && j0 + n <= whole_hi; }
  // N vectors of this lane from j0, lane-interleaved (j0 + 64 i + lane).
  template <int N>
  __device__ __forceinline__ void load(int32_t j0, int lane, u32x4 (&v)[N]) const {
    if (inside(j0, N * kWave)) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = vec((int64_t)j0 + i * kWave + lane);
    } else {
      edge<N>(j0 + lane, kWave, v);
    }
  }
};

// 2^t: t = n + r with |r| <= 1/2 by adding 1.5 x 2^52, and 2^r = 1 + r q(r) with q the
// interpolation of (2^r - 1) / r at the eight Chebyshev nodes (relative error 2.1e-12).  t = d k2
// enters both steps unrounded; |t| is below 2^31.
__device__ __forceinline__ double exp2_of(double d, double k2) {
  constexpr double kMagic = 0x1.8p52;
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

// Weights relative to a base logit (the maximum: its weight is exactly 1, so sums of equal weights are exact).
// -inf and NaN take the lower bound of d, whose weight is 0.
struct Frame {
  double base, k2, d_min;
  __device__ Frame(double base_, double k2_) : base(base_), k2(k2_), d_min(-1100.0 / k2_) {}
  __device__ double weight(float z) const { return exp2_of(fmax((double)z - base, d_min), k2); }
};

// Absolute weights, without a maximum found first: binary64 holds 2^(z k2) for |z k2| < 1000.  Beyond, a weight
// becomes 0 or infinity and the sum of a chunk that leaves [2^-900, 2^1000] says so.
struct NearFrame {
  double k2;
  float lo, hi;
  __device__ NearFrame(double k2_) : k2(k2_), lo((float)(-1100.0 / k2_)), hi((float)(1100.0 / k2_)) {}
  // Whether binary32 holds the bounds: below its normal numbers their rounding would move them.
  __device__ bool holds() const { return hi >= 0x1p-126f; }
  __device__ double weight(float z) const { return exp2_of((double)__builtin_amdgcn_fmed3f(z, lo, hi), k2); }
};
__device__ __forceinline__ bool near_sum(double s) { return s >= 0x1p-900 && s <= 0x1p1000; }

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

// A temperature given as a number is binary64; beyond these bounds the weights no longer change, and 1 / T or 1100 T could leave
// binary64.  Logits that differ do so by 2^-149 or more, which at T = 2^-160 is a weight of e^-2048, 0 in binary64; and by
// less than 2^129, which at T = 2^200 is a weight that rounds to 1.
constexpr double kLeastT = 0x1p-160, kMostT = 0x1p200;

// The row pass: 17 instructions of binary64 arithmetic per logit of a row whose weights are all needed take about 16 us
// for 256 x 128256, the loads 11: together 25 us (2.6 TB/s).  A row that only needs its maximum is bound by the
// loads.
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
  const Profile f = profile_of(a, row);
  Record r;
  r.s = 0.0;
  r.m = -__builtin_inff();
  r.far = 0;
  const int32_t j0 = c * (kVpl * kWave);
  u32x4 v[kVpl];
  const bool mass = f.ok && !f.greedy && (!f.cut || (f.top_p && !f.top_k));  // the nucleus is a share of the whole row
  const bool peak = f.ok && (f.greedy || f.cut);
  // A body for each way of loading: behind a common one the first vector would wait for the last.
  auto chunk = [&] {
    float m = -__builtin_inff();
    auto pass = [&](auto with_mass, auto with_peak, const auto& frame) {
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < kVpl; ++i) {
        // hides from the compiler that passes work on the same values: it would keep them all unpacked, and spill
        asm volatile("" : "+v"(v[i]));
        float z[E::kPerVec];
        E::unpack(v[i], z);
#pragma unroll
        for (int e = 0; e < E::kPerVec; ++e) {
          if constexpr (with_mass.value) s += frame.weight(z[e]);
          if constexpr (with_peak.value) m = fmaxf(m, z[e]);
        }
        __builtin_amdgcn_sched_barrier(0);  // vectors one after another: interleaved they spill
      }
      if constexpr (with_mass.value) r.s = wave_sum(s);
    };
    constexpr std::true_type yes{};
    constexpr std::false_type no{};
    const NearFrame near(kLog2e / f.T);
    const bool absolute = mass && near.holds();  // else r.s stays 0, and the maximum's frame is taken
    if (absolute && peak)
      pass(yes, yes, near);
    else if (absolute)
      pass(yes, no, near);
    else if (peak)
      pass(no, yes, near);
    if (mass && !near_sum(r.s)) {
      if (!peak) pass(no, yes, near);
      m = wave_max(m);
      pass(yes, no, Frame(m, kLog2e / f.T));
      r.far = 1;
    }
    r.m = wave_max(m);
  };
  if (view.inside(j0, kVpl * kWave)) {
#pragma unroll
    for (int i = 0; i < kVpl; ++i) {
      v[i] = view.vec((int64_t)j0 + i * kWave + lane);
      __builtin_amdgcn_sched_barrier(0);  // asked for in the order of their use
    }
    chunk();
  } else {
    view.template edge<kVpl>(j0 + lane, kWave, v);
    chunk();
  }
  if (lane == 0) a.rec[unit] = r;
}

template <int kThreads>
struct Shared {
  static constexpr int kWaves = kThreads / kWave;
  static constexpr int kRoom = 4096;  // logits of a bracket
  uint64_t hist[kWindow];
  u32x4 room[kRoom / 4];
  double wave_d[kWaves];
  uint64_t wave_u[kWaves];
  float wave_f[kWaves];
  int32_t wave_i[2][kWaves];
  uint64_t found_before, found_at;
  double mass_before;
  uint32_t found_bin, key, n_room;
  int32_t eq_last, chunk;
};

// Exclusive prefix over the workgroup's threads in thread order; the total in every thread.
template <int kWaves, class T>
__device__ __forceinline__ T block_scan(T v, T* wave_sums, T& total) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const T inc = wave_detail::inclusive_scan(v);
  __syncthreads();
  if (lane == kWave - 1) wave_sums[wave] = inc;
  __syncthreads();
  T base = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const T x = wave_sums[w];
    base += w < wave ? x : T(0);
    total += x;
  }
  return base + (inc - v);
}

// The first (or last) of the threads' ids in thread order, kNone from a thread that has none.
constexpr int32_t kNone = 0x7fffffff;
template <int kWaves>
__device__ __forceinline__ int32_t block_first(int32_t id, int32_t* wave_ids) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const uint64_t who = __ballot(id != kNone);
  __syncthreads();
  if (who ? lane == __ffsll((unsigned long long)who) - 1 : lane == 0) wave_ids[wave] = id;
  __syncthreads();
  int32_t first = kNone;
#pragma unroll
  for (int w = kWaves - 1; w >= 0; --w) first = wave_ids[w] != kNone ? wave_ids[w] : first;
  return first;
}
template <int kWaves>
__device__ __forceinline__ int32_t block_last(int32_t id, int32_t* wave_ids) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  const uint64_t who = __ballot(id != kNone);
  __syncthreads();
  if (who ? lane == 63 - __builtin_clzll(who) : lane == 0) wave_ids[wave] = id;
  __syncthreads();
  int32_t last = kNone;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) last = wave_ids[w] != kNone ? wave_ids[w] : last;
  return last;
}

// A row's vectors for the passes over it.  Each pass is a loop over single vectors, small enough
// to stay in the instruction cache: unrolled over a thread's whole share (32 logits) the passes of a row are
// 160 KiB of code that each workgroup fetches to run once, and that fetch set their time (56 us against 20 us for
// one row of 32000 under top-k).  A row is C chunks of vecs neighbouring vectors, a chunk at most one vector per
// thread; what a vector holds beside the row is -inf.
//
// In memory, a wave's vectors interleaved by lane and kAhead of them loaded ahead ...
constexpr int kAhead = 4;

template <class E, int kThreads, int kVpl>
struct MemorySource {
  static constexpr int P = E::kPerVec, vecs = kVpl * kWave;
  const RowView<E>& view;
  int32_t C;
  __device__ int32_t lead() const { return view.lead; }
  __device__ int32_t values() const { return view.end - view.lead; }
  __device__ __forceinline__ u32x4 one(int32_t j) const { return view.one(j); }
  // f(index of this lane's vector, vector)
  template <class F>
  __device__ __forceinline__ void vectors(int32_t j0, int32_t j1, int32_t step, F f) const {
    const int lane = threadIdx.x & (kWave - 1);
    u32x4 ahead[kAhead];
    auto load = [&](int32_t j, u32x4& v) {
      u32x4 one[1];
      if (j < j1) {
        view.template load<1>(j, lane, one);
        v = one[0];
      }
    };
#pragma unroll
    for (int i = 0; i < kAhead; ++i) load(j0 + i * step, ahead[i]);
#pragma unroll 1
    for (int32_t j = j0; j < j1; j += step) {
      const u32x4 v = ahead[0];
#pragma unroll
      for (int i = 0; i + 1 < kAhead; ++i) ahead[i] = ahead[i + 1];
      load(j + kAhead * step, ahead[kAhead - 1]);
      f(j + lane, v);
    }
  }
  // Every vector once, by the whole workgroup.
  template <class F>
  __device__ __forceinline__ void all(F f) const {
    const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x / kWave));
    vectors(wave * kWave, (view.end + P - 1) / P, kThreads, f);
  }
  // The vectors of a chunk, by one wave (lanes past the row's end get -inf).
  template <class F>
  __device__ __forceinline__ void chunk(int32_t c, F f) const {
    vectors(c * vecs, (c + 1) * vecs, kWave, f);
  }
};

// ... or in shared memory, a chunk per wave.
template <class E, int kThreads>
struct SharedSource {
  static constexpr int P = E::kPerVec;
  static constexpr int32_t C = kThreads / kWave;
  const u32x4* v;
  int32_t n, vecs;  // vectors of the row, of a chunk
  int32_t lead_, V;
  __device__ int32_t lead() const { return lead_; }
  __device__ int32_t values() const { return V; }
  __device__ __forceinline__ u32x4 one(int32_t j) const {
    u32x4 x = RowView<E>::nothing();
    if (j < n) x = v[j];
    return x;
  }
  template <class F>
  __device__ __forceinline__ void all(F f) const {
    // whole waves in every round: f may use the wave's other lanes
#pragma unroll 1
    for (int32_t j = threadIdx.x; j - (int32_t)(threadIdx.x & (kWave - 1)) < n; j += kThreads) f(j, one(j));
  }
  template <class F>
  __device__ __forceinline__ void chunk(int32_t c, F f) const {
    const int lane = threadIdx.x & (kWave - 1);
    const int32_t end = (c + 1) * vecs;
#pragma unroll 1
    for (int32_t j = c * vecs; j < end; j += kWave) {
      u32x4 x = RowView<E>::nothing();
      if (j + lane < end && j + lane < n) x = v[j + lane];
      f(j + lane, x);
    }
  }
};

// Every logit of the row once: f(z).
template <class E, class Source, class F>
__device__ __forceinline__ void each(const Source& source, F f) {
  const int32_t V = source.values(), lead = source.lead();
  source.all([&](int32_t j, u32x4 v) {
    float z[E::kPerVec];
    E::unpack(v, z);
#pragma unroll
    for (int e = 0; e < E::kPerVec; ++e)
      if ((uint32_t)(j * E::kPerVec + e - lead) < (uint32_t)V) f(z[e]);
  });
}

struct Selected {
  uint32_t key;
  uint64_t before, at, need;  // the sums above the key and at it, and the sum that was to be reached
};

// The largest key at which the running sum of value(z), from the largest key down, reaches
// need_of(total): one pass of the row per digit (11 + 5 bits of a bf16 key, 11 + 11 + 10 of a
// binary32 key) fills a histogram of the keys that share the digits found so far.  Sums are
// integers, so the order of the adds changes nothing.
template <class E, int kThreads, class Source, class Value, class Need>
__device__ Selected radix_select(const Source& source, Shared<kThreads>& sh, Value value, Need need_of) {
  constexpr int kLevels = E::kBytes == 2 ? 2 : 3, kBins = 2048, kPer = kBins / kThreads;
  const int t = threadIdx.x;
  Selected r;
  r.key = 0;
  r.before = r.need = r.at = 0;
#pragma unroll 1
  for (int level = 0; level < kLevels; ++level) {
    const int shift = level == 0 ? 21 : (E::kBytes == 2 ? 16 : (level == 1 ? 10 : 0));
    const int width = level == 0 ? 11 : (E::kBytes == 2 ? 5 : (level == 1 ? 11 : 10));
    const int bins = 1 << width;
    __syncthreads();
    for (int b = t; b < kBins; b += kThreads) sh.hist[b] = 0;
    __syncthreads();
    each<E>(source, [&](float z) {
      const uint32_t key = order_key(z);
      if (level > 0 && ((key ^ r.key) >> (shift + width)) != 0) return;
      const uint64_t x = value(z);
      if (x)
        atomicAdd(reinterpret_cast<unsigned long long*>(&sh.hist[(key >> shift) & (bins - 1)]), (unsigned long long)x);
    });
    __syncthreads();
    // kPer bins per thread, from the top bin down
    uint64_t own = 0;
    for (int b = 0; b < kPer; ++b) {
      const int bin = bins - 1 - (kPer * t + b);
      own += bin >= 0 ? sh.hist[bin] : 0;
    }
    uint64_t total;
    uint64_t pre = block_scan<kThreads / kWave>(own, sh.wave_u, total);
    if (level == 0) {
      r.need = need_of(total);
      if (r.need > total) r.need = total;
    }
    const uint64_t want = r.need - r.before;
    for (int b = 0; b < kPer; ++b) {
      const int bin = bins - 1 - (kPer * t + b);
      const uint64_t x = bin >= 0 ? sh.hist[bin] : 0;
      if (pre < want && pre + x >= want) {
        sh.found_bin = bin;
        sh.found_before = r.before + pre;
        sh.found_at = x;
      }
      pre += x;
    }
    __syncthreads();
    r.key |= sh.found_bin << shift;
    r.before = sh.found_before;
    r.at = sh.found_at;
  }
  if (E::kBytes == 2) r.key |= 0xffffu;
  return r;
}

// A mass within 2^-44 of its share reaches it: the sums carry roundings of about 2^-50, and copies of one logit
// that make the share exactly (500 of 1000) have to.
constexpr double kReach = 1.0 - 0x1p-44;

struct Cut {
  uint32_t key;  // kept: keys above it, and its first `copies` copies
  uint64_t copies;
};

// Top-k and top-p of a bf16 row from one pass: the counts of the 4096 keys at and below the maximum's
// (32 binades of positive logits) give ranks by prefix sums, and masses as count x weight, so no
// other logit's weight is computed.  False if a cut lies below the window.  S: the whole row's mass
// in the frame (used without top-k).
template <class E, int kThreads, class Source>
__device__ __forceinline__ bool window_cut(const Source& source, Shared<kThreads>& sh, const Profile& f, const Frame& frame,
                           uint32_t top, double S, Cut& cut) {
  constexpr int kPer = kWindow / kThreads, kWaves = kThreads / kWave;
  const int t = threadIdx.x;
  uint32_t* const count = reinterpret_cast<uint32_t*>(sh.hist);
  __syncthreads();
  for (int b = t; b < kWindow; b += kThreads) count[b] = 0;
  if (t == 0) sh.found_bin = kWindow;
  __syncthreads();
  const uint32_t top16 = top >> 16;
  if (top16 >= 0x8000u + kWindow) {
    // a maximum above the window's width over 0: the window holds positive logits alone, whose bits are their
    // order; zeros, negative ones, NaN and what lies beside the row wrap to a large distance
    const uint32_t max16 = top16 & 0x7fffu;
    source.all([&](int32_t, u32x4 v) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t lo = max16 - (v[w] & 0xffffu), hi = max16 - (v[w] >> 16);
        if (lo < kWindow) atomicAdd(&count[lo], 1u);
        if (hi < kWindow) atomicAdd(&count[hi], 1u);
      }
    });
  } else {
    each<E>(source, [&](float z) {
      const uint32_t d = top16 - (order_key(z) >> 16);
      if (d < kWindow) atomicAdd(&count[d], 1u);
    });
  }
  __syncthreads();
  uint64_t c[kPer], own = 0;
#pragma unroll
  for (int b = 0; b < kPer; ++b) {
    c[b] = count[kPer * t + b];
    own += c[b];
  }
  auto key_of = [&](uint32_t bin) { return ((top16 - bin) << 16) | 0xffffu; };
  if (f.top_k) {
    const uint64_t k = (uint64_t)f.k;
    uint64_t total;
    uint64_t pre = block_scan<kWaves>(own, sh.wave_u, total);
    if (total < k) return false;
#pragma unroll
    for (int b = 0; b < kPer; ++b) {
      if (pre < k && pre + c[b] >= k) {
        sh.found_bin = kPer * t + b;
        sh.found_before = k - pre;
      }
      pre += c[b];
      if (pre > k) c[b] = pre - c[b] >= k ? 0 : c[b] - (pre - k);  // ranks behind k
    }
    __syncthreads();
    cut.key = key_of(sh.found_bin);
    cut.copies = sh.found_before;
  }
  if (f.top_p) {
    double w[kPer], x = 0.0;
#pragma unroll
    for (int b = 0; b < kPer; ++b) {
      const uint32_t bin = kPer * t + b;
      w[b] = bin <= top16 ? frame.weight(row_key_logit<E>(key_of(bin))) : 0.0;
      x += (double)c[b] * w[b];
    }
    double total;
    double pre = block_scan<kWaves>(x, sh.wave_d, total);
    if (f.top_k) S = total;
    const double want = (double)f.p * S * kReach;  // thousandths of S
    int32_t bin = kNone;
#pragma unroll
    for (int b = kPer - 1; b >= 0; --b) {
      double before = pre;
#pragma unroll
      for (int q = 0; q < b; ++q) before += (double)c[q] * w[q];
      if (c[b] > 0 && (before + (double)c[b] * w[b]) * 1000.0 >= want) bin = kPer * t + b;
    }
    const int32_t first = block_first<kWaves>(bin, sh.wave_i[0]);
    if (first == kNone) {
      if (!f.top_k) return false;
      return true;  // the sums' rounding: every rank of the top-k set is needed
    }
    if (bin == first) {
      const int b = bin - kPer * t;
      double before = pre, one = 0.0;
      uint64_t n = 0;
#pragma unroll
      for (int q = 0; q < kPer; ++q) {
        if (q < b) before += (double)c[q] * w[q];
        if (q == b) {
          one = w[q];
          n = c[q];
        }
      }
      double need = ceil((want / 1000.0 - before) / one);
      need = need < 1.0 ? 1.0 : (need > (double)n ? (double)n : need);
      while (need > 1.0 && (before + (need - 1.0) * one) * 1000.0 >= want) need -= 1.0;
      while (need < (double)n && (before + need * one) * 1000.0 < want) need += 1.0;
      sh.found_before = (uint64_t)need;
    }
    __syncthreads();
    cut.key = key_of(first);
    cut.copies = sh.found_before;
  }
  return true;
}

// Top-k and top-p by radix selection over a source's logits.  Of a top-p without top-k, `above` is the mass of
// the logits that rank before all of the source's, and S the whole row's (S < 0: the source is the row).
template <class E, int kThreads, class Source>
__device__ __forceinline__ void select_cut(const Source& source, Shared<kThreads>& sh, int32_t V, const Profile& f,
                                           const Frame& frame, double above, double S, Cut& cut) {
  uint64_t k_copies_all = 0;
  cut.key = 0;
  cut.copies = ~0ull;
  if (f.top_k) {
    const uint64_t k = (uint64_t)f.k;
    const Selected r = radix_select<E, kThreads>(
        source, sh, [](float) { return (uint64_t)1; }, [k](uint64_t) { return k; });
    cut.key = r.key;
    cut.copies = k - r.before;
    k_copies_all = r.at;
  }
  if (f.top_p) {
    // Masses as integers, with room for V of them in 62 bits.  The copies of the top-k key behind
    // rank k count in the passes and are taken off the total; they rank last, so no prefix that
    // the smaller sum asks for reaches them.
    const int bits = 62 - (32 - __builtin_clz((unsigned)V));
    auto mass = [&](float z) { return (uint64_t)__builtin_rint(__builtin_amdgcn_ldexp(frame.weight(z), bits)); };
    const uint32_t k_key = cut.key;
    const uint64_t p = (uint64_t)f.p;
    const uint64_t over = f.top_k ? (k_copies_all - cut.copies) * mass(row_key_logit<E>(k_key)) : 0;
    const Selected r = radix_select<E, kThreads>(
        source, sh, [&](float z) { return row_key<E>(z) >= k_key ? mass(z) : (uint64_t)0; },
        [&](uint64_t total) {
          const double rest = (double)f.p * S * kReach / 1000.0 - above;
          const uint64_t need = S >= 0.0 ? (rest > 0.0 ? (uint64_t)__builtin_ceil(__builtin_amdgcn_ldexp(rest, bits)) : 0)
                                         : (uint64_t)(((unsigned __int128)(total - over) * p + 999) / 1000);
          return need ? need : (uint64_t)1;
        });
    const uint64_t one = mass(row_key_logit<E>(r.key));
    cut.key = r.key;
    cut.copies = (r.need - r.before + one - 1) / one;
  }
}

// Top-k and top-p of a binary32 row.  The counts of the 4096 leading 16-bit parts of keys below the maximum's
// bracket the cut: for top-k the bins down to rank k; for top-p, a bin's mass lying between its count times its
// smallest and its largest weight, the bins from where the nucleus may end to where it must.  A second pass
// gathers the bracket's logits in shared memory, where the selection is exact, and sums the mass above it.
// False if the cut lies below the window or more logits lie in the bracket than there is room for.
template <class E, int kThreads, class Source>
__device__ __forceinline__ bool bracket_cut(const Source& source, Shared<kThreads>& sh, int32_t V, const Profile& f,
                                            const Frame& frame, uint32_t top, double S, Cut& cut) {
  constexpr int kPer = kWindow / kThreads, kWaves = kThreads / kWave, P = E::kPerVec;
  constexpr int kRoom = Shared<kThreads>::kRoom, kList = (1 + P) * kWave;
  static_assert(kWaves * kList * sizeof(float) <= sizeof(sh.hist), "the lists take the histogram's place");
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const uint32_t top16 = top >> 16;
  if (top16 - (order_key(-__builtin_inff()) >> 16) < kWindow) return false;  // -inf must lie below the window
  uint32_t* const count = reinterpret_cast<uint32_t*>(sh.hist);
  __syncthreads();
  for (int b = t; b < kWindow; b += kThreads) count[b] = 0;
  if (t == 0) {
    sh.found_bin = kWindow;
    sh.n_room = 0;
  }
  __syncthreads();
  if (top16 >= 0x8000u + kWindow) {  // positive logits alone, as in window_cut
    const uint32_t max16 = top16 & 0x7fffu;
    source.all([&](int32_t, u32x4 v) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t d = max16 - (v[w] >> 16);
        if (d < kWindow) atomicAdd(&count[d], 1u);
      }
    });
  } else {
    source.all([&](int32_t, u32x4 v) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const uint32_t d = top16 - (order_key(__uint_as_float(v[w])) >> 16);
        if (d < kWindow) atomicAdd(&count[d], 1u);
      }
    });
  }
  __syncthreads();
  uint64_t c[kPer], own = 0;
#pragma unroll
  for (int b = 0; b < kPer; ++b) {
    c[b] = count[kPer * t + b];
    own += c[b];
  }
  uint64_t total;
  const uint64_t pre = block_scan<kWaves>(own, sh.wave_u, total);
  int32_t lo_bin = kNone, hi_bin = kNone;  // this thread's candidates for the bracket's ends
  if (f.top_k) {
    if (total < (uint64_t)f.k) return false;
    uint64_t run = pre;
#pragma unroll
    for (int b = 0; b < kPer; ++b) {
      run += c[b];
      if (hi_bin == kNone && run >= (uint64_t)f.k) hi_bin = kPer * t + b;
    }
  } else {
    double lo[kPer], hi[kPer], own_lo = 0.0, own_hi = 0.0;
#pragma unroll
    for (int b = 0; b < kPer; ++b) {
      const uint32_t bin = kPer * t + b;
      lo[b] = hi[b] = 0.0;
      if (c[b] > 0) {
        const uint32_t key = (top16 - bin) << 16;
        lo[b] = (double)c[b] * frame.weight(key_logit(key));
        hi[b] = (double)c[b] * fmin(frame.weight(key_logit(key | 0xffffu)), 1.0);
      }
      own_lo += lo[b];
      own_hi += hi[b];
    }
    // both ends a little wide: the sums carry roundings
    const double want = (double)f.p * S / 1000.0;
    double all, run_lo = block_scan<kWaves>(own_lo, sh.wave_d, all);
    double run_hi = block_scan<kWaves>(own_hi, sh.wave_d, all);
#pragma unroll
    for (int b = 0; b < kPer; ++b) {
      run_lo += lo[b];
      run_hi += hi[b];
      if (lo_bin == kNone && c[b] > 0 && run_hi * (1.0 + 1e-9) >= want) lo_bin = kPer * t + b;
      if (hi_bin == kNone && c[b] > 0 && run_lo * (1.0 - 1e-9) >= want) hi_bin = kPer * t + b;
    }
  }
  const int32_t first = f.top_k ? 0 : block_first<kWaves>(lo_bin, sh.wave_i[0]);
  const int32_t last = block_first<kWaves>(hi_bin, sh.wave_i[1]);
  if (first == kNone || last == kNone) return false;
  uint64_t mine = 0, held_total;
#pragma unroll
  for (int b = 0; b < kPer; ++b) mine += kPer * t + b >= first && kPer * t + b <= last ? c[b] : 0;
  (void)block_scan<kWaves>(mine, sh.wave_u, held_total);
  if (held_total > (uint64_t)kRoom) return false;
  __syncthreads();

  float* const list = reinterpret_cast<float*>(sh.hist) + wave * kList;
  float* const room = reinterpret_cast<float*>(sh.room);
  double s = 0.0;
  uint32_t held = 0;
  source.all([&](int32_t, u32x4 v) {
    float z[P];
    E::unpack(v, z);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const uint32_t d = top16 - (order_key(z[e]) >> 16);
      const bool before = d < (uint32_t)first, in = !before && d <= (uint32_t)last;
      const uint64_t over = __ballot(before), put = __ballot(in);
      if (before)
        list[held + __builtin_amdgcn_mbcnt_hi((uint32_t)(over >> 32),
                                              __builtin_amdgcn_mbcnt_lo((uint32_t)over, 0))] = z[e];
      held += __builtin_popcountll(over);
      if (put) {  // the order in the room does not matter: the selection goes by value
        const int leader = __ffsll((unsigned long long)put) - 1;
        uint32_t at = 0;
        if (lane == leader) at = atomicAdd(&sh.n_room, (uint32_t)__builtin_popcountll(put));
        at = lane_value(at, leader);
        at += __builtin_amdgcn_mbcnt_hi((uint32_t)(put >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)put, 0));
        if (in && at < (uint32_t)kRoom) room[at] = z[e];
      }
    }
    while (held >= kWave) {
      held -= kWave;
      s += frame.weight(list[held + lane]);
    }
  });
  if (lane < held) s += frame.weight(list[lane]);
  double above;
  (void)block_scan<kWaves>(s, sh.wave_d, above);
  const SharedSource<E, kThreads> chosen{sh.room, (int32_t)((held_total + P - 1) / P), 0, 0, (int32_t)held_total};
  select_cut<E, kThreads>(chosen, sh, V, f, frame, above, f.top_k ? -1.0 : S, cut);
  return true;
}

// The key of the smallest logit of weight min_p or more: the first of the row's type from m + T ln(min_p) on, which is no
// further than m.  The border itself, and not a search for it among weights: next to a border near zero lie more
// logits than the weights' rounding tells apart.
template <class E>
__device__ __forceinline__ uint32_t min_p_key(float m, const Profile& f) {
  const double border = fmax((double)m + f.T * log((double)f.min_p), -(double)__FLT_MAX__);  // every finite logit
  const float z = (float)border;
  uint32_t u = __float_as_uint(z);
  if ((double)z < border) u = z == 0.0f ? 1u : ((u >> 31) ? u - 1 : u + 1);  // the next one up
  if (E::kBytes == 2) u = (u >> 31) ? u & 0xffff0000u : (u + 0xffffu) & 0xffff0000u;
  return row_key<E>(__uint_as_float(u));
}

// The cut of a row's profile.  S: the whole row's mass in the frame (of a row with top-p, without top-k).
template <class E, int kThreads, class Source>
__device__ __forceinline__ Cut cut_of(const Source& source, Shared<kThreads>& sh, const Args& a, const Profile& f,
                                      const Frame& frame, float m, double S) {
  Cut cut;
  cut.key = 0;
  cut.copies = ~0ull;
  if (f.top_k || f.top_p) {
    bool done;
    if constexpr (E::kBytes == 2)
      done = window_cut<E, kThreads>(source, sh, f, frame, row_key<E>(m), S, cut);
    else
      done = bracket_cut<E, kThreads>(source, sh, a.V, f, frame, row_key<E>(m), S, cut);
    if (!done) select_cut<E, kThreads>(source, sh, a.V, f, frame, 0.0, -1.0, cut);
  }
  if (f.min_p > 0.0f) {
    __syncthreads();
    if (threadIdx.x == 0) sh.key = min_p_key<E>(m, f);
    __syncthreads();
    if (sh.key > cut.key) {
      cut.key = sh.key;
      cut.copies = ~0ull;
    }
  }
  return cut;
}

__device__ __forceinline__ RowState empty_state(int64_t slot, int32_t kind) {
  RowState st;
  st.base = st.k2 = 0.0;
  st.inv_s = 0.0f;
  st.exp_s = 0;
  st.key = 0;
  st.last = kNone;
  st.token = -1;
  st.kind = kind;
  st.slot = slot;
  return st;
}

__device__ __forceinline__ void write_token(const Args& a, int64_t slot, int32_t token, float prob, int32_t kept) {
  a.tokens[slot] = token;
  a.prob[slot] = prob;
  if (a.kept) a.kept[slot] = kept;
}

__device__ __forceinline__ RowState state_of(int64_t slot, double base, double k2, double S, const Cut& cut,
                                             int32_t eq_last) {
  RowState st = empty_state(slot, kDistribution);
  st.base = base;
  st.k2 = k2;
  st.exp_s = __builtin_amdgcn_frexp_exp(S);
  st.inv_s = (float)(1.0 / __builtin_amdgcn_frexp_mant(S));
  st.key = cut.key;
  st.last = eq_last;
  return st;
}

// p(v) in binary32: the exponent in binary64, its fraction alone through the binary32 exponential.
template <class E>
__device__ __forceinline__ float prob_of(const RowState& st, double d_min, float z, int32_t v) {
  const uint32_t key = row_key<E>(z);
  if (!(key > st.key || (key == st.key && v <= st.last))) return 0.0f;
  const double d = fmax((double)z - st.base, d_min);
  const double n = __builtin_rint(d * st.k2);
  return __builtin_amdgcn_ldexpf(fast_exp2((float)fma(d, st.k2, -n)) * st.inv_s, (int)n - st.exp_s);
}

template <int P>
__device__ __forceinline__ void write_probs(float* out, const float (&p)[P]) {
#pragma unroll
  for (int q = 0; q < P; q += 4) {
    u32x4 y;
    y.x = __float_as_uint(p[q]);
    y.y = __float_as_uint(p[q + 1]);
    y.z = __float_as_uint(p[q + 2]);
    y.w = __float_as_uint(p[q + 3]);
    __builtin_nontemporal_store(y, reinterpret_cast<u32x4*>(out + q));
  }
}

// Each chunk's kept mass of a cut row, into rec[c].s; the tokens kept, and the id of the cut key's last kept copy
// where some of its copies are not (kNone otherwise).  The logits above the cut are gathered in shared memory
// first, 64 to a weight: computing weights in place would cost every lane the exponential for the few that are kept.
template <class E, int kThreads, class Source>
__device__ __forceinline__ int64_t cut_masses(const Source& source, Shared<kThreads>& sh, const Frame& frame,
                                              const Cut& cut, Record* rec, int32_t& eq_last) {
  constexpr int P = E::kPerVec, kWaves = kThreads / kWave, kPart = 4, kList = (1 + kPart) * kWave;
  static_assert(kWaves * kList * sizeof(float) <= sizeof(sh.hist), "the lists take the histogram's place");
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  float* const list = reinterpret_cast<float*>(sh.hist) + wave * kList;
  const float z_cut = row_key_logit<E>(cut.key);
  const int32_t C = source.C, lead = source.lead(), end = lead + source.values();
  uint32_t above = 0;
  __syncthreads();
  for (int32_t c = wave; c < C; c += kWaves) {
    double s = 0.0;
    uint32_t eq = 0, held = 0;
    source.chunk(c, [&](int32_t, u32x4 v) {
      float z[P];
      E::unpack(v, z);
#pragma unroll
      for (int e0 = 0; e0 < P; e0 += kPart) {
#pragma unroll
        for (int e = e0; e < e0 + kPart; ++e) {
          const bool more = z[e] > z_cut;
          const uint64_t over = __ballot(more);
          if (more)
            list[held + __builtin_amdgcn_mbcnt_hi((uint32_t)(over >> 32),
                                                  __builtin_amdgcn_mbcnt_lo((uint32_t)over, 0))] = z[e];
          held += __builtin_popcountll(over);
          eq += fmaxf(z[e], -__builtin_inff()) == z_cut;  // NaN counts as -inf
        }
        while (held >= kWave) {
          held -= kWave;
          s += frame.weight(list[held + lane]);
          above += kWave;
        }
      }
    });
    if (lane < held) s += frame.weight(list[lane]);
    above += held;
    s = wave_sum(s);
    eq = wave_sum_u32(eq);
    if (z_cut == -__builtin_inff()) {  // what the chunk's loop saw beside the row came as -inf
      const int32_t rounds = (source.vecs + kWave - 1) / kWave;
      const int32_t lo = c * source.vecs * P, hi = lo + source.vecs * P;
      const int32_t own = (end < hi ? end : hi) - (lead > lo ? lead : lo);
      eq -= rounds * kWave * P - (own > 0 ? own : 0);
    }
    if (lane == 0) {
      rec[c].s = s;
      rec[c].far = eq;
    }
  }
  uint64_t n_above;
  (void)block_scan<kWaves>((uint64_t)(lane == 0 ? above : 0), sh.wave_u, n_above);
  __syncthreads();
  // the kept copies, first chunk first
  const double one = frame.weight(z_cut);
  uint64_t seen = 0;
  for (int32_t c0 = 0; c0 < C; c0 += kThreads) {
    const int32_t c = c0 + t;
    const uint64_t eq = c < C ? rec[c].far : 0;
    uint64_t total;
    const uint64_t pre = seen + block_scan<kWaves>(eq, sh.wave_u, total);
    const uint64_t take = pre >= cut.copies ? 0 : (cut.copies - pre < eq ? cut.copies - pre : eq);
    if (c < C) rec[c].s += (double)take * one;
    if (take > 0 && pre + take == cut.copies) {  // the last kept copy is in this chunk
      sh.chunk = c;
      sh.found_before = take;
    }
    seen += total;
  }
  __syncthreads();
  if (cut.copies < seen) {
    const int32_t j = sh.chunk * source.vecs + t;
    const uint64_t want = sh.found_before;
    uint64_t eq = 0;
    float z[P];
    E::unpack(source.one(t < source.vecs ? j : 0), z);
    auto is = [&](int e) {
      const int32_t at = j * P + e;
      return t < source.vecs && at >= lead && at < end && row_key<E>(z[e]) == cut.key;
    };
#pragma unroll
    for (int e = 0; e < P; ++e) eq += is(e);
    uint64_t total;
    uint64_t pre = block_scan<kWaves>(eq, sh.wave_u, total);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      if (is(e) && ++pre == want) sh.eq_last = j * P + e - lead;
    }
    __syncthreads();
    eq_last = sh.eq_last;
  }
  return (int64_t)(n_above + (cut.copies < seen ? cut.copies : seen));
}

// The draw: S, the chunk the uniform lands in (every wave for itself, 64 chunks at a time: no barrier, the same
// result in each), and the token in it.  mass_of(c): a chunk's mass in the frame.  Returns S.
template <class E, int kThreads, bool kCut, class Source, class Mass>
__device__ __forceinline__ double draw(const Args& a, const Source& source, Shared<kThreads>& sh, const Frame& frame,
                                       bool is_cut, const Cut& cut, int32_t eq_last, double u, int64_t slot,
                                       int64_t n_kept, Mass mass_of) {
  constexpr int P = E::kPerVec, kWaves = kThreads / kWave;
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int32_t C = source.C, lead = source.lead(), end = lead + source.values();
  double S = 0.0;
  for (int32_t c0 = 0; c0 < C; c0 += kWave) S += mass_of(c0 + lane);
  S = wave_sum(S);
  const double target = u * S;
  double carry = 0.0, before = 0.0;
  int32_t chunk = -1, last_chunk = 0;
  for (int32_t c0 = 0; c0 < C && chunk < 0; c0 += kWave) {
    const double x = mass_of(c0 + lane);
    const double inc = carry + wave_detail::inclusive_scan(x);
    const uint64_t hit = __ballot(x > 0.0 && inc > target), some = __ballot(x > 0.0);
    if (some) last_chunk = c0 + 63 - __builtin_clzll(some);
    if (hit) {
      const int who = __ffsll((unsigned long long)hit) - 1;
      chunk = c0 + who;
      before = lane_value(inc - x, who);
    }
    carry = lane_value(inc, kWave - 1);
  }
  // u S within rounding of S: the last chunk with a kept weight, and its last kept token
  const bool past = chunk < 0;
  if (past) chunk = last_chunk;
  const int32_t j = chunk * source.vecs + t;
  double w[P], sum = 0.0;
  {
    float z[P];
    E::unpack(source.one(t < source.vecs ? j : 0), z);
#pragma unroll
    for (int e = 0; e < P; ++e) {
      const int32_t at = j * P + e;
      bool keep = t < source.vecs && at >= lead && at < end;
      if (kCut && is_cut) {
        const uint32_t key = row_key<E>(z[e]);
        keep = keep && (key > cut.key || (key == cut.key && at - lead <= eq_last));
      }
      w[e] = keep ? frame.weight(z[e]) : 0.0;
      sum += w[e];
    }
  }
  double total;
  double run = before + block_scan<kWaves>(sum, sh.wave_d, total);
  int32_t first = kNone, last = kNone;
  double first_w = 0.0, last_w = 0.0;
#pragma unroll
  for (int e = 0; e < P; ++e) {
    if (!(w[e] > 0.0)) continue;
    run += w[e];
    last = j * P + e - lead;
    last_w = w[e];
    if (!past && run > target && first == kNone) {
      first = last;
      first_w = w[e];
    }
  }
  const int32_t y = block_first<kWaves>(first, sh.wave_i[0]);
  const int32_t y_last = block_last<kWaves>(last, sh.wave_i[1]);
  if (y != kNone ? first == y : last == y_last && last != kNone)
    write_token(a, slot, y != kNone ? y : y_last, (float)((y != kNone ? first_w : last_w) / S), (int32_t)n_kept);
  return S;
}

// The rest of a row: two passes over it where it is cut (counts, then the kept masses; from the last-level cache, 512 x
// 151936 103 us, of which shared-memory atomics and the gathering of kept logits take most), none where it is not (256 x
// 128256 8.8 us, the latency of the fold, the search of one chunk and its barriers).
template <class E, int kVpl, bool kCut>
__global__ __launch_bounds__(kDrawThreads) void row_draw(Args a) {
  constexpr int kWaves = kDrawThreads / kWave, P = E::kPerVec;
  static_assert(kVpl * kWave <= kDrawThreads, "one vector of a chunk per thread");
  __shared__ Shared<kDrawThreads> sh;
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int64_t row = blockIdx.x;
  const int64_t slot = slot_of(a, row);
  if (slot < 0) {
    if (a.probs && t == 0) a.state[row] = empty_state(slot, kSkipped);
    return;
  }
  const RowView<E> view(a, row);
  const Profile f = profile_of(a, row);
  Record* rec = a.rec + row * a.C;
  const int32_t C = a.C;
  const double u = f.greedy ? 0.0 : a.uniform[row];

  // Every wave folds the chunks for itself, 64 at a time: no barrier, and the same result in each.
  float m = -__builtin_inff();
  bool any_near = false, any_high = false;
  const double k2 = f.ok && !f.greedy ? kLog2e / f.T : 1.0;
  for (int32_t c = lane; c < C; c += kWave) {
    const Record r = rec[c];
    m = fmaxf(m, r.m);
    any_near = any_near || !r.far;
    any_high = any_high || (r.far && (double)r.m * k2 > 900.0);
  }
  m = wave_max(m);
  const bool plain = f.ok && !f.greedy && !(kCut && f.cut);
  const bool near = plain && __any(any_near) && !__any(any_high);
  const bool finite = near || (m > -__builtin_inff() && m < __builtin_inff());
  if (!f.ok || !finite || !(u >= 0.0 && u < 1.0)) {
    if (t == 0) {
      write_token(a, slot, -1, 0.0f, 0);
      if (a.probs) a.state[row] = empty_state(slot, kNothing);
    }
    return;
  }

  const MemorySource<E, kDrawThreads, kVpl> source{view, C};
  if (f.greedy) {  // the first chunk that holds the maximum, then its first element
    int32_t chunk = 0;
    for (int32_t c0 = 0; c0 < C; c0 += kWave) {
      const uint64_t who = __ballot(c0 + lane < C && rec[c0 + lane < C ? c0 + lane : 0].m == m);
      if (who) {
        chunk = c0 + __ffsll((unsigned long long)who) - 1;
        break;
      }
    }
    const int32_t j = chunk * source.vecs + t;
    int32_t id = kNone;
    if (t < source.vecs) {
      float z[P];
      E::unpack(view.one(j), z);
#pragma unroll
      for (int e = P - 1; e >= 0; --e)
        if (z[e] == m) id = j * P + e - view.lead;
    }
    const int32_t y = block_first<kWaves>(id, sh.wave_i[0]);
    if (t == 0) {
      write_token(a, slot, y, 1.0f, 1);
      if (a.probs) {
        RowState st = empty_state(slot, kOneToken);
        st.token = y;
        a.state[row] = st;
      }
    }
    return;
  }

  const double base = near ? 0.0 : (double)m;
  const Frame frame(base, k2);
  // A chunk's mass in the row's frame; 0 only where none of its tokens has a weight there, since the chunk is searched for the
  // token: of absolute weights a sum above 2^-1060 of at most 2^13 holds one above 2^-1074.
  const double near_scale = near ? 1.0 : frame.weight(0.0f);
  auto stats_mass = [&](const Record& r) {
    if (r.far) return r.s > 0.0 ? r.s * frame.weight(r.m) : 0.0;
    const double x = r.s * near_scale;
    return x > 0x1p-1060 ? x : 0.0;
  };
  Cut cut;
  cut.key = 0;
  cut.copies = ~0ull;
  int64_t n_kept = a.V;
  int32_t eq_last = kNone;
  if (kCut && f.cut) {
    double S = 0.0;
    if (f.top_p && !f.top_k) {
      for (int32_t c = lane; c < C; c += kWave) S += stats_mass(rec[c]);
      S = wave_sum(S);
    }
    cut = cut_of<E, kDrawThreads>(source, sh, a, f, frame, m, S);
    n_kept = cut_masses<E, kDrawThreads>(source, sh, frame, cut, rec, eq_last);
  }
  const double S = draw<E, kDrawThreads, kCut>(a, source, sh, frame, f.cut, cut, eq_last, u, slot, n_kept, [&](int32_t c) {
    return c < C ? (kCut && f.cut ? rec[c].s : stats_mass(rec[c])) : 0.0;
  });
  if (a.probs && t == 0) a.state[row] = state_of(slot, base, k2, S, cut, eq_last);
}

// A row of at most kThreads x kVecs vectors, in one launch: it stays in shared memory, read from memory once.  Bound by
// the latency of its passes one after another (64 rows of 32000 under every truncation 31 us, where reading the
// rows and writing the probabilities takes 2.5; one plain row of 1000 4 us).
template <class E, int kThreads, int kVecs, bool kCut>
__global__ __launch_bounds__(kThreads) void row_whole(Args a) {
  constexpr int kWaves = kThreads / kWave, P = E::kPerVec;
  __shared__ Shared<kThreads> sh;
  __shared__ u32x4 row_s[kThreads * kVecs];
  __shared__ Record rec[kWaves];
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int64_t row = blockIdx.x;
  const int64_t slot = slot_of(a, row);
  if (slot < 0) return;
  const RowView<E> view(a, row);
  const int32_t n = (view.end + P - 1) / P;
  const SharedSource<E, kThreads> source{row_s, n, (n + kWaves - 1) / kWaves, view.lead, a.V};
  float m = -__builtin_inff();
  {
    u32x4 v[kVecs];
    if (view.inside(0, kThreads * kVecs)) {
#pragma unroll
      for (int i = 0; i < kVecs; ++i) v[i] = view.vec(t + i * kThreads);
    } else {
      view.template edge<kVecs>(t, kThreads, v);
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      float z[P];
      E::unpack(v[i], z);
#pragma unroll
      for (int e = 0; e < P; ++e) m = fmaxf(m, z[e]);
      row_s[i * kThreads + t] = v[i];
    }
  }
  const Profile f = profile_of(a, row);
  const double u = f.greedy ? 0.0 : a.uniform[row];
  m = wave_max(m);
  if (lane == 0) sh.wave_f[wave] = m;
  if (t == 0) sh.chunk = kNone;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) m = fmaxf(m, sh.wave_f[w]);

  RowState st = empty_state(slot, kNothing);
  if (f.ok && m > -__builtin_inff() && m < __builtin_inff() && u >= 0.0 && u < 1.0) {
    if (f.greedy) {
      int32_t id = kNone;
      source.all([&](int32_t j, u32x4 v) {
        float z[P];
        E::unpack(v, z);
        const int32_t id0 = j * P - view.lead;
#pragma unroll
        for (int e = P - 1; e >= 0; --e) id = z[e] == m && id0 + e < id ? id0 + e : id;
      });
      if (id != kNone) atomicMin(&sh.chunk, id);
      __syncthreads();
      st.kind = kOneToken;
      st.token = sh.chunk;
      if (t == 0) write_token(a, slot, st.token, 1.0f, 1);
    } else {
      const Frame frame(m, kLog2e / f.T);
      Cut cut;
      cut.key = 0;
      cut.copies = ~0ull;
      int32_t eq_last = kNone;
      int64_t n_kept = a.V;
      const bool is_cut = kCut && f.cut;
      if (!is_cut || (f.top_p && !f.top_k)) {  // the whole row's masses, chunk by chunk
        double s = 0.0;
        source.chunk(wave, [&](int32_t, u32x4 v) {
          float z[P];
          E::unpack(v, z);
#pragma unroll
          for (int e = 0; e < P; ++e) s += frame.weight(z[e]);
        });
        s = wave_sum(s);
        if (lane == 0) rec[wave].s = s;
        __syncthreads();
      }
      if (is_cut) {
        double S = 0.0;
        if (f.top_p && !f.top_k) {
#pragma unroll
          for (int w = 0; w < kWaves; ++w) S += rec[w].s;
        }
        cut = cut_of<E, kThreads>(source, sh, a, f, frame, m, S);
        n_kept = cut_masses<E, kThreads>(source, sh, frame, cut, rec, eq_last);
      }
      const double S = draw<E, kThreads, kCut>(a, source, sh, frame, f.cut, cut, eq_last, u, slot, n_kept,
                                               [&](int32_t c) { return c < kWaves ? rec[c < kWaves ? c : 0].s : 0.0; });
      st = state_of(slot, frame.base, frame.k2, S, cut, eq_last);
    }
  } else if (t == 0) {
    write_token(a, slot, -1, 0.0f, 0);
  }
  if (!a.probs) return;
  float* out = a.probs + slot * a.V;
  const double d_min = st.kind == kDistribution ? -1100.0 / st.k2 : 0.0;
  const bool grid = ((reinterpret_cast<uintptr_t>(out) - view.lead * 4) & 15) == 0;
  source.all([&](int32_t j, u32x4 v) {
    float z[P], p[P];
    E::unpack(v, z);
    const int32_t id0 = j * P - view.lead;
#pragma unroll
    for (int e = 0; e < P; ++e)
      p[e] = st.kind == kDistribution ? prob_of<E>(st, d_min, z[e], id0 + e) : (id0 + e == st.token ? 1.0f : 0.0f);
    if (grid && id0 >= 0 && id0 <= a.V - P) {
      write_probs<P>(out + id0, p);
    } else {
#pragma unroll
      for (int e = 0; e < P; ++e)
        if ((uint32_t)(id0 + e) < (uint32_t)a.V) out[id0 + e] = p[e];
    }
  });
}

constexpr int kProbThreads = 256;

// The probability rows: a thread reads one vector of logits and writes its P values; on the 16-byte grid of
// both as whole vectors.  Bound by memory: 512 x 151936 67 to 85 us, 467 MB at 5.5 to 7 TB/s (the logits partly from the
// last-level cache).
template <class E>
__global__ __launch_bounds__(kProbThreads) void row_probs(Args a, int32_t tiles) {
  constexpr int P = E::kPerVec, kTile = kProbThreads * P;
  const int64_t row = blockIdx.x / tiles;
  const RowState st = a.state[row];
  if (st.kind == kSkipped) return;
  const int64_t v0 = (int64_t)(blockIdx.x - row * tiles) * kTile;
  float* out = a.probs + st.slot * a.V;
  const char* in = row_ptr_strided<E>(a, row);
  const double d_min = st.kind == kDistribution ? -1100.0 / st.k2 : 0.0;
  const int t = threadIdx.x;
  const bool grid = ((reinterpret_cast<uintptr_t>(in) | reinterpret_cast<uintptr_t>(out)) & 15) == 0;
  if (grid && v0 + kTile <= a.V) {
    const int32_t v = (int32_t)v0 + t * P;
    float z[P], p[P];
    u32x4 x;
    x.x = x.y = x.z = x.w = 0;
    if (st.kind == kDistribution) x = *reinterpret_cast<const u32x4*>(in + (int64_t)v * E::kBytes);
    E::unpack(x, z);
#pragma unroll
    for (int e = 0; e < P; ++e)
      p[e] = st.kind == kDistribution ? prob_of<E>(st, d_min, z[e], v + e) : (v + e == st.token ? 1.0f : 0.0f);
    write_probs<P>(out + v, p);
    return;
  }
#pragma unroll
  for (int e = 0; e < P; ++e) {
    const int64_t v = v0 + e * kProbThreads + t;
    if (v >= a.V) break;
    out[v] = st.kind == kDistribution ? prob_of<E>(st, d_min, E::at(in, v), (int32_t)v) : (v == st.token ? 1.0f : 0.0f);
  }
}

// Units below which the chunks are a quarter as long, so that a small batch spreads over the card (rows of 128256: 96 of
// them 17.3 us for 20.7 in long chunks; one 15.7 for 16.5).  From there on long chunks fill it, and a row has fewer
// of them to fold.
constexpr int64_t kFullUnits = 1024;
constexpr int32_t kMostChunks = 256;  // of short ones: a wave folds a row's chunks 64 at a time

struct Plan {
  int vpl;           // 16 or 4: chunks; 0: the row in one workgroup
  int threads, vecs; // then its shape
  int32_t C;
  size_t rec_bytes, bytes;
};

inline size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }

// Chunks of a row of V elements that may begin anywhere in its first 16-byte block.
// Rows that fit a workgroup's shared memory stay in one: 64 rows of 4000 under every truncation 19.3 us for 29.4 by
// chunks, of 32000 31.4 for 33.0; one plain row 12.8 for 15.6.  A row of at most 256 vectors takes 256
// threads (256 rows of 2000: 13.0 us for 13.6 with 1024), and one of at most 1024 no room for more, so that two rows share a
// compute unit (1024 plain rows of 8000: 21.0 us for 28.7).
inline Plan plan_of(int64_t n, int32_t V, int32_t dtype) {
  const int64_t per = dtype == SDV_BF16 ? 8 : 4, vecs = ((int64_t)V + 2 * per - 2) / per;
  Plan p = {};
  if (vecs <= 4 * kDrawThreads) {
    p.threads = vecs <= 256 ? 256 : kDrawThreads;
    p.vecs = vecs <= kDrawThreads ? 1 : 4;
    p.C = 1;
    p.bytes = 256;
    return p;
  }
  p.vpl = 16;
  if (n * ((vecs + 16 * kWave - 1) / (16 * kWave)) < kFullUnits && vecs <= 4 * kWave * kMostChunks) p.vpl = 4;
  p.C = (int32_t)((vecs + p.vpl * kWave - 1) / (p.vpl * kWave));
  p.rec_bytes = up256((size_t)n * p.C * sizeof(Record));
  p.bytes = p.rec_bytes + up256((size_t)n * sizeof(RowState));
  return p;
}

template <class E>
constexpr int64_t prob_tiles(int32_t V) {
  return ((int64_t)V + kProbThreads * E::kPerVec - 1) / (kProbThreads * E::kPerVec);
}

template <class E, int kVpl, bool kCut>
int launch_chunks(const Args& a, hipStream_t stream) {
  const int64_t groups = (a.n * a.C + kStatsWaves - 1) / kStatsWaves;
  hipLaunchKernelGGL((row_stats<E, kVpl>), dim3((unsigned)groups), dim3(kStatsWaves * kWave), 0, stream, a);
  hipLaunchKernelGGL((row_draw<E, kVpl, kCut>), dim3((unsigned)a.n), dim3(kDrawThreads), 0, stream, a);
  if (a.probs) {
    const int32_t tiles = (int32_t)prob_tiles<E>(a.V);
    hipLaunchKernelGGL((row_probs<E>), dim3((unsigned)(a.n * tiles)), dim3(kProbThreads), 0, stream, a, tiles);
  }
  return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
}

// kCut: the call carries a truncation.  Calls without take kernels that hold no code for one.
template <class E, bool kCut>
int launch(const Args& a, const Plan& p, hipStream_t stream) {
  if (p.vpl == 16) return launch_chunks<E, 16, kCut>(a, stream);
  if (p.vpl == 4) return launch_chunks<E, 4, kCut>(a, stream);
  const dim3 grid((unsigned)a.n), block((unsigned)p.threads);
  if (p.threads == 256)
    hipLaunchKernelGGL((row_whole<E, 256, 1, kCut>), grid, block, 0, stream, a);
  else if (p.vecs == 1)
    hipLaunchKernelGGL((row_whole<E, kDrawThreads, 1, kCut>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((row_whole<E, kDrawThreads, 4, kCut>), grid, block, 0, stream, a);
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
      n_rows * p.C > (int64_t)INT32_MAX || (o.probs && n_rows * prob_tiles<F32>(V) > INT32_MAX))
    return SDV_ERR_LIMIT;
  if (p.vpl > 0 ? too_many(n_rows, kDrawThreads) ||
                      too_many((n_rows * p.C + kStatsWaves - 1) / kStatsWaves, kStatsWaves * kWave) ||
                      (o.probs && too_many(n_rows * (dtype == SDV_BF16 ? prob_tiles<Bf16>(V) : prob_tiles<F32>(V)), kProbThreads))
                : too_many(n_rows, p.threads))
    return SDV_ERR_LIMIT;
  if (!workspace || reinterpret_cast<uintptr_t>(workspace) % 16 || workspace_bytes < p.bytes) return SDV_ERR_WORKSPACE;
  Args a = {};
  a.logits = logits;
  a.n = n_rows;
  a.stride = row_stride;
  a.V = V;
  a.C = p.C;
  a.T = temperature > 0.0 ? fmin(fmax(temperature, kLeastT), kMostT) : 0.0;
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
  if (a.top_k || a.top_p || a.min_p)
    return dtype == SDV_BF16 ? launch<Bf16, true>(a, p, s) : launch<F32, true>(a, p, s);
  return dtype == SDV_BF16 ? launch<Bf16, false>(a, p, s) : launch<F32, false>(a, p, s);
}
