// A round's pages from the requests' lengths: sdv_kv_pages.  Pages that no row sees any more go back to a ring of free
// ones, and the coming rows' slots get pages from it, in the order of the requests.
//
// What request i returns and takes follows from its own length and its row of the table alone; where its pages lie in the ring
// are sums over the requests before it.  So its row is read to count, and again where something changes to place it, with the sums
// between: a workgroup per request and a launch each, where every workgroup adds up the counts before its own (of many requests a
// launch between the two does).  Nothing is atomic, and the ring's order is that of the requests.  Bound by two chains of length,
// entries and counts: 512 rows of 4100 entries (8.5 MB, 1.8 us at a copy's rate) take 6.0 + 5.0 us (5.3 + 8.0 with the whole row
// read again), one request's 66 entries 2.3 in one launch.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cache_view.hpp"

namespace pages_impl {

using namespace sdv;

constexpr int kWaves = 4, kThreads = kWaves * kWave;

struct PagesArgs {
  int32_t* table;
  const int32_t* len;
  const int32_t* cu;
  int32_t* ring;
  int32_t* state;
  int32_t* placed;
  int64_t* slots;
  int32_t* freed;    // [B][kWaves] entries that a wave's part of a request's row of the table returns
  int32_t* wanted;   // [B][kWaves] and takes; none if its rows are beyond the table
  uint64_t* events;  // [B][kWaves] where
  int32_t* before;   // [2] the ring's state before the call
  uint64_t* sums;    // [B][2] pages returned and taken before each request: of many requests only
  int64_t n_d, n_pages;
  int32_t B, max_pages, page_log2, window, sinks;
};

// What a request keeps of its row of the table: entries [0, near) and [lo, hi); those of its rows are [rows, hi).
struct Keeps {
  bool known, open;  // not passed over; not ended
  int32_t near, lo, rows, hi;
  __device__ __forceinline__ bool fits(const PagesArgs& a) const { return open && hi <= a.max_pages; }
};
__device__ __forceinline__ Keeps keeps_of(const PagesArgs& a, const Request& r, int32_t len) {
  Keeps k;
  k.known = r.index >= 0 && (len == -1 || len_fits(len, r.k));
  k.open = k.known && len >= 0;
  k.near = k.lo = k.rows = k.hi = 0;
  if (!k.open) return k;
  const int32_t end = len + r.k + 1, page = 1 << a.page_log2;
  k.hi = (int32_t)(((int64_t)end + page - 1) >> a.page_log2);
  k.rows = len >> a.page_log2;
  if (a.window) {
    const int32_t low = len - a.window + 1 > 0 ? len - a.window + 1 : 0, sinks = a.sinks < end ? a.sinks : end;
    k.lo = low >> a.page_log2;
    k.near = (int32_t)(((int64_t)sinks + page - 1) >> a.page_log2);
  }
  return k;
}

// A ring's state within its bounds.
__device__ __forceinline__ bool ring_fits(const PagesArgs& a, int32_t first, int32_t count) {
  return first >= 0 && first < a.n_pages && count >= 0 && count <= a.n_pages;
}

__device__ __forceinline__ void ask(const PagesArgs& a, const Keeps& k, int32_t at, int32_t entry, bool& free, bool& want) {
  const bool have = entry >= 0 && entry < a.n_pages, in = at < a.max_pages;
  const bool keep = at < k.near || (at >= k.lo && at < k.hi);
  free = in && have && !keep;
  want = in && !have && at >= k.rows && at < k.hi;
}

// A part of a row of the table, looked at 64 entries at a time: its chunks, and in 64 bits those where something changes (a bit
// stands for 1 << shift chunks).
struct Part {
  int32_t lo, hi, n, shift;
  __device__ __forceinline__ Part(int32_t from, int32_t to) : lo(from), hi(to), n((to - from + kWave - 1) / kWave), shift(0) {
    while ((n - 1) >> shift > 63) ++shift;  // of the last chunk, too
  }
  // the first chunk from c on that one of `events` stands for, or n
  __device__ __forceinline__ int32_t next(uint64_t events, int32_t c) const {
    if (c >= n) return n;
    const int32_t bit = c >> shift;
    const uint64_t rest = bit < 64 ? events >> bit : 0;
    if (!rest) return n;
    const int32_t skip = __builtin_ctzll(rest);
    return skip ? (bit + skip) << shift : c;
  }
  __device__ __forceinline__ int32_t at(int32_t c) const { return lo + c * kWave + (int32_t)(threadIdx.x & (kWave - 1)); }
  __device__ __forceinline__ int32_t entry(const int32_t* row, int32_t c) const { return at(c) < hi ? row[at(c)] : -1; }
};

// The part of a request's row of the table that wave w takes.
__device__ __forceinline__ Part part_of(int32_t max_pages, int w) {
  const int32_t part = ((max_pages + kWaves * kWave - 1) / (kWaves * kWave)) * kWave;
  const int32_t lo = w * part < max_pages ? w * part : max_pages;
  return Part(lo, lo + part < max_pages ? lo + part : max_pages);
}

// Entries of a part that go back, and that the request's rows need, and where.  kAhead loads at once (two calls, where the whole row
// was read again to place it: 512 requests of 4100 entries 26.7 us, by twos 28.4, by eights 26.3, but one of 66 6.8, 6.7 and 7.3).
constexpr int kAhead = 4;
struct Counts {
  int32_t frees, wants;
  uint64_t events;
};
__device__ __forceinline__ Counts count_part(const PagesArgs& a, const Keeps& k, const int32_t* row, const Part& part) {
  Counts sum = {0, 0, 0};
  for (int32_t c0 = 0; c0 < part.n; c0 += kAhead) {
    int32_t entry[kAhead];
#pragma unroll
    for (int y = 0; y < kAhead; ++y) entry[y] = part.entry(row, c0 + y);
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      if (c0 + y >= part.n) break;
      const int32_t at = part.at(c0 + y);
      bool free, want;
      ask(a, k, at, entry[y], free, want);
      const uint64_t frees = __ballot(free && at < part.hi), wants = __ballot(want && at < part.hi);
      sum.frees += __popcll(frees);
      sum.wants += __popcll(wants);
      if (frees | wants) sum.events |= (uint64_t)1 << ((c0 + y) >> part.shift);
    }
  }
  return sum;
}

// Returns and takes them: `returned` and `taken` pages went before, in the ring as it was.  Only chunks with events are looked at
// again, each asked for before the one in front of it is done.
__device__ __forceinline__ void place_part(const PagesArgs& a, const Keeps& k, int32_t* row, const Part& part, uint64_t events,
                                           int32_t first, int32_t held, uint64_t returned, uint64_t taken, bool is_placed) {
  const int lane = threadIdx.x & (kWave - 1);
  const uint64_t below = ((uint64_t)1 << lane) - 1;
  // a place of the ring, whose sum with `first` is below 2^33
  auto place_of = [&](uint64_t x) { return x < (uint64_t)a.n_pages ? x : x - (uint64_t)a.n_pages; };
  int32_t c = part.next(events, 0), entry = c < part.n ? part.entry(row, c) : -1;
  while (c < part.n) {
    const int32_t c_1 = part.next(events, c + 1), entry_1 = c_1 < part.n ? part.entry(row, c_1) : -1;
    const int32_t at = part.at(c);
    bool free, want;
    ask(a, k, at, entry, free, want);
    free = free && at < part.hi;
    want = want && at < part.hi && is_placed;
    const uint64_t frees = __ballot(free), wants = __ballot(want);
    if (free) {
      const uint64_t to = (uint64_t)held + returned + __popcll(frees & below);
      if (to < (uint64_t)a.n_pages) a.ring[place_of(first + to)] = entry;
      row[at] = -1;
    }
    if (want) row[at] = a.ring[place_of(first + taken + __popcll(wants & below))];
    returned += __popcll(frees);
    taken += __popcll(wants);
    c = c_1;
    entry = entry_1;
  }
}

// The slots of a placed request's rows, by `threads` threads.
__device__ __forceinline__ void write_slots(const PagesArgs& a, const Request& r, const int32_t* row, int32_t len, int t,
                                            int threads) {
  for (int32_t j = t; j <= r.k; j += threads) {
    const int32_t s = len + j, page = row[s >> a.page_log2];
    a.slots[r.row0 + j] = page >= 0 && page < a.n_pages
                              ? ((int64_t)page << a.page_log2) + (s & ((1 << a.page_log2) - 1))
                              : -1;
  }
}

// The ring behind a call that returns `all` pages and takes `most`; what a full ring has no room for is dropped.
__device__ __forceinline__ void write_state(const PagesArgs& a, int32_t first, int32_t held, uint64_t all, uint64_t most) {
  const uint64_t room = (uint64_t)a.n_pages - held, back = all < room ? all : room, to = first + most;
  a.state[0] = (int32_t)(to < (uint64_t)a.n_pages ? to : to - (uint64_t)a.n_pages);
  a.state[1] = (int32_t)((uint64_t)held + back - most);
}

// Few requests with short rows of the table: one workgroup, a wave per request.  Two calls after one another in a replayed graph, by
// this and by the two launches: one request of 515 entries 8.5 us and 13.4, of 890 9.9 and 13.7, of 1540 13.2 and 14.2, of 2050 15.3
// and 15.0; 4 of 890 10.8 and 15.8, of 2050 16.2 and 17.3, of 3000 20.0 and 18.2; 16 of 515 13.2 and 15.7, of 890 15.7 and 15.7, of 1030
// 17.0 and 16.8.  One bound of the width for all: fewer than 16 requests would be faster by this up to about 1540 entries.  (A
// user's two calls from Python take 10 to 11 us at least.)
constexpr int kFewWaves = 16, kFewPages = 896;
__global__ __launch_bounds__(kFewWaves* kWave) void place_few(PagesArgs a) {
  __shared__ int32_t freed_s[kWave], wanted_s[kWave];
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int32_t first = a.state[0], held = a.state[1];
  const bool ring = ring_fits(a, first, held);
  if (a.slots)
    for (int64_t x = t; x < a.n_d + a.B; x += kFewWaves * kWave) a.slots[x] = -1;
  const int32_t i = wave;
  Request r = {};
  int32_t len = -1;
  Keeps k = {};
  Counts counts = {0, 0, 0};
  const Part part(0, a.max_pages);
  if (i < a.B) {
    r = request_at(a.cu, i, a.n_d);
    len = a.len[i];
    k = keeps_of(a, r, len);
    if (k.known && ring) counts = count_part(a, k, a.table + (int64_t)i * a.max_pages, part);
    if (!k.fits(a)) counts.wants = 0;
  }
  if (lane == 0) {
    freed_s[wave] = counts.frees;
    wanted_s[wave] = counts.wants;
  }
  if (t >= kFewWaves && t < kWave) freed_s[t] = wanted_s[t] = 0;
  __syncthreads();
  const uint64_t frees = freed_s[lane], wants = wanted_s[lane];
  const uint64_t returned = wave_inclusive_scan(frees), taken = wave_inclusive_scan(wants);
  if (wave == 0 && ring) {
    const uint64_t served = __ballot(taken <= (uint64_t)held);  // the sums ascend: a run of leading lanes
    const uint64_t most = served ? lane_value(taken, 63 - __builtin_clzll(served)) : 0;
    const uint64_t all = lane_value(returned, kWave - 1);
    if (lane == 0) write_state(a, first, held, all, most);
  }
  if (i >= a.B) return;
  const bool is_placed = ring && k.fits(a) && (counts.wants == 0 || lane_value(taken, i) <= (uint64_t)held);
  if (lane == 0) a.placed[i] = !ring || !k.known ? -1 : (is_placed ? 1 : 0);
  if (!ring || !k.known) return;
  int32_t* const row = a.table + (int64_t)i * a.max_pages;
  place_part(a, k, row, part, counts.events, first, held, lane_value(returned, i) - counts.frees,
             lane_value(taken, i) - counts.wants, is_placed);
  if (!is_placed || !a.slots) return;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");  // the wave's entries
  write_slots(a, r, row, len, lane, kWave);
}

// What each request returns and takes; slots are -1 until they are known.
__global__ __launch_bounds__(kThreads) void count(PagesArgs a) {
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int32_t i = blockIdx.x;
  if (a.slots)
    for (int64_t x = (int64_t)i * kThreads + t; x < a.n_d + a.B; x += (int64_t)a.B * kThreads) a.slots[x] = -1;
  const int32_t first = a.state[0], held = a.state[1];
  if (i == 0 && t == 0) {
    a.before[0] = first;
    a.before[1] = held;
  }
  const Keeps k = keeps_of(a, request_at(a.cu, i, a.n_d), a.len[i]);
  const bool works = k.known && ring_fits(a, first, held);
  Counts counts = {0, 0, 0};
  if (works) counts = count_part(a, k, a.table + (int64_t)i * a.max_pages, part_of(a.max_pages, wave));
  if (lane == 0) {
    a.freed[(int64_t)i * kWaves + wave] = counts.frees;
    a.wanted[(int64_t)i * kWaves + wave] = k.fits(a) ? counts.wants : 0;
    a.events[(int64_t)i * kWaves + wave] = counts.events;
  }
}

// The workgroup's sums of two values, in every thread.
__device__ __forceinline__ void group_sums(uint64_t& x, uint64_t& y, uint64_t (*of_wave)[2]) {
  const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
  x = wave_inclusive_scan(x);
  y = wave_inclusive_scan(y);
  __syncthreads();
  if (lane == kWave - 1) {
    of_wave[wave][0] = x;
    of_wave[wave][1] = y;
  }
  __syncthreads();
  x = y = 0;
  for (int w = 0; w < kWaves; ++w) {
    x += of_wave[w][0];
    y += of_wave[w][1];
  }
}

// A request's counts, of its row's parts.
__device__ __forceinline__ uint64_t sum_of(const int32_t* of_waves, int32_t x) {
  static_assert(kWaves == 4, "one load");
  const int4 n = reinterpret_cast<const int4*>(of_waves)[x];
  return (uint64_t)(uint32_t)n.x + (uint32_t)n.y + (uint32_t)n.z + (uint32_t)n.w;
}

// Many requests: the sums before each, and the ring's state behind the call, by one workgroup, since adding them up in every
// workgroup of `place` reads the square of the requests.
constexpr int kSumWaves = 16, kSumThreads = kSumWaves * kWave;
__global__ __launch_bounds__(kSumThreads) void sum_up(PagesArgs a) {
  __shared__ uint64_t of_wave[2][kSumWaves][2];
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int32_t first = a.before[0], held = a.before[1];
  uint64_t returned = 0, taken = 0, most = 0;  // before the requests at hand; the largest sum that the ring held
  uint64_t back = t < a.B ? sum_of(a.freed, t) : 0, want = t < a.B ? sum_of(a.wanted, t) : 0;
  for (int32_t x0 = 0, turn = 0; x0 < a.B; x0 += kSumThreads, turn ^= 1) {
    const int32_t x = x0 + t, x_1 = x + kSumThreads;
    const uint64_t back_1 = x_1 < a.B ? sum_of(a.freed, x_1) : 0, want_1 = x_1 < a.B ? sum_of(a.wanted, x_1) : 0;
    const uint64_t back_to = wave_inclusive_scan(back), want_to = wave_inclusive_scan(want);
    if (lane == kWave - 1) {
      of_wave[turn][wave][0] = back_to;
      of_wave[turn][wave][1] = want_to;
    }
    __syncthreads();  // (the next requests go to the other half)
    uint64_t back_before = returned, want_before = taken;
#pragma unroll
    for (int w = 0; w < kSumWaves; ++w) {
      const uint64_t b = of_wave[turn][w][0], n = of_wave[turn][w][1];
      back_before += w < wave ? b : 0;
      want_before += w < wave ? n : 0;
      returned += b;
      taken += n;
    }
    if (x < a.B) {
      a.sums[2 * (int64_t)x] = back_before + back_to - back;
      a.sums[2 * (int64_t)x + 1] = want_before + want_to - want;
    }
    const uint64_t here = want_before + want_to;
    if (here <= (uint64_t)(uint32_t)held && here > most) most = here;
    back = back_1;
    want = want_1;
  }
#pragma unroll
  for (int step = 1; step < kWave; step *= 2) {
    const uint64_t o = __shfl_xor((unsigned long long)most, step);
    most = o > most ? o : most;
  }
  __syncthreads();
  if (lane == 0) of_wave[0][wave][0] = most;
  __syncthreads();
  if (t != 0 || !ring_fits(a, first, held)) return;
  for (int w = 1; w < kSumWaves; ++w) most = of_wave[0][w][0] > most ? of_wave[0][w][0] : most;
  write_state(a, first, held, returned, most);
}

// A workgroup per request returns its pages and takes those that it has a right to.
template <bool kSummed>
__global__ __launch_bounds__(kThreads) void place(PagesArgs a) {
  __shared__ uint64_t sum_s[kWaves][2];
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int32_t i = blockIdx.x;
  const int32_t first = a.before[0], held = a.before[1];
  const Request r = request_at(a.cu, i, a.n_d);
  const int32_t len = a.len[i];
  const Keeps k = keeps_of(a, r, len);
  const bool ring = ring_fits(a, first, held);
  const uint64_t events = a.events[(int64_t)i * kWaves + wave];
  // pages returned and taken before this request
  uint64_t returned = 0, taken = 0;
  if constexpr (kSummed) {
    returned = a.sums[2 * (int64_t)i];
    taken = a.sums[2 * (int64_t)i + 1];
  } else {
    for (int32_t x = t; x < i; x += kThreads) {
      returned += sum_of(a.freed, x);
      taken += sum_of(a.wanted, x);
    }
    group_sums(returned, taken, sum_s);
  }
  const uint64_t wants = sum_of(a.wanted, i);
  const bool is_placed = ring && k.fits(a) && (wants == 0 || taken + wants <= (uint64_t)held);
  if (t == 0) a.placed[i] = !ring || !k.known ? -1 : (is_placed ? 1 : 0);

  if (!kSummed && i == 0 && ring) {  // the ring's state behind the call
    uint64_t all = 0, sum = 0, most = 0;
    for (int32_t x0 = 0; x0 < a.B; x0 += kThreads) {
      const int32_t x = x0 + t;
      const uint64_t mine = x < a.B ? sum_of(a.wanted, x) : 0;
      uint64_t back = x < a.B ? sum_of(a.freed, x) : 0;
      const uint64_t inc = wave_inclusive_scan(mine);
      uint64_t whole = mine;
      group_sums(back, whole, sum_s);
      all += back;
      uint64_t here = sum + inc;
      for (int w = 0; w < wave; ++w) here += sum_s[w][1];
      sum += whole;
      // the largest sum that the ring held
      uint64_t top = here <= (uint64_t)held ? here : 0;
#pragma unroll
      for (int step = 1; step < kWave; step *= 2) {
        const uint64_t o = __shfl_xor((unsigned long long)top, step);
        top = o > top ? o : top;
      }
      __syncthreads();
      if (lane == 0) sum_s[wave][0] = top;
      __syncthreads();
      for (int w = 0; w < kWaves; ++w) most = sum_s[w][0] > most ? sum_s[w][0] : most;
      __syncthreads();
    }
    if (t == 0) write_state(a, first, held, all, most);
  }

  if (!ring || !k.known) return;
  for (int w = 0; w < wave; ++w) {
    returned += (uint32_t)a.freed[(int64_t)i * kWaves + w];
    taken += (uint32_t)a.wanted[(int64_t)i * kWaves + w];
  }
  int32_t* const row = a.table + (int64_t)i * a.max_pages;
  place_part(a, k, row, part_of(a.max_pages, wave), events, first, held, returned, taken, is_placed);
  if (!is_placed || !a.slots) return;
  __syncthreads();
  write_slots(a, r, row, len, t, kThreads);
}

inline size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
constexpr int32_t kMostRequests = 1 << 24;
// The sums before each request by a launch of their own above this many (a replayed call, rows of 64 entries, by place's workgroups
// and by the launch: 512 requests 9.3 and 13.2 us, 8192 56.2 and 60.4, 10240 71.4 and 72.4, 12288 95 and 85, 16384 155 and 111; of
// 8 entries 65536 2164 and 420, 131072 8580 and 832).
constexpr int32_t kManyRequests = 10240;
inline bool is_many(int32_t B) { return B > kManyRequests; }
inline bool is_few(int32_t B, int32_t max_pages) { return B <= kFewWaves && max_pages <= kFewPages; }

}  // namespace pages_impl

extern "C" size_t sdv_kv_pages_workspace_bytes(int32_t B, int32_t max_pages) {
  using namespace pages_impl;
  if (B < 1 || B >= kMostRequests || max_pages < 1 || is_few(B, max_pages)) return 0;
  return 2 * up256((size_t)B * kWaves * 4) + up256((size_t)B * kWaves * 8) + 256 + (is_many(B) ? (size_t)B * 16 : 0);
}

extern "C" int sdv_kv_pages(int32_t* page_table, int32_t B, int32_t max_pages, int32_t page_size,
                            const int32_t* cache_len, int64_t n_draft_rows, const int32_t* ragged_offsets,
                            int64_t n_pages, int32_t* free_pages, int32_t* free_state, int32_t window, int32_t sinks,
                            int32_t* placed, int64_t* slots, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace pages_impl;
  auto aligned = [](const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  if (!page_table || !cache_len || !ragged_offsets || !free_pages || !free_state || !placed || B < 1 || n_draft_rows < 0 ||
      max_pages < 1 || n_pages < 1 || page_size < 1 || page_size > 1024 || (page_size & (page_size - 1)) || window < 0 ||
      sinks < 0 || !aligned(page_table, 4) || !aligned(cache_len, 4) || !aligned(ragged_offsets, 4) ||
      !aligned(free_pages, 4) || !aligned(free_state, 4) || !aligned(placed, 4) || !aligned(slots, 8))
    return SDV_ERR_INVALID_ARG;
  if (B >= kMostRequests || too_many(B, kThreads) || n_draft_rows + B > INT32_MAX - 1024 || n_pages > INT32_MAX ||
      max_pages > INT32_MAX - 1024)
    return SDV_ERR_LIMIT;
  // what is written lies apart from everything else
  struct Span {
    const void* at;
    int64_t bytes;
  };
  const size_t need = sdv_kv_pages_workspace_bytes(B, max_pages);
  const Span span[] = {{page_table, (int64_t)B * max_pages * 4}, {free_pages, n_pages * 4}, {free_state, 8},
                       {placed, (int64_t)B * 4}, {slots, slots ? (n_draft_rows + B) * 8 : 0},
                       {workspace, workspace ? (int64_t)need : 0},
                       {cache_len, (int64_t)B * 4}, {ragged_offsets, ((int64_t)B + 1) * 4}};
  for (int x = 0; x < 6; ++x)
    for (int y = x + 1; y < 8; ++y)
      if (span[x].bytes && span[y].bytes && overlap(span[x].at, span[x].bytes, span[y].at, span[y].bytes))
        return SDV_ERR_INVALID_ARG;
  if (need > 0 && (!workspace || !aligned16(workspace) || workspace_bytes < need)) return SDV_ERR_WORKSPACE;
  PagesArgs a;
  a.table = page_table;
  a.len = cache_len;
  a.cu = ragged_offsets;
  a.ring = free_pages;
  a.state = free_state;
  a.placed = placed;
  a.slots = slots;
  char* const work = static_cast<char*>(workspace);
  const size_t counts = up256((size_t)B * kWaves * 4);
  a.freed = reinterpret_cast<int32_t*>(work);
  a.wanted = reinterpret_cast<int32_t*>(work + counts);
  a.events = reinterpret_cast<uint64_t*>(work + 2 * counts);
  a.before = reinterpret_cast<int32_t*>(work + 2 * counts + up256((size_t)B * kWaves * 8));
  a.sums = reinterpret_cast<uint64_t*>(a.before + 64);
  a.n_d = n_draft_rows;
  a.n_pages = n_pages;
  a.B = B;
  a.max_pages = max_pages;
  a.page_log2 = log2_of(page_size);
  a.window = window;
  a.sinks = sinks;
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (is_few(B, max_pages)) {
    hipLaunchKernelGGL(place_few, dim3(1), dim3(kFewWaves * kWave), 0, s, a);
    return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
  }
  hipLaunchKernelGGL(count, dim3((unsigned)B), dim3(kThreads), 0, s, a);
  if (is_many(B)) {
    hipLaunchKernelGGL(sum_up, dim3(1), dim3(kSumThreads), 0, s, a);
    hipLaunchKernelGGL(place<true>, dim3((unsigned)B), dim3(kThreads), 0, s, a);
  } else {
    hipLaunchKernelGGL(place<false>, dim3((unsigned)B), dim3(kThreads), 0, s, a);
  }
  return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
}
