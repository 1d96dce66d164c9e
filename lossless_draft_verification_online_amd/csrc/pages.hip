// A round's pages from the requests' lengths: sdv_kv_pages.  Pages that no row sees any more go back to a ring of free
// ones, and the coming rows' slots get pages from it, in the order of the requests.
//
// What request i returns and takes follows from its own length and its row of the table alone; where its pages lie in the ring
// are sums over the requests before it.  So its row is read twice, once to count and once to place, with the sums between: a
// workgroup per request and a launch each, where every workgroup adds up the counts before its own.  Nothing is atomic, and
// the ring's order is that of the requests.  Bound by two chains of length, entries and counts: 512 rows of 4100
// entries (8.5 MB, 1.8 us at a copy's rate) take 5.3 + 8.0 us, one request's 66 entries 3.7 in one launch.
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
  int32_t* freed;   // [B][kWaves] entries that a wave's part of a request's row of the table returns
  int32_t* wanted;  // [B] pages that a request takes
  int32_t* before;  // [2] the ring's state before the call
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

// The part of a request's row of the table that wave w takes.
__device__ __forceinline__ void part_of(int32_t max_pages, int w, int32_t& lo, int32_t& hi) {
  const int32_t part = ((max_pages + kWaves * kWave - 1) / (kWaves * kWave)) * kWave;
  lo = w * part < max_pages ? w * part : max_pages;
  hi = lo + part < max_pages ? lo + part : max_pages;
}

__device__ __forceinline__ void ask(const PagesArgs& a, const Keeps& k, int32_t at, int32_t entry, bool& free, bool& want) {
  const bool have = entry >= 0 && entry < a.n_pages, in = at < a.max_pages;
  const bool keep = at < k.near || (at >= k.lo && at < k.hi);
  free = in && have && !keep;
  want = in && !have && at >= k.rows && at < k.hi;
}

// Entries of [lo, hi) of a request's row of the table that go back, and that its rows need.  kAhead loads at once.
constexpr int kAhead = 4;
__device__ __forceinline__ void count_part(const PagesArgs& a, const Keeps& k, const int32_t* row, int32_t lo, int32_t hi,
                                           int32_t& frees, int32_t& wants) {
  const int lane = threadIdx.x & (kWave - 1);
  for (int32_t x0 = lo; x0 < hi; x0 += kAhead * kWave) {
    int32_t entry[kAhead];
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      const int32_t at = x0 + y * kWave + lane;
      entry[y] = at < hi ? row[at] : -1;
    }
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      if (x0 + y * kWave >= hi) break;
      const int32_t at = x0 + y * kWave + lane;
      bool free, want;
      ask(a, k, at, entry[y], free, want);
      frees += __popcll(__ballot(free && at < hi));
      wants += __popcll(__ballot(want && at < hi));
    }
  }
}

// Returns and takes them: `returned` and `taken` pages went before, in the ring as it was.
__device__ __forceinline__ void place_part(const PagesArgs& a, const Keeps& k, int32_t* row, int32_t lo, int32_t hi,
                                           int32_t first, int32_t held, uint64_t returned, uint64_t taken, bool is_placed) {
  const int lane = threadIdx.x & (kWave - 1);
  const uint64_t below = ((uint64_t)1 << lane) - 1;
  // a place of the ring, whose sum with `first` is below 2^33
  auto place_of = [&](uint64_t x) { return x < (uint64_t)a.n_pages ? x : x - (uint64_t)a.n_pages; };
  for (int32_t x0 = lo; x0 < hi; x0 += kAhead * kWave) {
    int32_t entry[kAhead];
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      const int32_t at = x0 + y * kWave + lane;
      entry[y] = at < hi ? row[at] : -1;
    }
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      if (x0 + y * kWave >= hi) break;
      const int32_t at = x0 + y * kWave + lane;
      bool free, want;
      ask(a, k, at, entry[y], free, want);
      free = free && at < hi;
      want = want && at < hi && is_placed;
      const uint64_t frees = __ballot(free), wants = __ballot(want);
      if (free) {
        const uint64_t to = (uint64_t)held + returned + __popcll(frees & below);
        if (to < (uint64_t)a.n_pages) a.ring[place_of(first + to)] = entry[y];
        row[at] = -1;
      }
      if (want) row[at] = a.ring[place_of(first + taken + __popcll(wants & below))];
      returned += __popcll(frees);
      taken += __popcll(wants);
    }
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

// Few requests with short rows of the table: one workgroup, a wave per request.  Two calls after one another, by this and by the two
// launches: one request of 66 entries 7.4 us and 12.6, 4 of 515 10.1 and 14.0, 16 of 260 10.7 and 14.2, but 16 of 1028 20.7 and
// 14.8, one of 4100 26.8 and 17.6, and 64 of 67 (four to a wave) 29 and 14.2.
constexpr int kFewWaves = 16, kFewPages = 640;
__global__ __launch_bounds__(kFewWaves* kWave) void place_few(PagesArgs a) {
  __shared__ int32_t freed_s[kWave], wanted_s[kWave];
  const int t = threadIdx.x, lane = t & (kWave - 1);
  const int wave = __builtin_amdgcn_readfirstlane(t / kWave);
  const int32_t first = a.state[0], held = a.state[1];
  const bool ring = ring_fits(a, first, held);
  if (t < kWave) freed_s[t] = wanted_s[t] = 0;
  if (a.slots)
    for (int64_t x = t; x < a.n_d + a.B; x += kFewWaves * kWave) a.slots[x] = -1;
  __syncthreads();
  for (int32_t i = wave; i < a.B; i += kFewWaves) {
    const Keeps k = keeps_of(a, request_at(a.cu, i, a.n_d), a.len[i]);
    int32_t frees = 0, wants = 0;
    if (k.known && ring) count_part(a, k, a.table + (int64_t)i * a.max_pages, 0, a.max_pages, frees, wants);
    if (lane == 0) {
      freed_s[i] = frees;
      wanted_s[i] = k.fits(a) ? wants : 0;
    }
  }
  __syncthreads();
  const uint64_t frees = freed_s[lane], wants = wanted_s[lane];
  const uint64_t returned = wave_inclusive_scan(frees), taken = wave_inclusive_scan(wants);
  const bool has_room = taken <= (uint64_t)held;
  if (wave == 0 && ring) {
    const uint64_t served = __ballot(has_room);  // the sums ascend: a run of leading lanes
    const uint64_t most = served ? lane_value(taken, 63 - __builtin_clzll(served)) : 0;
    const uint64_t all = lane_value(returned, kWave - 1);
    if (lane == 0) write_state(a, first, held, all, most);
  }
  for (int32_t i = wave; i < a.B; i += kFewWaves) {
    const Request r = request_at(a.cu, i, a.n_d);
    const int32_t len = a.len[i];
    const Keeps k = keeps_of(a, r, len);
    const uint64_t mine = lane_value(wants, i);
    const bool is_placed = ring && k.fits(a) && (mine == 0 || lane_value(taken, i) <= (uint64_t)held);
    if (lane == 0) a.placed[i] = !ring || !k.known ? -1 : (is_placed ? 1 : 0);
    if (!ring || !k.known) continue;
    int32_t* const row = a.table + (int64_t)i * a.max_pages;
    place_part(a, k, row, 0, a.max_pages, first, held, lane_value(returned, i) - lane_value(frees, i),
               lane_value(taken, i) - mine, is_placed);
    if (!is_placed || !a.slots) continue;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");  // the wave's entries
    write_slots(a, r, row, len, lane, kWave);
  }
}

// What each request returns and takes; slots are -1 until they are known.
__global__ __launch_bounds__(kThreads) void count(PagesArgs a) {
  __shared__ int32_t wanted_s[kWaves];
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
  int32_t frees = 0, wants = 0, lo, hi;
  part_of(a.max_pages, wave, lo, hi);
  if (works) count_part(a, k, a.table + (int64_t)i * a.max_pages, lo, hi, frees, wants);
  if (lane == 0) {
    a.freed[(int64_t)i * kWaves + wave] = frees;
    wanted_s[wave] = wants;
  }
  __syncthreads();
  if (t == 0) {
    int32_t n = 0;
    for (int w = 0; w < kWaves; ++w) n += wanted_s[w];
    a.wanted[i] = works && k.fits(a) ? n : 0;
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

// A workgroup per request returns its pages and takes those that it has a right to.
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
  auto freed_of = [&](int32_t x) {
    const int4 n = reinterpret_cast<const int4*>(a.freed)[x];
    return (uint64_t)(uint32_t)n.x + (uint32_t)n.y + (uint32_t)n.z + (uint32_t)n.w;
  };
  // pages returned and taken before this request
  uint64_t returned = 0, taken = 0;
  for (int32_t x = t; x < i; x += kThreads) {
    returned += freed_of(x);
    taken += (uint32_t)a.wanted[x];
  }
  group_sums(returned, taken, sum_s);
  const int32_t wants = a.wanted[i];
  const bool is_placed = ring && k.fits(a) && (wants == 0 || taken + wants <= (uint64_t)held);
  if (t == 0) a.placed[i] = !ring || !k.known ? -1 : (is_placed ? 1 : 0);

  if (i == 0 && ring) {  // the ring's state behind the call
    uint64_t all = 0, sum = 0, most = 0;
    for (int32_t x0 = 0; x0 < a.B; x0 += kThreads) {
      const int32_t x = x0 + t;
      const uint64_t mine = x < a.B ? (uint32_t)a.wanted[x] : 0;
      uint64_t back = x < a.B ? freed_of(x) : 0;
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
  int32_t lo, hi;
  part_of(a.max_pages, wave, lo, hi);
  for (int w = 0; w < wave; ++w) returned += (uint32_t)a.freed[(int64_t)i * kWaves + w];
  int32_t* const row = a.table + (int64_t)i * a.max_pages;
  // what the parts before this wave's take: counted from the table as it was (entries are written behind the barrier)
  if (is_placed) {
    int32_t none = 0, mine = 0;
    count_part(a, k, row, k.rows > lo ? k.rows : lo, k.hi < hi ? k.hi : hi, none, mine);
    __syncthreads();
    if (lane == 0) sum_s[wave][0] = (uint32_t)mine;
    __syncthreads();
    for (int w = 0; w < wave; ++w) taken += sum_s[w][0];
  }
  place_part(a, k, row, lo, hi, first, held, returned, taken, is_placed);
  if (!is_placed || !a.slots) return;
  __syncthreads();
  write_slots(a, r, row, len, t, kThreads);
}

inline size_t up256(size_t n) { return (n + 255) & ~(size_t)255; }
constexpr int32_t kMostRequests = 1 << 24;
inline bool is_few(int32_t B, int32_t max_pages) { return B <= kFewWaves && max_pages <= kFewPages; }

}  // namespace pages_impl

extern "C" size_t sdv_kv_pages_workspace_bytes(int32_t B, int32_t max_pages) {
  using namespace pages_impl;
  if (B < 1 || B >= kMostRequests || max_pages < 1 || is_few(B, max_pages)) return 0;
  return up256((size_t)B * kWaves * 4) + up256((size_t)B * 4) + 256;
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
  a.freed = static_cast<int32_t*>(workspace);
  a.wanted = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + up256((size_t)B * kWaves * 4));
  a.before = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + up256((size_t)B * kWaves * 4) + up256((size_t)B * 4));
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
  hipLaunchKernelGGL(place, dim3((unsigned)B), dim3(kThreads), 0, s, a);
  return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
}
