// The paged cache of a ragged batch: sdv_kv_append writes the batch's keys and values into their
// pages, rotating keys (and queries) by their positions on the way, and sdv_kv_settle moves the
// accepted path of a verified token tree to where the sequence continues.  Both move each byte
// once; the append is bound by memory, the settling by the latency of its dependent loads.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "cache_view.hpp"

namespace cache_impl {

using namespace sdv;

constexpr int kThreads = 256;

struct AppendArgs {
  CacheView cache;
  int32_t B, D, rotary, n_q;
  int64_t n_d, key_stride, value_stride, query_stride;
  const int32_t* cu;
  const int32_t* parents;
  const char* keys;
  const char* values;
  const float* inv_freq;
  const char* queries;
  char* queries_out;
};

template <class E>
__device__ __forceinline__ u32x4 pack(const float (&f)[E::kPerVec]) {
  u32x4 v;
  if constexpr (E::kBytes == 4) {
    v.x = __float_as_uint(f[0]);
    v.y = __float_as_uint(f[1]);
    v.z = __float_as_uint(f[2]);
    v.w = __float_as_uint(f[3]);
  } else {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bf16x2 h;
      h.x = (__bf16)f[2 * i];
      h.y = (__bf16)f[2 * i + 1];
      w[i] = __builtin_bit_cast(uint32_t, h);
    }
    v.x = w[0];
    v.y = w[1];
    v.z = w[2];
    v.w = w[3];
  }
  return v;
}

// One workgroup per row: the row's angles once, then its heads' vectors.  256 requests of K in 0..8 (48 heads of 128, bf16,
// 33 MB in and out) 9.8 us, 3.4 TB/s: the offsets, length, angles and table entry are loaded one after another, and the row's
// own vectors behind them, though those depend on none of it.  Prompts of 10467 rows 22 to 26 us, at the rate of a copy.
template <class E, bool kInterleaved>
__global__ __launch_bounds__(kThreads) void append(AppendArgs a) {
  constexpr int P = E::kPerVec;
  __shared__ float cos_s[128], sin_s[128];
  __shared__ int32_t parent_s[kWave], depth_s[kMaxNodes + 1];
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x;
  const Request r = request_of_row(a.cu, a.B, a.n_d, row);
  const int64_t j = row - r.row0;
  if (r.index < 0 || j > r.k) return;
  const int64_t len = a.cache.len[r.index];
  if (!len_fits((int32_t)len, r.k)) return;
  int64_t depth = j;
  if (a.parents) {
    if (!tree_depths(a.parents, r, parent_s, depth_s)) return;
    depth = depth_s[j];
  }
  const int half = a.rotary / 2;
  if (t < half) {
    // the angle in turns, reduced in binary64: far positions keep their phase
    const double turns = (double)(len + depth) * (double)a.inv_freq[t] * 0.15915494309189535;
    const float part = (float)(turns - rint(turns));
    sincospif(2.0f * part, &sin_s[t], &cos_s[t]);
  }
  __syncthreads();
  const int64_t slot = len + j;
  const int32_t page = a.cache.page(r.index, slot);
  const int64_t line = (int64_t)a.D * E::kBytes;
  const int vecs = a.D / P;  // vectors of a head

  const int n_k = a.cache.n_heads;
  // rotated heads (queries, then keys): a unit is a pair of vectors half a rotation apart, or one
  // vector behind the rotated part; interleaved, a unit is one vector
  const int pairs = kInterleaved ? 0 : half / P;
  const int per_head = vecs - pairs;
  const int n_rot = (a.n_q + n_k) * per_head;
  for (int w = t; w < n_rot; w += kThreads) {
    const int head = w / per_head, k = w - head * per_head;
    const bool is_q = head < a.n_q;
    const int h = is_q ? head : head - a.n_q;
    if (!is_q && page < 0) continue;
    const char* src = is_q ? a.queries + (row * a.query_stride) * E::kBytes + h * line
                           : a.keys + (row * a.key_stride) * E::kBytes + h * line;
    char* dst = is_q ? a.queries_out + (row * a.n_q + h) * line : a.cache.keys + a.cache.row(page, h, slot) * line;
    if (!kInterleaved && k < pairs) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(src + k * 16);
      const u32x4 y = *reinterpret_cast<const u32x4*>(src + (k + pairs) * 16);
      float p[P], q[P], u[P], v[P];
      E::unpack(x, p);
      E::unpack(y, q);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const float c = cos_s[k * P + e], s = sin_s[k * P + e];
        u[e] = p[e] * c - q[e] * s;
        v[e] = q[e] * c + p[e] * s;
      }
      *reinterpret_cast<u32x4*>(dst + k * 16) = pack<E>(u);
      *reinterpret_cast<u32x4*>(dst + (k + pairs) * 16) = pack<E>(v);
    } else {
      const int at = k + pairs;
      u32x4 x = *reinterpret_cast<const u32x4*>(src + at * 16);
      if (kInterleaved && at * P < a.rotary) {
        float p[P], u[P];
        E::unpack(x, p);
#pragma unroll
        for (int e = 0; e < P; e += 2) {
          const float c = cos_s[(at * P + e) / 2], s = sin_s[(at * P + e) / 2];
          u[e] = p[e] * c - p[e + 1] * s;
          u[e + 1] = p[e + 1] * c + p[e] * s;
        }
        x = pack<E>(u);
      }
      *reinterpret_cast<u32x4*>(dst + at * 16) = x;
    }
  }
  if (page < 0) return;
  for (int w = t; w < n_k * vecs; w += kThreads) {
    const int h = w / vecs, k = w - h * vecs;
    *reinterpret_cast<u32x4*>(a.cache.values + a.cache.row(page, h, slot) * line + k * 16) =
        *reinterpret_cast<const u32x4*>(a.values + (row * a.value_stride) * E::kBytes + h * line + k * 16);
  }
}

struct SettleArgs {
  CacheView cache;
  int64_t n_d, layer_bytes;
  const int32_t* cu;
  const int32_t* accepted_len;
  const int32_t* accepted_nodes;
  int32_t* new_len;
  int32_t line;  // bytes of a row
};

// One workgroup per request and (layer, keys or values, head).  The accepted nodes ascend, so node_d
// >= d: a source is never behind the places already written, and a group of rows that is
// read, then (behind a barrier) written, cannot overwrite a row that a later group reads.  Bound by the chain of offsets,
// lengths, nodes, pages and rows: 64 trees in four layers 7.1 us for 8 MB, one tree in one layer 2.9 us.
__global__ __launch_bounds__(kThreads) void settle(SettleArgs a) {
  __shared__ int64_t from_s[kMaxNodes], to_s[kMaxNodes];
  __shared__ int32_t ok_s;
  const int t = threadIdx.x;
  const int32_t i = blockIdx.x;
  const int32_t head = blockIdx.y % a.cache.n_heads, rest = blockIdx.y / a.cache.n_heads;
  char* const base = ((rest & 1) ? a.cache.values : a.cache.keys) + (rest >> 1) * a.layer_bytes;
  const Request r = request_at(a.cu, i, a.n_d);
  const int32_t len = a.cache.len[i], acc = a.accepted_len[i];
  bool ok = r.index >= 0 && len_fits(len, r.k) && acc >= 0 && acc <= r.k && r.k <= kMaxNodes;
  if (t < kWave) {
    bool fine = true;
    int64_t from = -1, to = -1;
    if (ok && t < acc) {
      const int32_t node = a.accepted_nodes[r.first + t];
      const int32_t before = t > 0 ? a.accepted_nodes[r.first + t - 1] : -1;
      fine = node > before && node < r.k && before >= -1;
      if (fine && node != t) {
        const int64_t src = (int64_t)len + 1 + node, dst = (int64_t)len + 1 + t;
        const int32_t sp = a.cache.page(i, src), dp = a.cache.page(i, dst);
        if (sp >= 0 && dp >= 0) {
          from = a.cache.row(sp, head, src);
          to = a.cache.row(dp, head, dst);
        }
      }
    }
    fine = __ballot(!fine) == 0;
    if (t < kMaxNodes) {
      from_s[t] = from;
      to_s[t] = to;
    }
    if (t == 0) ok_s = ok && fine;
  }
  __syncthreads();
  ok = ok_s;
  if (t == 0 && blockIdx.y == 0) a.new_len[i] = ok ? len + 1 + acc : len;
  if (!ok) return;
  const int vecs = a.line / 16;         // 8 to 64, a power of two
  const int rows = kThreads / vecs;     // rows of a group
  const int k = t & (vecs - 1), d0 = t / vecs;
  for (int32_t g = 0; g < acc; g += rows) {
    const int32_t d = g + d0;
    const bool move = d < acc && from_s[d < kMaxNodes ? d : 0] >= 0;
    u32x4 v;
    if (move) v = *reinterpret_cast<const u32x4*>(base + from_s[d] * a.line + k * 16);
    __syncthreads();
    if (move) *reinterpret_cast<u32x4*>(base + to_s[d] * a.line + k * 16) = v;
  }
}

}  // namespace cache_impl

extern "C" int sdv_kv_append(const sdv_cache* cache, int32_t B, int64_t n_draft_rows, const int32_t* ragged_offsets,
                             const int32_t* parents, const void* keys, int64_t key_stride, const void* values,
                             int64_t value_stride, const float* inv_freq, int32_t rotary, int32_t interleaved,
                             const void* queries, int64_t query_stride, int32_t n_q_heads, void* queries_out,
                             void* stream) {
  using namespace cache_impl;
  const int rc = check_cache(cache, B, n_draft_rows, ragged_offsets);
  if (rc != SDV_OK) return rc;
  const int64_t per = cache->dtype == SDV_BF16 ? 8 : 4, row = (int64_t)cache->n_kv_heads * cache->head_dim;
  if (!keys || !values || !aligned16(keys) || !aligned16(values) || key_stride < row || value_stride < row ||
      key_stride % per || value_stride % per || rotary < 0 || rotary > cache->head_dim || rotary % 16 ||
      (rotary > 0) != (inv_freq != nullptr) || n_q_heads < 0 || (n_q_heads > 0) != (queries != nullptr) ||
      (n_q_heads > 0) != (queries_out != nullptr))
    return SDV_ERR_INVALID_ARG;
  const int64_t q_row = (int64_t)n_q_heads * cache->head_dim;
  if (n_q_heads > 0 &&
      (!aligned16(queries) || !aligned16(queries_out) || query_stride < q_row || query_stride % per ||
       (queries == queries_out && query_stride != q_row)))
    return SDV_ERR_INVALID_ARG;
  if (too_many(n_draft_rows + B, kThreads) || n_q_heads > 1024 || key_stride > ((int64_t)1 << 31) || value_stride > ((int64_t)1 << 31) ||
      query_stride > ((int64_t)1 << 31))
    return SDV_ERR_LIMIT;
  AppendArgs a;
  a.cache = view_of(cache);
  a.B = B;
  a.D = cache->head_dim;
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
  const dim3 grid((unsigned)(n_draft_rows + B)), block(kThreads);
  const hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (cache->dtype == SDV_BF16) {
    if (interleaved)
      hipLaunchKernelGGL((append<Bf16, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((append<Bf16, false>), grid, block, 0, s, a);
  } else {
    if (interleaved)
      hipLaunchKernelGGL((append<F32, true>), grid, block, 0, s, a);
    else
      hipLaunchKernelGGL((append<F32, false>), grid, block, 0, s, a);
  }
  return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
}

extern "C" int sdv_kv_settle(const sdv_cache* cache, int32_t n_layers, int32_t B, int64_t n_draft_rows,
                             const int32_t* ragged_offsets, const int32_t* accepted_len,
                             const int32_t* accepted_nodes, int32_t* new_len, void* stream) {
  using namespace cache_impl;
  const int rc = check_cache(cache, B, n_draft_rows, ragged_offsets);
  if (rc != SDV_OK) return rc;
  if (n_layers < 1 || !accepted_len || (n_draft_rows > 0 && !accepted_nodes) || !new_len) return SDV_ERR_INVALID_ARG;
  if ((int64_t)n_layers * cache->n_kv_heads * 2 > 65535 || too_many(B, kThreads)) return SDV_ERR_LIMIT;
  // every workgroup of a request reads these while one of them writes new_len
  const int64_t word = sizeof(int32_t), own = B * word;
  if (overlap(new_len, own, cache->cache_len, own) || overlap(new_len, own, accepted_len, own) ||
      overlap(new_len, own, ragged_offsets, own + word) || overlap(new_len, own, accepted_nodes, n_draft_rows * word) ||
      overlap(new_len, own, cache->page_table, own * cache->max_pages))
    return SDV_ERR_INVALID_ARG;
  SettleArgs a;
  a.cache = view_of(cache);
  a.n_d = n_draft_rows;
  a.line = cache->head_dim * (cache->dtype == SDV_BF16 ? 2 : 4);
  a.layer_bytes = cache->n_pages * cache->n_kv_heads * (int64_t)cache->page_size * a.line;
  a.cu = ragged_offsets;
  a.accepted_len = accepted_len;
  a.accepted_nodes = accepted_nodes;
  a.new_len = new_len;
  hipLaunchKernelGGL(settle, dim3((unsigned)B, (unsigned)(n_layers * cache->n_kv_heads * 2)), dim3(kThreads), 0,
                     reinterpret_cast<hipStream_t>(stream), a);
  return hipGetLastError() == hipSuccess ? SDV_OK : SDV_ERR_HIP;
}
