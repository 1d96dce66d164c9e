// What the kernels over a paged cache in 8 bits share: the scales' places, codes brought from one scale to another,
// and the checks of a call's arguments.
#pragma once

#include "cache_view.hpp"

namespace sdv {

constexpr int kMaxBlock = 64;

struct Cache8View {
  CacheView cache;
  uint8_t* key_scales;
  uint8_t* value_scales;
  int32_t block_log2;

  // The scale of slot s's block in its page.
  __device__ __forceinline__ int64_t scale_at(int32_t page, int32_t head, int64_t s) const {
    const int64_t in = s & ((1 << cache.page_log2) - 1);
    return (((int64_t)page * cache.n_heads + head) << (cache.page_log2 - block_log2)) + (in >> block_log2);
  }
};

// A scale's byte b is 2^(b - 127), from 10 to 246: every code times every scale is then a normal binary32 (and bf16) number.
constexpr int32_t kScaleLow = 10, kScaleHigh = 246;
__device__ __forceinline__ int32_t scale_byte(int32_t b) { return b < kScaleLow ? kScaleLow : (b > kScaleHigh ? kScaleHigh : b); }
__device__ __forceinline__ float scale_of(int32_t byte) { return __uint_as_float((uint32_t)scale_byte(byte) << 23); }

// Four codes times 2^-shift (shift > 0): exact in binary32, rounded to the nearest code.
__device__ __forceinline__ uint32_t shifted_codes(uint32_t v, int32_t shift) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const float by = shift > 126 ? 0.0f : __uint_as_float((uint32_t)(127 - shift) << 23);
  const f32x2 lo = __builtin_amdgcn_cvt_pk_f32_fp8(v, false), hi = __builtin_amdgcn_cvt_pk_f32_fp8(v, true);
  const uint32_t w = __builtin_amdgcn_cvt_pk_fp8_f32(lo.x * by, lo.y * by, 0, false);
  return __builtin_amdgcn_cvt_pk_fp8_f32(hi.x * by, hi.y * by, w, true);
}

inline int check_cache8(const sdv_cache8* c, int32_t B, int64_t n_d, const int32_t* cu) {
  if (!c) return SDV_ERR_INVALID_ARG;
  const int rc = check_cache(&c->cache, B, n_d, cu);
  if (rc != SDV_OK) return rc;
  if (!c->key_scales || !c->value_scales || c->block < 1 || c->block > kMaxBlock || c->block > c->cache.page_size ||
      (c->block & (c->block - 1)))
    return SDV_ERR_INVALID_ARG;
  return SDV_OK;
}

inline Cache8View view_of(const sdv_cache8* c) {
  Cache8View v;
  v.cache = view_of(&c->cache);
  v.key_scales = c->key_scales;
  v.value_scales = c->value_scales;
  v.block_log2 = log2_of(c->block);
  return v;
}

}  // namespace sdv
