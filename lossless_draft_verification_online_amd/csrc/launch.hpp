// The bound that every launch of the drafting and cache operators keeps.
#pragma once

#include <stdint.h>

namespace sdv {

// A launch holds fewer than 2^32 threads.
inline bool too_many(int64_t workgroups, int64_t threads) { return workgroups > (int64_t)UINT32_MAX / threads; }

}  // namespace sdv
