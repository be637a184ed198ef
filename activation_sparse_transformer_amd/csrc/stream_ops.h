// Loads and stores of data that a kernel touches once (no reuse to keep in the
// caches).
#pragma once

#include "common.h"

namespace twell {

// One 16-byte vector per lane and many small workgroups reach 6.2
// TB/s for a copy and 6.9 for a fill (512 MiB and up); workgroups that loop
// over the grid's stride 4.3 and 4.6.
typedef __attribute__((__vector_size__(4 * sizeof(uint32_t)))) uint32_t u32x4_t;

__device__ __forceinline__ uint4 load_once(const uint4* p) {
  const u32x4_t v = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p));
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_once(void* p, const uint4& v) {
  const u32x4_t w = {v.x, v.y, v.z, v.w};
  __builtin_nontemporal_store(w, reinterpret_cast<u32x4_t*>(p));
}

}  // namespace twell
