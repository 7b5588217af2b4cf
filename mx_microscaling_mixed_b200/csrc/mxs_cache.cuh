// mxs_cache.cuh -- the K/V cache pool as the serving kernels see it.
#pragma once

#include "mxs_internal.cuh"

namespace mxs {

struct CacheView {
  uint8_t *codes[2], *scales[2];          // K, V
  int64_t code_pitch[2], scale_pitch[2];
  int64_t n_slots;
  int32_t n_kvh, d, bits;
};

// Host: checks the cache (one width, identity layout, matching rows) and
// fills *v.
mxs_status cache_view(const mxs_kv_cache *c, CacheView *v);

// Records an index out of range in the device status word (a timeout that
// is already there stays).
__device__ __forceinline__ void record_bad_index(int *status) { atomicCAS(status, 0, static_cast<int>(MXS_ERR_SHAPE)); }

}  // namespace mxs
