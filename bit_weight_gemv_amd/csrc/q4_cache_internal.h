// q4_cache_internal.h -- launchers behind q4_cache.h (host side, not
// exported).  Arguments are validated by the caller.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_cache.h"

namespace q4 {

struct CacheAppend {
    q4_cache cache;
    const void *k, *v, *q;
    bool bf16;
    int64_t T, k_stride, v_stride, q_stride, q_heads;
    const int32_t *slots, *positions;
    const float *inv_freq;
    int64_t rot;
    bool interleaved;
    float amplitude;
    uint16_t *q_out;
};
hipError_t launch_cache_append(const CacheAppend &a, hipStream_t stream);

hipError_t launch_cache_read(const q4_cache &cache, const int32_t *slots, int64_t n, bool bf16, void *k_out,
                             void *v_out, hipStream_t stream);

struct CacheAttend {
    const uint16_t *q;
    int64_t T, q_heads, q_stride;
    q4_cache cache;
    const int32_t *table;
    int64_t B, table_pages;
    const int32_t *lens, *q_offsets;
    int64_t max_q;
    bool causal;
    int64_t window;
    float scale;
    bool bf16;
    void *out;
    float *lse;
};
size_t attend_ws_bytes(int64_t T, int64_t q_heads, int64_t heads, int64_t D, int64_t B, int64_t max_q);
hipError_t launch_cache_attend(const CacheAttend &a, void *workspace, hipStream_t stream);

}  // namespace q4
