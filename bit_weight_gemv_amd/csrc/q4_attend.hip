// q4_attend.hip -- attention over the 4-bit key/value cache.
//
// A wave per (token, query head) walks the seen keys once with the running
// maximum m and sum l of the softmax: with a key's score s,
//   m' = max(m, s),  l' = l e^(m - m') + e^(s - m'),  o' = o e^(m - m') + e^(s - m') v.
// A lane holds dimensions lane + 64 b.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "q4_cache_internal.h"
#include "q4_device.h"

namespace q4 {

struct AttendArgs {
    CacheAttend a;
    int page_shift;
};

// The sequence that token t belongs to: the last b with q_offsets[b] <= t.
__device__ __forceinline__ int64_t sequence_of(const int32_t *offsets, int64_t B, int64_t t) {
    int64_t lo = 0, hi = B + 1;  // offsets before lo are <= t, from hi on > t
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (offsets[mid] <= t) lo = mid + 1;
        else hi = mid;
    }
    return lo - 1;
}

template <int ND>
__global__ __launch_bounds__(64) void attend_row_kernel(AttendArgs g) {
    const CacheAttend &a = g.a;
    const int lane = (int)threadIdx.x, D = ND * 64;
    const int64_t t = blockIdx.x / a.q_heads, hq = blockIdx.x % a.q_heads;
    int64_t b = t, n = 1, j = 0;
    if (a.q_offsets) {
        b = sequence_of(a.q_offsets, a.B, t);
        if (b < 0 || b >= a.B) return;
        const int64_t first = a.q_offsets[b] < 0 ? 0 : a.q_offsets[b];
        n = a.q_offsets[b + 1];
        n = (n > a.T ? a.T : n) - first;
        j = t - first;
        if (j >= a.max_q) return;
    }
    const int64_t heads = a.cache.heads, page = a.cache.page, h = hq / (a.q_heads / heads);
    int64_t len = a.lens[b];
    const int64_t most = a.table_pages * page;
    len = len < 0 ? 0 : len > most ? most : len;
    const int64_t pos = len - n + j;
    const int64_t hi = a.causal ? pos + 1 : len;
    const int64_t lo = a.window > 0 && pos - a.window + 1 > 0 ? pos - a.window + 1 : 0;
    float q[ND], o[ND];
#pragma unroll
    for (int i = 0; i < ND; ++i) {
        q[i] = __builtin_bit_cast(float, (uint32_t)a.q[t * a.q_stride + hq * D + 64 * i + lane] << 16);
        o[i] = 0;
    }
    float m = -INFINITY, l = 0;
    for (int64_t i = lo; i < hi; ++i) {
        const int32_t id = a.table[b * a.table_pages + (i >> g.page_shift)];
        if (id < 0 || id >= a.cache.pages) continue;
        const int64_t r = ((int64_t)id * heads + h) * page + (i & (page - 1));
        float s = 0;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            const int c = (a.cache.k_codes[r * (D / 2) + 32 * d + lane / 2] >> (4 * (lane & 1))) & 15;
            s += q[d] * ((float)c - f16_bits_to_f32(a.cache.k_zeros[r * ND + d])) * f16_bits_to_f32(a.cache.k_scales[r * ND + d]);
        }
        s = wave_sum(s) * a.scale;
        const float top = fmaxf(m, s);
        const float base = top == -INFINITY ? 0.0f : top;
        const float fade = expf(m - base), p = expf(s - base);
        m = top;
        l = l * fade + p;
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            const int c = (a.cache.v_codes[r * (D / 2) + 32 * d + lane / 2] >> (4 * (lane & 1))) & 15;
            const float v = ((float)c - f16_bits_to_f32(a.cache.v_zeros[r * ND + d])) * f16_bits_to_f32(a.cache.v_scales[r * ND + d]);
            o[d] = o[d] * fade + p * v;
        }
    }
    const float inv = l == 0 ? 0.0f : 1.0f / l;
#pragma unroll
    for (int d = 0; d < ND; ++d) {
        const int64_t at = (t * a.q_heads + hq) * D + 64 * d + lane;
        const float y = l == 0 ? 0.0f : o[d] * inv;
        if (a.bf16)
            static_cast<__bf16 *>(a.out)[at] = (__bf16)y;
        else
            static_cast<float *>(a.out)[at] = y;
    }
    if (a.lse && lane == 0) a.lse[t * a.q_heads + hq] = l == 0 ? -INFINITY : m + logf(l);
}

size_t attend_ws_bytes(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_cache_attend(const CacheAttend &a, void *, hipStream_t stream) {
    AttendArgs g = {};
    g.a = a;
    g.page_shift = __builtin_ctzll((unsigned long long)a.cache.page);
    const void *fn[4] = {reinterpret_cast<const void *>(&attend_row_kernel<1>),
                         reinterpret_cast<const void *>(&attend_row_kernel<2>),
                         reinterpret_cast<const void *>(&attend_row_kernel<3>),
                         reinterpret_cast<const void *>(&attend_row_kernel<4>)};
    void *args[] = {&g};
    return hipLaunchKernel(fn[a.cache.D / 64 - 1], dim3((unsigned)(a.T * a.q_heads)), dim3(64), args, 0, stream);
}

}  // namespace q4
