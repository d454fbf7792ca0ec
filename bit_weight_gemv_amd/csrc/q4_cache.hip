// q4_cache.hip -- rows of the 4-bit key/value cache: appended (rotated and
// packed) and read back.
//
// Appending.  A pair of dimensions turns by a = position * inv_freq:
//   x1' = f (x1 cos a - x2 sin a),  x2' = f (x2 cos a + x1 sin a),
// then every 64 values of a key or a value are packed by the rule of
// q4_pack_affine: lo, hi widened to 0; s = fp16((hi - lo) / 15); z the integer
// nearest to -lo / s; code the level (j - z) s nearest to x, midpoints down.
// Rotation and decisions are in fp64, so that a row is the formula's, bit for
// bit, whatever order a compiler gives the products: a position times an fp32
// frequency is exact in 53 bits below position 2^29, and a midpoint (at most
// 5 + 11 bits) is compared exactly.
//
// Work split: a workgroup per token (several where there are few tokens)
// makes the token's sines once in LDS for all heads; 8 values a lane, so 8
// lanes hold a block of 64 and find its extremes in three DPP steps.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_cache_internal.h"
#include "q4_device.h"

namespace q4 {

constexpr int kAppendThreads = 256;

template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xF, 0xF, true);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xF, 0xF, true);
    return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}

// The largest of 8 lanes' values (lanes 8i .. 8i + 7); all get it.
__device__ __forceinline__ double oct_max(double v) {
    v = fmax(v, dpp_d<kDppQuadXor1>(v));
    v = fmax(v, dpp_d<kDppQuadXor2>(v));
    return fmax(v, dpp_d<kDppRowHalfMirror>(v));
}

// A non-negative double as fp16 bits, nearest even (an infinity from 65520).
__device__ __forceinline__ uint32_t f16_of(double v) {
    if (!(v < 65520.0)) return 0x7C00u;
    // A step of fp16 at v: 2^-24 below 2^-14, 2^(e - 10) in a binade.
    int e = (int)(__builtin_bit_cast(uint64_t, v) >> 52) - 1023;
    e = e < -14 ? -14 : e;
    const double n = rint(ldexp(v, 10 - e));  // nearest even
    return (uint32_t)((e + 14) << 10) + (uint32_t)n;  // (a carry moves to the next binade)
}

template <bool BF16>
__device__ __forceinline__ void load8(const void *p, int64_t at, double (&x)[8]) {
    if constexpr (BF16) {
        const u32x4_t w = *reinterpret_cast<const u32x4_t *>(static_cast<const uint16_t *>(p) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = w[i];
            x[2 * i] = (double)__builtin_bit_cast(float, u << 16);
            x[2 * i + 1] = (double)__builtin_bit_cast(float, u & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float4_t w = *reinterpret_cast<const float4_t *>(static_cast<const float *>(p) + at + 4 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) x[4 * h + i] = (double)w[i];
        }
    }
}

struct AppendArgs {
    CacheAppend a;
    int tasks, lanes;  // lanes a token needs; lanes a row needs
    int parts;         // workgroups a token
};

template <bool BF16>
__global__ __launch_bounds__(kAppendThreads) void cache_append_kernel(AppendArgs g) {
    __shared__ double2 turn[Q4_CACHE_MAX_D / 2];
    const CacheAppend &a = g.a;
    const int64_t t = blockIdx.x / g.parts;
    const int part = (int)(blockIdx.x % g.parts);
    const int D = (int)a.cache.D, rot = (int)a.rot, half = rot / 2;
    const int32_t slot = a.slots[t];
    const bool live = slot >= 0 && slot < a.cache.pages * a.cache.page;
    if ((int)threadIdx.x < half) {
        const double angle = (double)a.positions[t] * (double)a.inv_freq[threadIdx.x];
        double sn, cs;
        sincos(angle, &sn, &cs);
        turn[threadIdx.x] = make_double2((double)a.amplitude * cs, (double)a.amplitude * sn);
    }
    __syncthreads();
    const int heads = (int)a.cache.heads;
    for (int i = part * kAppendThreads + (int)threadIdx.x; i < g.tasks; i += g.parts * kAppendThreads) {
        const int row = i / g.lanes, k0 = (i - row * g.lanes) * 8;
        // Rows of a token: its keys, its values, its queries.
        const bool is_v = row >= heads && row < 2 * heads, is_q = row >= 2 * heads;
        if (!is_q && !live) continue;
        const int h = is_q ? row - 2 * heads : is_v ? row - heads : row;
        const void *src = is_q ? a.q : is_v ? a.v : a.k;
        const int64_t base = t * (is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride) + (int64_t)h * D;
        double x[8];
        load8<BF16>(src, base + k0, x);
        if (!is_v && k0 < rot) {
            if (a.interleaved) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const double2 r = turn[k0 / 2 + e];
                    const double x1 = x[2 * e], x2 = x[2 * e + 1];
                    x[2 * e] = x1 * r.x - x2 * r.y;
                    x[2 * e + 1] = x2 * r.x + x1 * r.y;
                }
            } else {
                const bool first = k0 < half;  // half is a multiple of 8
                double o[8];
                load8<BF16>(src, base + (first ? k0 + half : k0 - half), o);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const double2 r = turn[(first ? k0 : k0 - half) + e];
                    x[e] = first ? x[e] * r.x - o[e] * r.y : x[e] * r.x + o[e] * r.y;
                }
            }
        }
        if (is_q) {
            typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
            bf8 v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (__bf16)(float)x[e];
            *reinterpret_cast<bf8 *>(a.q_out + (t * a.q_heads + h) * D + k0) = v;
            continue;
        }
        double hi = 0, nlo = 0;
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            bad = bad || !__builtin_isfinite(x[e]);
            hi = fmax(hi, x[e]);
            nlo = fmax(nlo, -x[e]);
        }
        hi = oct_max(hi);
        nlo = oct_max(nlo);
        bad = ((__ballot(bad) >> (__lane_id() & ~7u)) & 0xFF) != 0;
        uint32_t s16 = f16_of((hi + nlo) / 15.0);
        bad = bad || s16 == 0x7C00u;
        const float s = f16_bits_to_f32(s16);
        const double sd = (double)s;
        int z = 0;
        uint32_t word = 0;
        if (!bad && s16 != 0) {
            // The nearest integer, from an estimate that is off by one at
            // most, corrected by comparisons that are exact.
            const float inv = 1.0f / s;
            z = (int)ceilf((float)nlo * inv - 0.5f);
            z = z < 0 ? 0 : z > 15 ? 15 : z;
            if (z < 15 && nlo > ((double)z + 0.5) * sd) ++z;
            else if (z > 0 && !(nlo > ((double)z - 0.5) * sd)) --z;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                int c = (int)ceilf((float)x[e] * inv + ((float)z - 0.5f));
                c = c < 0 ? 0 : c > 15 ? 15 : c;
                if (c < 15 && x[e] > ((double)(c - z) + 0.5) * sd) ++c;
                else if (c > 0 && !(x[e] > ((double)(c - z) - 0.5) * sd)) --c;
                word |= (uint32_t)c << (4 * e);
            }
        }
        if (bad) s16 = 0x7E00u;
        const int64_t page = a.cache.page;
        const int64_t r = ((int64_t)slot / page * heads + h) * page + slot % page;
        uint8_t *codes = is_v ? a.cache.v_codes : a.cache.k_codes;
        *reinterpret_cast<uint32_t *>(codes + r * (D / 2) + k0 / 2) = word;
        if ((k0 & 63) == 0) {
            const int64_t b = r * (D / 64) + k0 / 64;
            (is_v ? a.cache.v_scales : a.cache.k_scales)[b] = (uint16_t)s16;
            (is_v ? a.cache.v_zeros : a.cache.k_zeros)[b] = __builtin_bit_cast(unsigned short, (_Float16)(float)z);
        }
    }
}

hipError_t launch_cache_append(const CacheAppend &a, hipStream_t stream) {
    AppendArgs g = {};
    g.a = a;
    g.lanes = (int)(a.cache.D / 8);
    g.tasks = (int)((2 * a.cache.heads + a.q_heads) * g.lanes);
    // A workgroup per token where the tokens fill the card, else one for
    // every 256 lanes of work.
    const int rounds = (g.tasks + kAppendThreads - 1) / kAppendThreads;
    g.parts = a.T >= 1024 ? 1 : rounds;
    void *args[] = {&g};
    return hipLaunchKernel(a.bf16 ? reinterpret_cast<const void *>(&cache_append_kernel<true>)
                                  : reinterpret_cast<const void *>(&cache_append_kernel<false>),
                           dim3((unsigned)(a.T * g.parts)), dim3(kAppendThreads), args, 0, stream);
}

// Reading: a lane makes 8 values (4 bytes of codes, 16 or 32 bytes out).
// (code - z) s is exact in fp32 for an integer z (5 by 11 bits), so a bf16
// value is rounded once.
struct ReadArgs {
    q4_cache c;
    const int32_t *slots;
    void *out[2];
    int64_t units;  // lanes of work a plane
    int lanes;      // lanes a row
};

template <bool BF16>
__global__ __launch_bounds__(256) void cache_read_kernel(ReadArgs g) {
    const int64_t step = (int64_t)gridDim.x * 256;
    const bool is_v = blockIdx.y == 1 || !g.out[0];
    const uint8_t *codes = is_v ? g.c.v_codes : g.c.k_codes;
    const uint16_t *scales = is_v ? g.c.v_scales : g.c.k_scales;
    const uint16_t *zeros = is_v ? g.c.v_zeros : g.c.k_zeros;
    void *out = is_v ? g.out[1] : g.out[0];
    const int heads = (int)g.c.heads, D = (int)g.c.D, page = (int)g.c.page;
    for (int64_t u = (int64_t)blockIdx.x * 256 + threadIdx.x; u < g.units; u += step) {
        const int64_t row = u / g.lanes;
        const int k0 = (int)(u - row * g.lanes) * 8;
        const int64_t i = row / heads;
        const int h = (int)(row - i * heads);
        const int32_t slot = g.slots[i];
        float y[8] = {};
        if (slot >= 0 && slot < g.c.pages * page) {
            const int64_t r = ((int64_t)(slot / page) * heads + h) * page + slot % page;
            const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + r * (D / 2) + k0 / 2);
            const int64_t b = r * (D / 64) + k0 / 64;
            const float s = f16_bits_to_f32(scales[b]), z = f16_bits_to_f32(zeros[b]);
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = ((float)((w >> (4 * e)) & 15) - z) * s;
        }
        if constexpr (BF16) {
            typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
            bf8 v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (__bf16)y[e];
            *reinterpret_cast<bf8 *>(static_cast<uint16_t *>(out) + row * D + k0) = v;
        } else {
            float *o = static_cast<float *>(out) + row * D + k0;
            *reinterpret_cast<float4_t *>(o) = float4_t{y[0], y[1], y[2], y[3]};
            *reinterpret_cast<float4_t *>(o + 4) = float4_t{y[4], y[5], y[6], y[7]};
        }
    }
}

hipError_t launch_cache_read(const q4_cache &cache, const int32_t *slots, int64_t n, bool bf16, void *k_out,
                             void *v_out, hipStream_t stream) {
    ReadArgs g = {};
    g.c = cache;
    g.slots = slots;
    g.out[0] = k_out;
    g.out[1] = v_out;
    g.lanes = (int)(cache.D / 8);
    g.units = n * cache.heads * g.lanes;
    int64_t grid = (g.units + 255) / 256;
    if (grid > 65536) grid = 65536;
    void *args[] = {&g};
    return hipLaunchKernel(bf16 ? reinterpret_cast<const void *>(&cache_read_kernel<true>)
                                : reinterpret_cast<const void *>(&cache_read_kernel<false>),
                           dim3((unsigned)grid, k_out && v_out ? 2 : 1), dim3(256), args, 0, stream);
}

}  // namespace q4
