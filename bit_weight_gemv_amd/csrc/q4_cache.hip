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
// lanes hold a block of 64 and find its extremes in three DPP steps.  Bound by
// bytes in prompts: 8191 tokens of 40 + 8 heads of 128 in 53.5 us, 3.9 TB/s
// (the sines and the keys in 64 bits are made before most of the queries
// stream; queries in 64 bits too cost 15 us more); by a chain of loads, sine
// and packing for few tokens, 4.8 us.
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
__device__ __forceinline__ float oct_max(float v) {
    v = fmaxf(v, dpp_f<kDppQuadXor1>(v));
    v = fmaxf(v, dpp_f<kDppQuadXor2>(v));
    return fmaxf(v, dpp_f<kDppRowHalfMirror>(v));
}
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

// 8 values as they lie in memory.
template <bool BF16>
struct Raw8 {
    u32x4_t w[BF16 ? 1 : 2];
};

template <bool BF16>
__device__ __forceinline__ Raw8<BF16> load8(const void *p, int64_t at) {
    Raw8<BF16> r;
    const char *q = static_cast<const char *>(p) + at * (BF16 ? 2 : 4);
#pragma unroll
    for (int h = 0; h < (BF16 ? 1 : 2); ++h) r.w[h] = reinterpret_cast<const u32x4_t *>(q)[h];
    return r;
}

template <bool BF16>
__device__ __forceinline__ void widen8(const Raw8<BF16> &r, float (&x)[8]) {
    if constexpr (BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t u = r.w[0][i];
            x[2 * i] = __builtin_bit_cast(float, u << 16);
            x[2 * i + 1] = __builtin_bit_cast(float, u & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t u = r.w[h][i];
                x[4 * h + i] = __builtin_bit_cast(float, u);
            }
    }
}

struct AppendArgs {
    CacheAppend a;
    int tasks, lanes;  // lanes a token needs; lanes a row needs
    int parts;         // workgroups a token
    int page_shift;
};

// The 8 values of the lane, turned: x the lane's, o those of the other half
// (pairs (i, i + rot/2)); cos and sin of pair i are turn[i].x and turn[i].y.
template <class F, class F2>
__device__ __forceinline__ void turn8(F (&x)[8], const F (&o)[8], const F2 *turn, int k0, int half, bool interleaved) {
    if (interleaved) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const F2 r = turn[k0 / 2 + e];
            const F x1 = x[2 * e], x2 = x[2 * e + 1];
            x[2 * e] = x1 * r.x - x2 * r.y;
            x[2 * e + 1] = x2 * r.x + x1 * r.y;
        }
    } else {
        const bool first = k0 < half;  // half is a multiple of 8
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const F2 r = turn[(first ? k0 : k0 - half) + e];
            x[e] = first ? x[e] * r.x - o[e] * r.y : x[e] * r.x + o[e] * r.y;
        }
    }
}

struct Packed8 {
    uint32_t codes, scale, zero;
};

// Packs the block of 64 that 8 lanes hold.  F is double where the values are
// not exact in fp32; a midpoint (at most 5 + 11 bits) is exact in both.
template <class F>
__device__ __forceinline__ Packed8 pack8(const F (&x)[8]) {
    F hi = 0, nlo = 0;
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
    Packed8 p = {0, f16_of(((double)hi + (double)nlo) / 15.0), 0};
    bad = bad || p.scale == 0x7C00u;
    if (bad) {
        p.scale = 0x7E00u;
    } else if (p.scale != 0) {
        const float s = f16_bits_to_f32(p.scale);
        // The nearest integer, from an estimate that is off by one at most,
        // corrected by comparisons that are exact.
        const float inv = 1.0f / s;
        const F sf = (F)s, half = (F)0.5;
        int z = (int)ceilf((float)nlo * inv - 0.5f);
        z = z < 0 ? 0 : z > 15 ? 15 : z;
        const bool z_up = nlo > ((F)z + half) * sf, z_down = !(nlo > ((F)z - half) * sf);
        z = z_up && z < 15 ? z + 1 : z_down && z > 0 ? z - 1 : z;
        const float zf = (float)z;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            // j = code - zero, an integer from -z to 15 - z.
            float j = ceilf((float)x[e] * inv - 0.5f);
            j = fminf(fmaxf(j, -zf), 15.0f - zf);
            const F m = (F)j * sf, h = half * sf;
            const bool up = x[e] > m + h, down = !(x[e] > m - h);
            j = up ? fminf(j + 1.0f, 15.0f - zf) : down ? fmaxf(j - 1.0f, -zf) : j;
            p.codes |= (uint32_t)(int)(j + zf) << (4 * e);
        }
        p.zero = __builtin_bit_cast(unsigned short, (_Float16)zf);
    }
    return p;
}

template <bool BF16>
__global__ __launch_bounds__(kAppendThreads) void cache_append_kernel(AppendArgs g) {
    __shared__ double2 turn[Q4_CACHE_MAX_D / 2];
    __shared__ float2 turn32[Q4_CACHE_MAX_D / 2];
    const CacheAppend &a = g.a;
    const int64_t t = blockIdx.x / g.parts;
    const int part = (int)(blockIdx.x % g.parts);
    const int D = (int)a.cache.D, rot = (int)a.rot, half = rot / 2, heads = (int)a.cache.heads;
    const int32_t slot = a.slots[t];
    const bool live = slot >= 0 && slot < a.cache.pages * a.cache.page;

    // Rows of a token: its keys, its values, its queries.
    struct Task {
        Raw8<BF16> x, o;
        int row, k0;
        bool is_v, is_q, turns;
    };
    auto load = [&](int i) {
        Task s;
        s.row = i / g.lanes;
        s.k0 = (i - s.row * g.lanes) * 8;
        s.is_v = s.row >= heads && s.row < 2 * heads;
        s.is_q = s.row >= 2 * heads;
        s.turns = !s.is_v && s.k0 < rot;
        if (i < g.tasks) {
            const void *src = s.is_q ? a.q : s.is_v ? a.v : a.k;
            const int h = s.is_q ? s.row - 2 * heads : s.is_v ? s.row - heads : s.row;
            const int64_t at = t * (s.is_q ? a.q_stride : s.is_v ? a.v_stride : a.k_stride) + (int64_t)h * D + s.k0;
            s.x = load8<BF16>(src, at);
            s.o = s.turns && !a.interleaved ? load8<BF16>(src, s.k0 < half ? at + half : at - half) : s.x;
        }
        return s;
    };
    // The first values are on their way while the sines are made, and behind
    // what the sines need (loads arrive in order).
    double angle = 0;
    if ((int)threadIdx.x < half) angle = (double)a.positions[t] * (double)a.inv_freq[threadIdx.x];
    const int first = part * kAppendThreads + (int)threadIdx.x, step = g.parts * kAppendThreads;
    Task s = load(first);
    if ((int)threadIdx.x < half) {
        double sn, cs;
        sincos(angle, &sn, &cs);
        const double2 r = make_double2((double)a.amplitude * cs, (double)a.amplitude * sn);
        turn[threadIdx.x] = r;
        turn32[threadIdx.x] = make_float2((float)r.x, (float)r.y);
    }
    __syncthreads();
    for (int i = first; i < g.tasks; i += step) {
        const Task c = s;
        s = load(i + step);
        if (c.is_q) {
            // Queries leave in bf16: fp32 is enough.
            typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
            float x[8], o[8];
            widen8<BF16>(c.x, x);
            widen8<BF16>(c.o, o);
            if (c.turns) turn8(x, o, turn32, c.k0, half, a.interleaved);
            bf8 v;
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = (__bf16)x[e];
            *reinterpret_cast<bf8 *>(a.q_out + (t * a.q_heads + c.row - 2 * heads) * D + c.k0) = v;
            continue;
        }
        if (!live) continue;
        float x[8];
        widen8<BF16>(c.x, x);
        Packed8 p;
        if (c.is_v) {
            p = pack8<float>(x);
        } else {
            double xd[8], od[8];
            float o[8];
            widen8<BF16>(c.o, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                xd[e] = (double)x[e];
                od[e] = (double)o[e];
            }
            if (c.turns) turn8(xd, od, turn, c.k0, half, a.interleaved);
            p = pack8<double>(xd);
        }
        const int h = c.is_v ? c.row - heads : c.row;
        const int page = (int)a.cache.page;
        const int64_t r = ((int64_t)(slot >> g.page_shift) * heads + h) * page + (slot & (page - 1));
        *reinterpret_cast<uint32_t *>((c.is_v ? a.cache.v_codes : a.cache.k_codes) + r * (D / 2) + c.k0 / 2) = p.codes;
        if ((c.k0 & 63) == 0) {
            const int64_t b = r * (D / 64) + c.k0 / 64;
            (c.is_v ? a.cache.v_scales : a.cache.k_scales)[b] = (uint16_t)p.scale;
            (c.is_v ? a.cache.v_zeros : a.cache.k_zeros)[b] = (uint16_t)p.zero;
        }
    }
}

hipError_t launch_cache_append(const CacheAppend &a, hipStream_t stream) {
    AppendArgs g = {};
    g.a = a;
    g.page_shift = __builtin_ctzll((unsigned long long)a.cache.page);
    g.lanes = (int)(a.cache.D / 8);
    g.tasks = (int)((2 * a.cache.heads + a.q_heads) * g.lanes);
    // A workgroup per token where the tokens fill the card, else one for
    // every 256 lanes of work (which makes the sines again in each).  Appended
    // and read back, 40 + 8 heads of 128: 256 tokens 9.3 us against 8.5 split,
    // 512 tokens 10.6 against 11.7, 8191 tokens 59 against 102; 16 + 2 heads:
    // 512 tokens 8.6 against 8.3, 1024 tokens 9.5 against 11.2.
    const int rounds = (g.tasks + kAppendThreads - 1) / kAppendThreads;
    g.parts = a.T * rounds >= 1536 ? 1 : rounds;
    void *args[] = {&g};
    return hipLaunchKernel(a.bf16 ? reinterpret_cast<const void *>(&cache_append_kernel<true>)
                                  : reinterpret_cast<const void *>(&cache_append_kernel<false>),
                           dim3((unsigned)(a.T * g.parts)), dim3(kAppendThreads), args, 0, stream);
}

// Reading: a lane makes 8 values (4 bytes of codes, 16 or 32 bytes out) of
// each of ROUNDS rows, whose loads go out together.  (code - z) s is exact in
// fp32 for an integer z (5 by 11 bits), so a bf16 value is rounded once.  Bound
// by the bytes written: 20000 rows of 8 heads of 128 in 24.5 us, 4.3 TB/s, with
// 4 rounds (27.9 with one); 37 rows of 12 heads of 64 in 3.2 us with one (4.0
// with 4), which holds while the workgroups do not fill the card.

struct ReadArgs {
    q4_cache c;
    const int32_t *slots;
    void *out[2];
    int64_t rows;  // n heads
    int page_shift;
};

template <bool BF16, int ND, int kReadRounds>
__global__ __launch_bounds__(256) void cache_read_kernel(ReadArgs g) {
    constexpr int D = ND * 64, kLanes = 8 * ND, kRows = 256 / kLanes;  // rows a round
    const bool is_v = blockIdx.y == 1 || !g.out[0];
    const uint8_t *codes = is_v ? g.c.v_codes : g.c.k_codes;
    const uint16_t *scales = is_v ? g.c.v_scales : g.c.k_scales;
    const uint16_t *zeros = is_v ? g.c.v_zeros : g.c.k_zeros;
    void *out = is_v ? g.out[1] : g.out[0];
    const uint32_t heads = (uint32_t)g.c.heads;
    const int page = (int)g.c.page;
    const int in = (int)threadIdx.x / kLanes, k0 = (int)(threadIdx.x % kLanes) * 8;
    if (in >= kRows) return;
    for (int64_t row0 = (int64_t)blockIdx.x * (kRows * kReadRounds) + in; row0 < g.rows;
         row0 += (int64_t)gridDim.x * (kRows * kReadRounds)) {
        int32_t slot[kReadRounds];
        uint32_t h[kReadRounds], w[kReadRounds], sb[kReadRounds], zb[kReadRounds];
#pragma unroll
        for (int j = 0; j < kReadRounds; ++j) {
            const int64_t row = row0 + j * kRows;
            const uint32_t u = (uint32_t)(row < g.rows ? row : row0), i = u / heads;  // rows are below 2^32
            h[j] = u - i * heads;
            slot[j] = g.slots[i];
        }
#pragma unroll
        for (int j = 0; j < kReadRounds; ++j) {
            const bool ok = slot[j] >= 0 && slot[j] < g.c.pages * page;
            w[j] = sb[j] = zb[j] = 0;
            if (ok) {
                const int64_t r = ((int64_t)(slot[j] >> g.page_shift) * heads + h[j]) * page + (slot[j] & (page - 1));
                w[j] = *reinterpret_cast<const uint32_t *>(codes + r * (D / 2) + k0 / 2);
                sb[j] = scales[r * ND + k0 / 64];
                zb[j] = zeros[r * ND + k0 / 64];
            }
        }
#pragma unroll
        for (int j = 0; j < kReadRounds; ++j) {
            const int64_t row = row0 + j * kRows;
            if (row >= g.rows) break;
            const float s = f16_bits_to_f32(sb[j]), z = f16_bits_to_f32(zb[j]);
            float y[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) y[e] = ((float)((w[j] >> (4 * e)) & 15) - z) * s;
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
}

template <int ND, int ROUNDS>
static const void *read_kernel(bool bf16) {
    return bf16 ? reinterpret_cast<const void *>(&cache_read_kernel<true, ND, ROUNDS>)
                : reinterpret_cast<const void *>(&cache_read_kernel<false, ND, ROUNDS>);
}

hipError_t launch_cache_read(const q4_cache &cache, const int32_t *slots, int64_t n, bool bf16, void *k_out,
                             void *v_out, hipStream_t stream) {
    ReadArgs g = {};
    g.c = cache;
    g.slots = slots;
    g.out[0] = k_out;
    g.out[1] = v_out;
    g.rows = n * cache.heads;
    g.page_shift = __builtin_ctzll((unsigned long long)cache.page);
    const int64_t per = 256 / (cache.D / 8);
    const bool many = g.rows >= per * 2048;  // 8 workgroups a compute unit and plane
    int64_t grid = (g.rows + per * (many ? 4 : 1) - 1) / (per * (many ? 4 : 1));
    if (grid > 1 << 20) grid = 1 << 20;
    void *args[] = {&g};
    const void *few_f[4] = {read_kernel<1, 1>(bf16), read_kernel<2, 1>(bf16), read_kernel<3, 1>(bf16), read_kernel<4, 1>(bf16)};
    const void *many_f[4] = {read_kernel<1, 4>(bf16), read_kernel<2, 4>(bf16), read_kernel<3, 4>(bf16), read_kernel<4, 4>(bf16)};
    return hipLaunchKernel((many ? many_f : few_f)[cache.D / 64 - 1], dim3((unsigned)grid, k_out && v_out ? 2 : 1), dim3(256), args,
                           0, stream);
}

}  // namespace q4
