// q4_route.hip -- which experts a token goes to, the order that groups the
// tokens by expert, and the weighted sum of the experts' outputs.
//
// Top k: 16 lanes a token (a wave, above 256 experts), the logits spread over
// them as bits in an order that compares as unsigned; k times the largest of
// them (maxima over lanes by DPP) goes to the lowest index that holds it.
//
// Grouping is a counting sort that keeps the slots' order: workgroups take
// consecutive runs of slots; the first launch leaves each run's count of
// every expert, the second adds up the counts before its run and ranks its
// own slots (a wave at a time, by ballots over the expert's bits).  A run
// that holds every slot needs one launch.  No atomics on memory: the same
// input gives the same plan.
//
// Measured (graph replay): 1 token, 64 experts, top 8 5.1 us in one launch (an
// empty kernel takes 1.6; the k maxima and the ranks come one after the
// other).  8192 tokens, 128 experts, top 8 14.2 us in two launches (6.8 + 7.4
// by themselves) for 5.2 MB: bound by the k rounds of two maxima (the value,
// then the index: 4 DPP steps and 8 compares a lane each), by the ranks (a
// ballot a bit, the waves one after the other), and by every workgroup of the
// second launch reading all runs' counts, not by the bytes (1 us).  With a
// wave a token it took 29 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_experts.h"
#include "q4_ragged.h"
#include "q4_ragged_device.h"

namespace q4 {

namespace {

constexpr int kRouteThreads = 512;
constexpr int kRouteWaves = kRouteThreads / 64;
constexpr int kMaxRuns = 256;    // runs of the counting sort at most
constexpr int kRunTokens = 32;   // tokens of a run at least (slots, for a plain sort: 512)

__host__ __device__ constexpr int hist_pitch(int64_t E) { return (int)(E + 3) & ~3; }

struct RouteArgs {
    const void *logits;
    int bf16, T, E, k, all;
    int32_t *experts;
    float *weights;
    int32_t *hist;    // [runs][hist_pitch(E)], or null: one run, sorted in the same launch
    int run;          // tokens of a run
    int32_t *offsets, *rows, *pos;
};

struct SortArgs {
    const int32_t *bins;
    int slots, E, per, run;  // run: slots of a run
    const int32_t *hist;     // [runs][hist_pitch(E)], or null: one run
    int32_t *offsets, *rows, *pos;
};

// A logit's bits in an order that compares as unsigned; every logit's is
// above 0.  NaN as -infinity, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float v) {
    v = v != v ? -__builtin_inff() : v + 0.0f;
    const uint32_t b = __builtin_bit_cast(uint32_t, v);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float value_of(uint32_t order) {
    return __builtin_bit_cast(float, order & 0x80000000u ? order & 0x7FFFFFFFu : ~order);
}

__device__ __forceinline__ uint32_t load_logit(const RouteArgs &a, int t, int e) {
    if (t >= a.T || e >= a.E) return 0;  // below every logit's
    const int64_t at = (int64_t)t * a.E + e;
    return order_of(a.bf16 ? bf16_f32(static_cast<const uint16_t *>(a.logits)[at])
                           : static_cast<const float *>(a.logits)[at]);
}

// Reductions over the LANES (16 or 64) lanes of a token; every one gets it.
template <int LANES>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
    if constexpr (LANES == 64) return wave_max_u32(v);
    v = dpp_max_u32<kDppQuadXor1>(v);
    v = dpp_max_u32<kDppQuadXor2>(v);
    v = dpp_max_u32<kDppRowHalfMirror>(v);
    return dpp_max_u32<kDppRowMirror>(v);
}
template <int LANES>
__device__ __forceinline__ float lanes_sum(float v) {
    if constexpr (LANES == 64) return wave_sum(v);
    v += dpp_f<kDppQuadXor1>(v);
    v += dpp_f<kDppQuadXor2>(v);
    v += dpp_f<kDppRowHalfMirror>(v);
    return v + dpp_f<kDppRowMirror>(v);
}

// The choice of token t by LANES lanes, which hold logits e = lane + LANES i.
// The lowest index among equals is the largest complement of an index.
template <int EPL, int LANES>
__device__ __forceinline__ void choose(const RouteArgs &a, int t, const uint32_t (&o)[EPL]) {
    const int lane = threadIdx.x & (LANES - 1);
    uint32_t key[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = o[i];
    float mine = 0.0f, largest = 0.0f;
    int chosen = 0;
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < EPL; ++i) best = max(best, key[i]);
        best = lanes_max<LANES>(best);
        uint32_t index = 0;
#pragma unroll
        for (int i = EPL - 1; i >= 0; --i)
            if (key[i] == best) index = ~(uint32_t)(lane + LANES * i);
        const int at = (int)~lanes_max<LANES>(index);
#pragma unroll
        for (int i = 0; i < EPL; ++i)
            if (at == lane + LANES * i) key[i] = 0;
        const float v = value_of(best);
        if (j == 0) largest = v;
        if (lane == j) {
            mine = v;
            chosen = at;
        }
    }
    const float p = lane >= a.k ? 0.0f : mine == largest ? 1.0f : expf(mine - largest);
    float s = p;
    if (a.all) {
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
            const float v = value_of(o[i]);
            if (o[i]) s += v == largest ? 1.0f : expf(v - largest);
        }
    }
    const float total = lanes_sum<LANES>(s);
    if (lane < a.k && t < a.T) {
        a.experts[(int64_t)t * a.k + lane] = chosen;
        a.weights[(int64_t)t * a.k + lane] = largest == -__builtin_inff() ? 0.0f : p / total;
    }
}

// Ranks slots s0 .. s1 - 1; next[e] is the position that the next slot of bin
// e takes (bin E: none).  Whole workgroup.
__device__ __forceinline__ void rank_run(const int32_t *bins, int s0, int s1, int E, int per, int32_t *next,
                                         int32_t *rows, int32_t *pos) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int bits = 1;
    while ((1 << bits) <= E) ++bits;
    for (int base = s0; base < s1; base += kRouteThreads) {
        const int s = base + threadIdx.x;
        const bool live = s < s1;
        int e = live ? bins[s] : E;
        if (e < 0 || e > E) e = E;
        uint64_t same = __builtin_amdgcn_ballot_w64(live);
        for (int b = 0; b < bits; ++b) {
            const uint64_t with = __builtin_amdgcn_ballot_w64((e >> b) & 1);
            same &= (e >> b) & 1 ? with : ~with;
        }
        const int before = __builtin_popcountll(same & ((1ull << lane) - 1));
        const int waves = min(kRouteWaves, (s1 - base + 63) >> 6);
        for (int w = 0; w < waves; ++w) {
            if (wave == w && live) {
                const int p = next[e] + before;
                if (before == 0) next[e] += __builtin_popcountll(same);
                rows[p] = s / per;
                if (pos) pos[s] = p;
            }
            __syncthreads();
        }
    }
}

// From counts[e] (this run's first slot of each bin comes after `before[e]`
// earlier ones, `total[e]` in all): offsets and the first positions.  LDS
// arrays of E + 1; whole workgroup.
__device__ __forceinline__ void first_positions(int E, int slots, const int32_t *total, int32_t *next, int32_t *sum,
                                                int32_t *offsets, bool write) {
    // Exclusive sums over the bins: each wave's lanes take runs of bins.
    const int n = (E + kRouteThreads - 1) / kRouteThreads;
    const int e0 = threadIdx.x * n;
    int s = 0;
    for (int i = 0; i < n; ++i)
        if (e0 + i < E) s += total[e0 + i];
    int incl = s;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int o = __shfl_up(incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 63) sum[wave] = incl;
    __syncthreads();
    int at = incl - s;
    for (int w = 0; w < wave; ++w) at += sum[w];
    for (int i = 0; i < n; ++i) {
        const int e = e0 + i;
        if (e < E) {
            if (write) offsets[e] = at;
            next[e] += at;
            at += total[e];
        }
    }
    int all = 0;
    for (int w = 0; w < kRouteWaves; ++w) all += sum[w];
    if (threadIdx.x == 0) {
        if (write) offsets[E] = all;
        next[E] += all;  // slots of no bin
    }
    __syncthreads();
    (void)slots;
}

template <int EPL, int LANES>
__global__ __launch_bounds__(kRouteThreads) void route_kernel(const RouteArgs a) {
    __shared__ int32_t total[Q4_MAX_EXPERTS + 1], next[Q4_MAX_EXPERTS + 1], sum[kRouteWaves];
    const int t0 = blockIdx.x * a.run, t1 = min(t0 + a.run, a.T);
    for (int e = threadIdx.x; e <= a.E; e += kRouteThreads) total[e] = next[e] = 0;
    for (int t = t0; t < t1; t += kRouteThreads / LANES) {
        const int mine = t + (int)threadIdx.x / LANES;
        if (mine - (int)(threadIdx.x & 63) / LANES >= t1) continue;  // the whole wave's are past the run
        uint32_t o[EPL];
        const int lt = mine < t1 ? mine : a.T;                       // (a.T: no token)
#pragma unroll
        for (int i = 0; i < EPL; ++i) o[i] = load_logit(a, lt, (threadIdx.x & (LANES - 1)) + LANES * i);
        choose<EPL, LANES>(a, lt, o);
    }
    __threadfence_block();
    __syncthreads();
    const int s0 = t0 * a.k, s1 = t1 * a.k;
    for (int s = s0 + threadIdx.x; s < s1; s += kRouteThreads) atomicAdd(&total[a.experts[s]], 1);
    __syncthreads();
    if (a.hist) {
        for (int e = threadIdx.x; e < hist_pitch(a.E); e += kRouteThreads)
            a.hist[(int64_t)blockIdx.x * hist_pitch(a.E) + e] = e < a.E ? total[e] : 0;
        return;
    }
    first_positions(a.E, s1, total, next, sum, a.offsets, true);
    rank_run(a.experts, s0, s1, a.E, a.k, next, a.rows, a.pos);
}

// Counts of each run, for a plain sort.
__global__ __launch_bounds__(kRouteThreads) void sort_count_kernel(const SortArgs a, int32_t *hist) {
    __shared__ int32_t total[Q4_MAX_EXPERTS + 1];
    for (int e = threadIdx.x; e <= a.E; e += kRouteThreads) total[e] = 0;
    __syncthreads();
    const int s0 = blockIdx.x * a.run, s1 = min(s0 + a.run, a.slots);
    for (int s = s0 + threadIdx.x; s < s1; s += kRouteThreads) {
        const int e = a.bins[s];
        if (e >= 0 && e < a.E) atomicAdd(&total[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < hist_pitch(a.E); e += kRouteThreads)
        hist[(int64_t)blockIdx.x * hist_pitch(a.E) + e] = e < a.E ? total[e] : 0;
}

__global__ __launch_bounds__(kRouteThreads) void sort_kernel(const SortArgs a) {
    __shared__ int32_t total[Q4_MAX_EXPERTS + 1], next[Q4_MAX_EXPERTS + 1], sum[kRouteWaves];
    const int s0 = blockIdx.x * a.run, s1 = min(s0 + a.run, a.slots);
    for (int e = threadIdx.x; e <= a.E; e += kRouteThreads) total[e] = next[e] = 0;
    __syncthreads();
    if (a.hist) {
        // A thread adds up four neighbouring bins of every parts'th run.
        const int quads = hist_pitch(a.E) / 4, parts = max(kRouteThreads / quads, 1);
        const int4 *h = reinterpret_cast<const int4 *>(a.hist);
        int sum_before = 0;
        for (int i = threadIdx.x; i < quads * parts; i += kRouteThreads) {
            const int quad = i % quads;
            int4 before = make_int4(0, 0, 0, 0), all = make_int4(0, 0, 0, 0);
#pragma unroll 8
            for (int b = i / quads; b < (int)gridDim.x; b += parts) {
                const int4 n = h[b * quads + quad];
                const int w = b < (int)blockIdx.x ? 1 : 0;
                before.x += n.x * w, before.y += n.y * w, before.z += n.z * w, before.w += n.w * w;
                all.x += n.x, all.y += n.y, all.z += n.z, all.w += n.w;
            }
            const int be[4] = {before.x, before.y, before.z, before.w}, al[4] = {all.x, all.y, all.z, all.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (4 * quad + e >= a.E) break;
                atomicAdd(&total[4 * quad + e], al[e]);
                atomicAdd(&next[4 * quad + e], be[e]);
                sum_before += be[e];
            }
        }
        // Slots of no bin before this run: those that the bins do not count.
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) sum_before += __shfl_xor(sum_before, d);
        if ((threadIdx.x & 63) == 0) atomicAdd(&total[a.E], sum_before);
        __syncthreads();
        if (threadIdx.x == 0) next[a.E] = s0 - total[a.E];
        __syncthreads();
    } else {
        for (int s = s0 + threadIdx.x; s < s1; s += kRouteThreads) {
            const int e = a.bins[s];
            if (e >= 0 && e < a.E) atomicAdd(&total[e], 1);
        }
        __syncthreads();
    }
    first_positions(a.E, a.slots, total, next, sum, a.offsets, blockIdx.x == 0);
    rank_run(a.bins, s0, s1, a.E, a.per, next, a.rows, a.pos);
}

struct CombineArgs {
    const void *Y;
    int y_bf16, R, M;
    const float *weights;
    const int32_t *pos;
    int T, k, out_bf16, per;  // per: workgroups a token
    void *out;
};

// A lane adds 8 neighbouring columns (VEC: rows of whole 16-byte pieces) or
// one: 4096 tokens x 8 rows of 2048, 151 MB, take 23.1 us (6.5 TB/s, most of it
// from the Infinity Cache) with 8 columns and 66.5 with one.  Bound by the
// bytes; one token's 8 rows by the launch (3.8 us).
template <bool VEC>
__global__ __launch_bounds__(256) void combine_kernel(const CombineArgs a) {
    constexpr int W = VEC ? 8 : 1;
    const int t = blockIdx.x / a.per;
    const int m = ((blockIdx.x % a.per) * 256 + threadIdx.x) * W;
    if (m >= a.M) return;
    float s[W];
#pragma unroll
    for (int i = 0; i < W; ++i) s[i] = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        const int p = a.pos[(int64_t)t * a.k + j];
        if (p < 0 || p >= a.R) continue;
        const float w = a.weights[(int64_t)t * a.k + j];
        const int64_t at = (int64_t)p * a.M + m;
        if constexpr (VEC) {
            if (a.y_bf16) {
                const uint4 v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.Y) + at);
                const uint32_t d[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s[2 * i] = fmaf(w, bf16_lo(d[i]), s[2 * i]);
                    s[2 * i + 1] = fmaf(w, bf16_hi(d[i]), s[2 * i + 1]);
                }
            } else {
                const float4 *y = reinterpret_cast<const float4 *>(static_cast<const float *>(a.Y) + at);
                const float4 u = y[0], v = y[1];
                const float d[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] = fmaf(w, d[i], s[i]);
            }
        } else {
            const float y = a.y_bf16 ? bf16_f32(static_cast<const uint16_t *>(a.Y)[at])
                                     : static_cast<const float *>(a.Y)[at];
            s[0] = fmaf(w, y, s[0]);
        }
    }
    const int64_t at = (int64_t)t * a.M + m;
    if constexpr (VEC) {
        if (a.out_bf16) {
            uint32_t d[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                d[i] = (uint32_t)f32_bf16(s[2 * i]) | (uint32_t)f32_bf16(s[2 * i + 1]) << 16;
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at) = make_uint4(d[0], d[1], d[2], d[3]);
        } else {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at);
            o[0] = make_float4(s[0], s[1], s[2], s[3]);
            o[1] = make_float4(s[4], s[5], s[6], s[7]);
        }
    } else {
        store_out(a.out, a.out_bf16, at, s[0]);
    }
}

// Items of a run, so that at most kMaxRuns runs of whole `least` cover n.
int64_t run_of(int64_t n, int64_t least) {
    const int64_t per = (n + kMaxRuns - 1) / kMaxRuns;
    return per <= least ? least : (per + least - 1) / least * least;
}

// Workgroups of the weighted sum for each token: eight columns a lane where
// every row starts on 16 bytes.
int64_t combine_per(int64_t M) {
    const int64_t columns = M % 8 == 0 ? 2048 : 256;
    return (M + columns - 1) / columns;
}

const void *route_fn(int64_t E) {
    if (E <= 16) return reinterpret_cast<const void *>(&route_kernel<1, 16>);
    if (E <= 64) return reinterpret_cast<const void *>(&route_kernel<4, 16>);
    if (E <= 128) return reinterpret_cast<const void *>(&route_kernel<8, 16>);
    if (E <= 256) return reinterpret_cast<const void *>(&route_kernel<16, 16>);
    if (E <= 512) return reinterpret_cast<const void *>(&route_kernel<8, 64>);
    return reinterpret_cast<const void *>(&route_kernel<16, 64>);
}

}  // namespace

size_t sort_ws_bytes(int64_t slots, int64_t E) {
    const int64_t run = run_of(slots, kRouteThreads), runs = (slots + run - 1) / run;
    return runs > 1 ? (size_t)runs * hist_pitch(E) * 4 : 0;
}

hipError_t launch_sort(const int32_t *bins, int64_t slots, int64_t E, int64_t per, int32_t *offsets, int32_t *rows,
                       int32_t *pos, void *workspace, hipStream_t stream) {
    SortArgs a = {};
    a.bins = bins;
    a.slots = (int)slots;
    a.E = (int)E;
    a.per = (int)per;
    a.run = (int)run_of(slots, kRouteThreads);
    a.offsets = offsets;
    a.rows = rows;
    a.pos = pos;
    int64_t runs = (slots + a.run - 1) / a.run;
    if (runs < 1) runs = 1;  // offsets are still written
    if (runs > 1) {
        int32_t *hist = static_cast<int32_t *>(workspace);
        void *cargs[] = {&a, &hist};
        const hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&sort_count_kernel), dim3((unsigned)runs),
                                             dim3(kRouteThreads), cargs, 0, stream);
        if (e != hipSuccess) return e;
        a.hist = hist;
    }
    void *args[] = {&a};
    return hipLaunchKernel(reinterpret_cast<const void *>(&sort_kernel), dim3((unsigned)runs), dim3(kRouteThreads),
                           args, 0, stream);
}

size_t route_ws_bytes(int64_t T, int64_t E, int64_t k) {
    const int64_t run = run_of(T, kRunTokens), runs = (T + run - 1) / run;
    (void)k;
    return runs > 1 ? (size_t)runs * hist_pitch(E) * 4 : 0;
}

hipError_t launch_route(const void *logits, bool bf16, int64_t T, int64_t E, int64_t k, bool all, int32_t *experts,
                        float *weights, int32_t *offsets, int32_t *rows, int32_t *pos, void *workspace,
                        hipStream_t stream) {
    RouteArgs a = {};
    a.logits = logits;
    a.bf16 = bf16;
    a.T = (int)T;
    a.E = (int)E;
    a.k = (int)k;
    a.all = all;
    a.experts = experts;
    a.weights = weights;
    a.run = (int)run_of(T, kRunTokens);
    a.offsets = offsets;
    a.rows = rows;
    a.pos = pos;
    int64_t runs = (T + a.run - 1) / a.run;
    if (runs < 1) runs = 1;
    if (runs > 1) a.hist = static_cast<int32_t *>(workspace);
    void *args[] = {&a};
    const hipError_t e = hipLaunchKernel(route_fn(E), dim3((unsigned)runs), dim3(kRouteThreads), args, 0, stream);
    if (e != hipSuccess || runs == 1) return e;
    SortArgs b = {};
    b.bins = experts;
    b.slots = (int)(T * k);
    b.E = (int)E;
    b.per = (int)k;
    b.run = (int)(a.run * k);
    b.hist = a.hist;
    b.offsets = offsets;
    b.rows = rows;
    b.pos = pos;
    void *sargs[] = {&b};
    return hipLaunchKernel(reinterpret_cast<const void *>(&sort_kernel), dim3((unsigned)runs), dim3(kRouteThreads),
                           sargs, 0, stream);
}

bool combine_fits(int64_t M, int64_t T) {
    return T * combine_per(M) * 256 < INT64_C(1) << 32;  // threads of one launch
}

hipError_t launch_combine(const void *Y, bool y_bf16, int64_t R, int64_t M, const float *weights, const int32_t *pos,
                          int64_t T, int64_t k, bool out_bf16, void *out, hipStream_t stream) {
    CombineArgs a = {};
    a.Y = Y;
    a.y_bf16 = y_bf16;
    a.R = (int)R;
    a.M = (int)M;
    a.weights = weights;
    a.pos = pos;
    a.T = (int)T;
    a.k = (int)k;
    a.out_bf16 = out_bf16;
    a.out = out;
    const bool vec = M % 8 == 0;
    a.per = (int)combine_per(M);
    void *args[] = {&a};
    return hipLaunchKernel(vec ? reinterpret_cast<const void *>(&combine_kernel<true>)
                               : reinterpret_cast<const void *>(&combine_kernel<false>),
                           dim3((unsigned)(T * a.per)), dim3(256), args, 0, stream);
}

}  // namespace q4
