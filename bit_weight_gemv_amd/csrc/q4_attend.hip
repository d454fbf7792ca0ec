// q4_attend.hip -- attention over the 4-bit key/value cache.
//
// For a row (a token's query head) with scores s_i = scale q . k_i over the
// keys it sees: out = sum p_i v_i / sum p_i, p_i = 2^(c (s_i - m)), c = log2 e.
// One pass over the keys, with the running maximum m; sums are fp32.
#include <float.h>
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "q4_cache_internal.h"
#include "q4_device.h"

namespace q4 {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef int int2_t __attribute__((ext_vector_type(2)));

// A tile of rows of the tile kernel, for the joining: parts is 0 where it has none.
struct TileRows {
    int first, row0, rows, parts;
};

typedef __attribute__((address_space(4))) int32_t scalar_int;  // read-only: uniform loads are scalar

// Where the pieces of a (sequence, key head) lie that the split kernel dealt to
// several waves; first == last: it was not.
struct Pieces {
    int first, last;  // the waves of the first and the last piece
};  // A wave's slots: 2 w for a piece that goes on, 2 w + 1 for one that begins.

struct AttendArgs {
    CacheAttend a;
    int page_shift;
    int G;            // query heads a key head
    uint32_t inv_G;   // 2^16 / G, rounded up: r inv_G / 2^16 is r / G for r < 64, G <= 64
    float c;          // scale log2 e = c 2^c_exp, c from 1/2 to 1
    int c_exp;
    int limit;        // the split kernel takes sequences of at most this many rows
    int max_rows;     // rows a partial result is kept for
    float *part;      // partial results: [slot][max_rows][D], then (ref, sum) pairs
    float *part_sums;
    Pieces *pieces;     // split kernel: [sequence][key head]
    int waves;          // its waves at most
    TileRows *tile_rows;  // tile kernel: [tile of rows]
    int64_t row_tiles;  // tile kernel: tiles of rows at most
    int parts;          // workgroups the keys of one are dealt to at most,
    int prefix_parts, prompt_parts;  // behind a long prefix, and without one
};

// A row of q enters the products times 2^ex, its largest magnitude (of these
// bf16 bits) 2^top to 2^(top + 1) then; kappa = scale log2 e 2^(shift - ex)
// makes exponents of 2 of the scores.  kappa times 2^low stays a normal number
// (a masked score is -infinity, and -infinity times 0 a NaN), so that rows of
// zeros, and rows so small that no score reaches 2^-60, get a smaller ex; and
// kappa times 2^high stays finite, so that scores of 0 stay 0.
struct RowScale {
    int ex;
    float kappa;
};
template <int TOP, int SHIFT, int LOW, int HIGH>
__device__ __forceinline__ RowScale row_scale(float c, int c_exp, uint32_t most, bool live) {
    const int most_ex = c_exp + SHIFT + LOW + 125;
    int ex = live ? 127 + TOP - (int)(most >> 7) : -300;
    ex = ex < most_ex ? ex : most_ex;
    const int k = c_exp + SHIFT - ex;
    return RowScale{ex, ldexpf(c, k < 127 - HIGH ? k : 127 - HIGH)};
}

// A sequence as a kernel sees it, every value within its bounds.
struct Sequence {
    int first, n;   // its new tokens
    int len;        // its keys
};

__device__ __forceinline__ Sequence sequence_at(const CacheAttend &a, int64_t b) {
    Sequence s;
    if (a.q_offsets) {
        const int lo = a.q_offsets[b], hi = a.q_offsets[b + 1], T = (int)a.T;
        s.first = lo < 0 ? 0 : lo > T ? T : lo;
        const int end = hi < s.first ? s.first : hi > T ? T : hi;
        s.n = end - s.first;
    } else {
        s.first = (int)b;
        s.n = 1;
    }
    const int64_t most = a.table_pages * a.cache.page;
    const int len = a.lens[b];
    s.len = len < 0 ? 0 : len > most ? (int)most : len;
    return s;
}

// The same for a uniform b, by scalar loads.
__device__ __forceinline__ Sequence sequence_uniform(const CacheAttend &a, int64_t b) {
    Sequence s;
    s.first = (int)b;
    s.n = 1;
    const int T = (int)a.T;
    if (a.q_offsets) {
        const scalar_int *o = (const scalar_int *)a.q_offsets;
        const int lo = o[b], hi = o[b + 1];
        s.first = lo < 0 ? 0 : lo > T ? T : lo;
        s.n = (hi < s.first ? s.first : hi > T ? T : hi) - s.first;
    }
    const int64_t most = a.table_pages * a.cache.page;
    const int len = ((const scalar_int *)a.lens)[b];
    s.len = len < 0 ? 0 : len > most ? (int)most : len;
    return s;
}

// ---------------------------------------------------------------------------
// Few rows a sequence (single tokens, drafts): the split kernel.
//
// Bound by the bytes of the cache.  Rows of one key head go through the matrix
// cores together, 16 to a tile, so that a key is decoded once for all of them:
//   S^T = K Q^T  (16 keys x 16 rows, 32 dimensions a product), then
//   O^T = V^T P^T (16 dimensions x 16 rows, 32 keys a product).
// The scores of a lane (4 consecutive keys of a tile of 16, one row) are then
// the operand of the second product as they stand: no data moves between
// lanes.  V is turned by the transposing 4-bit LDS read.
//
// Decoding costs 7 operations for 8 codes: a code c in bits 4 to 7 of an fp16
// is the subnormal c 2^-20, which enters the product as it is.  (The matrix
// core aligns a subnormal by the smallest exponent and drops what lies 2^-24
// below the largest product: with the codes in bits 0 to 3, 5 operations, a
// sum of 32 was off by up to 2^-10.7 of a code at the largest weight, always
// down; in bits 4 to 7 by 2^-14.9, and 2^-16.4 for codes as normal numbers.)
// Zero points and scales stay outside: with Q_b the sum of a row's q over
// block b of 64 dimensions,
//   s = sum_b scale_b (sum_d q_d c_d - zero_b Q_b),
// and p' = p scale_b for the second product, whose zero points are
// subtracted at the end as the sum of p' zero_b.
// p' enters as fp16 (2^-11, random): scaled by 2^F so that a value scale of 2^E,
// times a weight of 1, is 2^9; when the maximum grows by less than 2^6 nothing is
// rescaled.  All value scales of a tile are from 2^(E - 10) to 2^E, so that what fp16
// loses of a weight (2^-25) is 2^-24 of the largest one with its own block's
// scale, whatever the other blocks' and keys' are, seen or not.  E moves up and
// down with them, and a tile whose scales are further apart is taken more than
// once: with E above all scales so far, values of scale 0.0015 beside others of
// 65504, seen or not, were off by 1.4e-3 of themselves and those of 2^-14 by 0.03,
// now by 2.6e-4.  (64 decode tokens over scales from 2^-20 to 1: 175 us, over
// scales within 2^10 75.)
//
// The work is the list of all tiles of 32 keys of all (sequence, key head),
// dealt evenly to a fixed number of waves, whatever the lengths: each finds its
// share from the lengths.  What a wave begins and does not end, or ends and did
// not begin, goes to the workspace, and a second launch joins the pieces in
// order (the same bits on every call).  64 tokens on up to 8192 ragged keys, 40
// + 8 heads of 128: 66 us, 4.2 TB/s, and 9 for the joining (a kernel trace;
// dealt by workgroups instead of waves 115 in all; a copy of the same bytes 64).  Vector
// instructions are under way for two thirds of the cycles, products for 0.11.
// ---------------------------------------------------------------------------

constexpr int kTile = 32;        // keys a wave takes at a time
constexpr int kSplitWaves = 4;
constexpr int kSplitThreads = 64 * kSplitWaves;
constexpr int kMinTiles = 2;       // tiles a wave should have at least, beside kBegin
// What beginning a piece costs a wave, in tiles: its tables, queries and first
// codes arrive one after the other (5 us where a further tile takes 0.85; 6
// units instead of 3 took 3 us more where waves have few tiles, and nothing
// less elsewhere).
constexpr int kBegin = 3;
constexpr int kHeadroom = 6;       // powers of two that weights may pass 1 by
constexpr int kSplitSpan = 10;     // powers of two that the value scales of a tile may lie within

// Tiles of one key head of a sequence (one at least where it has rows, so
// that rows without keys are written).  In the list that is dealt to the waves
// it has kBegin units and one for each tile.
__device__ __forceinline__ int tiles_of(const AttendArgs &g, const Sequence &s, int *lo_key) {
    const CacheAttend &a = g.a;
    int lo = 0;
    if (a.window > 0) {
        const int64_t l = (int64_t)s.len - s.n - a.window + 1;
        lo = l > 0 ? (int)(l < s.len ? l : s.len) & ~(kTile - 1) : 0;
    }
    *lo_key = lo;
    const int n = s.n < a.max_q ? s.n : (int)a.max_q;
    if (n <= 0 || (int64_t)n * g.G > g.limit) return 0;
    const int t = (s.len - lo + kTile - 1) / kTile;
    return t < 1 ? 1 : t;
}

// `total` tiles dealt to at most `waves` waves: the first `more` get each + 1,
// the others each.  (32-bit arithmetic where it holds: a 64-bit division is
// 100 scalar instructions.)
struct Shares {
    int64_t each, more, workers;
    __device__ __forceinline__ Shares(int64_t total, int waves) {
        workers = waves;
        if (total <= (int64_t)waves * (kBegin + kMinTiles)) workers = ((uint32_t)total + kBegin + kMinTiles - 1) / (kBegin + kMinTiles);
        each = (uint64_t)total >> 32 ? total / workers : (int64_t)((uint32_t)total / (uint32_t)workers);
        more = total - each * workers;
    }
    __device__ __forceinline__ int64_t start(int64_t w) const { return each * w + (w < more ? w : more); }
    // The wave that holds tile i.
    __device__ __forceinline__ int64_t at(int64_t i) const {
        const int64_t large = more * (each + 1);
        const int64_t x = i < large ? i : i - large, by = i < large ? each + 1 : each;
        const int64_t n = ((uint64_t)x | (uint64_t)by) >> 32 ? x / by : (int64_t)((uint32_t)x / (uint32_t)by);
        return i < large ? n : more + n;
    }
};

// Exclusive prefix sums of the sequences' counts by a workgroup of THREADS:
// found(b, before, count) for every sequence; the total.
template <int THREADS, class Count, class Found>
__device__ __forceinline__ int64_t scan_sequences(int64_t B, int64_t *sums, Count count, Found found) {
    const int tid = (int)threadIdx.x, wave = tid >> 6;
    int64_t before = 0;
    for (int64_t b0 = 0; b0 < B; b0 += THREADS) {
        const int64_t b = b0 + tid;
        const uint32_t t = b < B ? count(b) : 0;  // below 2^26
        uint32_t x = t;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const uint32_t y = __shfl_up(x, d);
            if ((tid & 63) >= d) x += y;
        }
        if ((tid & 63) == 63) sums[wave] = x;
        __syncthreads();
        int64_t off = before, all = 0;
        // (Unrolled, 8 waves' sums cost the tile kernel scalar registers, and one
        // vector register to spill them: D = 256 413 us instead of 363.)
#pragma unroll(THREADS > 256 ? 1 : THREADS / 64)
        for (int w = 0; w < THREADS / 64; ++w) {
            if (w < wave) off += sums[w];
            all += sums[w];
        }
        if (b < B) found(b, off + x - t, (int64_t)t);
        before += all;
        __syncthreads();
    }
    return before;
}

__device__ __forceinline__ float xor16(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, v), 0x401F));
}
__device__ __forceinline__ float sum4(float v) {  // over lanes l, l ^ 16, l ^ 32, l ^ 48
    v += xor16(v);
    return v + __shfl_xor(v, 32);
}
__device__ __forceinline__ float max4(float v) {
    v = fmaxf(v, xor16(v));
    return fmaxf(v, __shfl_xor(v, 32));
}

// The larger of two pairs of 16-bit integers.
__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2_t, a), __builtin_bit_cast(u16x2_t, b)));
}
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}
// Each of two 16-bit integers less that of b, and 0 where it is 0.
__device__ __forceinline__ uint32_t pk_sub_but_0(uint32_t a, uint32_t b) {
    const u16x2_t x = __builtin_bit_cast(u16x2_t, a), one = {1, 1};
    return __builtin_bit_cast(uint32_t, (u16x2_t)(x - __builtin_elementwise_min(x, one) * __builtin_bit_cast(u16x2_t, b)));
}
__device__ __forceinline__ uint32_t half_max(uint32_t v) { return (v >> 16) > (v & 0xFFFF) ? v >> 16 : v & 0xFFFF; }
// The larger of pairs of 16-bit integers over the wave.
__device__ __forceinline__ uint32_t wave_pk_max(uint32_t v) {
    v = pk_max(v, dpp_u32<kDppQuadXor1>(v));
    v = pk_max(v, dpp_u32<kDppQuadXor2>(v));
    v = pk_max(v, dpp_u32<kDppRowHalfMirror>(v));
    v = pk_max(v, dpp_u32<kDppRowMirror>(v));
    v = pk_max(v, (uint32_t)__builtin_amdgcn_ds_swizzle((int)v, 0x401F));
    return (uint32_t)__builtin_amdgcn_readfirstlane((int)pk_max(v, (uint32_t)__shfl_xor((int)v, 32)));
}
// The largest 16-bit integer over lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ uint32_t half_max4(uint32_t v) {
    v = pk_max(v, (uint32_t)__builtin_amdgcn_ds_swizzle((int)v, 0x401F));
    return half_max(pk_max(v, (uint32_t)__shfl_xor((int)v, 32)));
}

// 8 codes as 8 fp16 subnormals c 2^-20, in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ half8_t subnormals(uint32_t w) {
    constexpr uint32_t kMask = 0x00F000F0u;
    u32x4_t r;
    r[0] = (w << 4) & kMask;
    r[1] = w & kMask;
    r[2] = (w >> 4) & kMask;
    r[3] = (w >> 8) & kMask;
    return __builtin_bit_cast(half8_t, r);
}

__device__ __forceinline__ float half_at(const uint32_t *w, int i) {
    const uint32_t u = w[i >> 1];
    return (float)__builtin_bit_cast(_Float16, (unsigned short)(i & 1 ? u >> 16 : u));
}

// Stores 4 outputs.
__device__ __forceinline__ void store4(const CacheAttend &a, int64_t at, float4_t v) {
    if (a.bf16) {
        typedef __bf16 bf4 __attribute__((ext_vector_type(4)));
        const bf4 b = {(__bf16)v.x, (__bf16)v.y, (__bf16)v.z, (__bf16)v.w};
        *reinterpret_cast<bf4 *>(static_cast<uint16_t *>(a.out) + at) = b;
    } else {
        *reinterpret_cast<float4_t *>(static_cast<float *>(a.out) + at) = v;
    }
}

// What a wave has asked for of a tile of 32 keys.
template <int ND>
struct Tile {
    u32x2_t k[2][ND];   // 16 codes of the lane's key (of 16) and block
    u32x4_t v[ND];      // 16 bytes of the values' codes, as they lie
    uint32_t par[ND];   // scales and zeros: [plane][half of the tile][key][block], dealt a dword a lane
};

// Orders a wave's own LDS accesses for the compiler (the hardware keeps them
// in order).
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Reads scales or zeros of the lane's 4 keys of half t of the tile: ND halves a key.
enum { kKeyScales, kKeyZeros, kValueScales, kValueZeros };
template <int ND>
__device__ __forceinline__ void read_par(const uint32_t *lds, int plane, int t, int grp, uint32_t (&out)[2 * ND]) {
    const u32x2_t *p = reinterpret_cast<const u32x2_t *>(lds + (plane * 2 + t) * 8 * ND + grp * 2 * ND);
#pragma unroll
    for (int i = 0; i < ND; ++i) {
        const u32x2_t v = p[i];
        out[2 * i] = v.x;
        out[2 * i + 1] = v.y;
    }
}

// The exponent e with a finite fp16 of these bits below 2^e.
__device__ __forceinline__ int exponent_above(uint32_t bits) {
    return bits == 0 ? -24 : bits < 0x400u ? -14 : (int)(bits >> 10) - 14;
}
// The exponent e with a finite fp16 of these bits (not 0) at 2^e or above.
__device__ __forceinline__ int exponent_of(uint32_t bits) {
    return bits < 0x400u ? 7 - __builtin_clz(bits) : (int)(bits >> 10) - 15;
}

// Scales from 2^(e - SPAN) to 2^e, and 0, are within exponent e (-24: only 0).
// The bits of the smallest, and of the one past the largest.
template <int SPAN>
__device__ __forceinline__ uint32_t from(int e) {
    const int f = e - SPAN;
    return f <= -24 ? 1 : f < -14 ? 1u << (f + 24) : (uint32_t)(f + 15) << 10;
}
__device__ __forceinline__ uint32_t past(int e) { return e < -14 ? 1 : (uint32_t)(e + 15) << 10; }
template <int SPAN>
__device__ __forceinline__ bool outside(uint32_t bits, int e) {
    return bits != 0 && bits - from<SPAN>(e) >= past(e) - from<SPAN>(e);
}

// The exponent that scales from `least` to `top` (bits; 0: none) are within, in
// the middle, so that larger and smaller ones later on are too; false, and
// that of the largest, where there is none.
template <int SPAN>
__device__ __forceinline__ bool fit(uint32_t top, uint32_t least, int *e) {
    const int lo = exponent_above(top), hi = top == 0 ? lo : SPAN + exponent_of(least);
    const int mid = lo + (hi > lo ? (hi - lo + 1) / 2 : 0);
    *e = mid < 16 ? mid : 16;
    return lo <= hi;
}

// Workgroups a compute unit: what the registers allow.
constexpr int split_occupancy(int ND, int NT) { return NT * ND <= 2 ? 3 : NT * ND <= 4 ? 2 : 1; }

template <int ND, int NT, bool DIRECT>
struct SplitShared {
    struct In {
        uint8_t v[kSplitWaves][kTile * ND * 32];
        uint32_t par[kSplitWaves][64 * ND];
        float kept[kSplitWaves][2 * NT][64];
    };
    struct Out {  // of the waves that share a (sequence, key head)
        float o[kSplitWaves][16][ND * 64 + 4];
        float ref[kSplitWaves][16], sum[kSplitWaves][16];
    };
    struct None {};
    union {
        In in;
        std::conditional_t<DIRECT, Out, None> out;
    };
    int64_t sums[kSplitWaves];
    int64_t start_b[kSplitWaves], start_at[kSplitWaves];
};

template <int ND, int NT, bool DIRECT>
__global__ __launch_bounds__(kSplitThreads, split_occupancy(ND, NT)) void attend_split_kernel(AttendArgs g) {
    constexpr int D = ND * 64;
    __shared__ __attribute__((aligned(16))) SplitShared<ND, NT, DIRECT> sh;
    const CacheAttend &a = g.a;
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, grp = lane >> 4;
    const int heads = (int)a.cache.heads, page = (int)a.cache.page, pages = (int)a.cache.pages;

    int64_t w = DIRECT ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * kSplitWaves + wave;
    int64_t begin = 0, end = 1, b, at = 0;  // the wave's share; tiles before sequence b
    int64_t one_b = 0, one_at = 0, one_t = 0, total = 0;
    Shares shares(1, 1);
    if (DIRECT) {
        // A workgroup per sequence and key head: its waves take tiles in turn.
        b = w / heads;
    } else {
        auto count = [&](int64_t x) {
            int lo;
            const int t = tiles_of(g, sequence_at(a, x), &lo);
            return t > 0 ? (uint32_t)t + kBegin : 0u;
        };
        total = heads * scan_sequences<kSplitThreads>(
                            a.B, sh.sums, count, [&](int64_t x, int64_t before, int64_t t) { one_b = x; one_at = before; one_t = t; });
        if (total == 0) return;
        shares = Shares(total, g.waves);
        auto place = [&](int64_t x, int64_t before, int64_t t) {
#pragma unroll
            for (int y = 0; y < kSplitWaves; ++y) {
                const int64_t i = shares.start((int64_t)blockIdx.x * kSplitWaves + y);
                if (i >= before * heads && i < (before + t) * heads) {
                    sh.start_b[y] = x;
                    sh.start_at[y] = before * heads;
                }
            }
        };
        if (a.B <= kSplitThreads) {  // what the scan left with each thread
            place(one_b, one_at, one_t);
            __syncthreads();
        } else {
            scan_sequences<kSplitThreads>(a.B, sh.sums, count, place);
        }
        // From here on the waves go their own ways.
        if (w >= shares.workers) return;
        begin = shares.start(w);
        end = shares.start(w + 1);
        b = uniform64(sh.start_b[wave]);
        at = uniform64(sh.start_at[wave]);
    }

    int64_t i = begin;
    while (i < end) {
        const Sequence s = sequence_uniform(a, b);
        int lo_key;
        const int nt = tiles_of(g, s, &lo_key);
        if (DIRECT) {
            if (nt == 0) return;
        } else if (nt == 0 || i >= at + (int64_t)(nt + kBegin) * heads) {
            if (nt > 0) at += (int64_t)(nt + kBegin) * heads;
            ++b;
            continue;
        }
        int h, t0 = 0, t1 = nt;
        int64_t row_start = 0;
        if (DIRECT) {
            h = (int)(w % heads);
        } else {
            const int64_t ahead = i - at;
            const int units = nt + kBegin;
            h = (int)((uint64_t)ahead >> 32 ? ahead / units : (int64_t)((uint32_t)ahead / (uint32_t)units));
            row_start = at + (int64_t)h * units;
            t0 = (int)(i - row_start) - kBegin;
            t1 = (int)(end - row_start < units ? end - row_start : units) - kBegin;
            i = row_start + t1 + kBegin;
            if (t1 <= 0) continue;
            if (t0 < 0) t0 = 0;
        }
        const int n = s.n < a.max_q ? s.n : (int)a.max_q;
        const int rows = n * g.G;

        // Scalar loads: a vector load here would wait for the codes on the way.
        const scalar_int *table = (const scalar_int *)(a.table + b * a.table_pages);
        const int last_page = (s.len - 1) >> g.page_shift;
        auto entry = [&](int key) -> int {
            const int p = key >> g.page_shift;
            return table[p < last_page ? p : last_page];
        };
        // Whether the lane's d-th dword of the scales and zeros is of values' scales.
        auto has_scales = [&](int d) {
            return 64 * d < 48 * ND && 64 * d + 63 >= 32 * ND && (lane + 64 * d) / (16 * ND) == kValueScales;
        };
        // Where the lane's dwords of the scales and zeros lie.
        const uint32_t *par_base[ND];
        bool par_second[ND];
#pragma unroll
        for (int d = 0; d < ND; ++d) {
            const int c = lane + 64 * d, plane = c / (16 * ND), in = c - plane * 16 * ND;
            const uint16_t *pp = plane == 0 ? a.cache.k_scales : plane == 1 ? a.cache.k_zeros : plane == 2 ? a.cache.v_scales : a.cache.v_zeros;
            par_second[d] = in >= 8 * ND;
            par_base[d] = reinterpret_cast<const uint32_t *>(pp) + (in >= 8 * ND ? in - 8 * ND : in);
        }
        auto rows_of = [&](int tile, int id0, int id1, int64_t (&row)[2]) {
            const int key = lo_key + tile * kTile;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const int id = t ? id1 : id0;
                row[t] = ((int64_t)((uint32_t)id < (uint32_t)pages ? id : 0) * heads + h) * page + ((key + 16 * t) & (page - 1));
            }
        };
        auto load_keys = [&](const int64_t (&row)[2], Tile<ND> &T) {
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const uint8_t *kc = a.cache.k_codes + row[t] * (D / 2) + (col * (D / 2) + 8 * grp);
#pragma unroll
                for (int d = 0; d < ND; ++d) T.k[t][d] = *reinterpret_cast<const u32x2_t *>(kc + 32 * d);
            }
        };
        auto load_values = [&](const int64_t (&row)[2], Tile<ND> &T) {
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const int c = lane + 64 * d;
                const bool t = c >= 32 * ND;
                T.v[d] = *reinterpret_cast<const u32x4_t *>(a.cache.v_codes + (t ? row[1] : row[0]) * (D / 2) +
                                                            (t ? c - 32 * ND : c) * 16);
                T.par[d] = par_base[d][(par_second[d] ? row[1] : row[0]) * ND / 2];
            }
        };

        // The loads of the next tile are made in the last round too (of the
        // same tile), so that no wait has to hold for both cases.
        const int tend = s.len > 0 ? t1 : t0;
        constexpr int kStep = DIRECT ? kSplitWaves : 1;
        int tile = t0 + (DIRECT ? wave : 0);
        Tile<ND> T;
        int id0 = -1, id1 = -1, next0 = -1, next1 = -1;  // table entries of this tile and the next
        int64_t row[2];
        uint32_t *const par = sh.in.par[wave];
        auto later = [&](int by) { return tile + by * kStep < tend ? tile + by * kStep : tile; };
        if (tile < tend) {
            id0 = entry(lo_key + tile * kTile);
            id1 = entry(lo_key + tile * kTile + 16);
            next0 = entry(lo_key + later(1) * kTile);
            next1 = entry(lo_key + later(1) * kTile + 16);
            rows_of(tile, id0, id1, row);
            load_values(row, T);
            load_keys(row, T);
        }
        // Queries: the lane's row of each tile of 16, its 8 dimensions of every 32.
        half8_t qf[NT][ND][2];
        float qsum[NT][ND], kappa[NT];
        int seen_to[NT], seen_from[NT];  // keys seen by the lane's row
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            const int r = 16 * x + col;
            const int j = r < rows ? (int)(r * g.inv_G >> 16) : 0, hq = h * g.G + (r < rows ? r - j * g.G : 0);
            const uint16_t *q = a.q + (int64_t)(s.first + j) * a.q_stride + (hq * D + 16 * grp);
            u32x4_t raw[ND][2];
            uint32_t most = 0;  // of the magnitudes' bits
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    raw[d][e] = *reinterpret_cast<const u32x4_t *>(q + 64 * d + 8 * e);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t p = raw[d][e][y];
                        most = pk_max(most, p & 0x7FFF7FFFu);
                    }
                }
            // The row's largest to 2^14 .. 2^15 (a row with an infinity has no
            // finite result, whatever its other values become).
            const RowScale rs = row_scale<14, 20, 0, 0>(g.c, g.c_exp, half_max4(most), r < rows);
            const int ex = rs.ex;
            kappa[x] = rs.kappa;
            const uint32_t one = 0x00100010u;  // the code 1, twice
            const half8_t ones = __builtin_bit_cast(half8_t, u32x4_t{one, one, one, one});
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                float4_t sum = {0, 0, 0, 0};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    half8_t f;
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        // Codes come in the order 0 4 1 5 2 6 3 7.
                        const uint32_t p = raw[d][e][y];
                        const int to0 = 2 * y < 4 ? 4 * y : 4 * y - 7, to1 = to0 + 2;
                        f[to0] = (_Float16)ldexpf(__builtin_bit_cast(float, p << 16), ex);
                        f[to1] = (_Float16)ldexpf(__builtin_bit_cast(float, p & 0xFFFF0000u), ex);
                    }
                    qf[x][d][e] = f;
                    sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(ones, f, sum, 0, 0, 0);
                }
                qsum[x][d] = sum[0];
            }
            const int pos = s.len - s.n + j;
            seen_to[x] = r < rows ? (a.causal ? pos : s.len - 1) : -1;
            seen_from[x] = a.window > 0 ? pos - (int)a.window + 1 : 0;
        }
        // The first key that some row sees, and keys that all rows see: tiles
        // within need no mask.
        const int64_t low = a.window > 0 ? (int64_t)s.len - s.n - a.window + 1 : 0;
        const int low_key = low > 0 ? (int)(low < s.len ? low : s.len) : 0;
        const int all_to = a.causal ? s.len - s.n : s.len - 1;
        const int64_t all_from = a.window > 0 ? (int64_t)s.len - s.n + (n - 1) - a.window + 1 : 0;

        float m[NT], l[NT], nk[NT], ck[NT], zs[NT][ND];
        float4_t o[NT][ND][4];
        // The value scales of a tile are within E: two of them less low2 are at
        // most span2.  (Begun with 0, which holds for values of common sizes.)
        int E = 0;
        uint32_t low2 = from<kSplitSpan>(0) * 0x10001u, span2 = (past(0) - 1 - from<kSplitSpan>(0)) * 0x10001u;
        uint32_t cut = 0x7C00u;        // a tile that is taken again: scales from here on have been
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            m[x] = -INFINITY;
            l[x] = 0;
            nk[x] = (float)(9 - E);
            ck[x] = INFINITY;
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                zs[x][d] = 0;
#pragma unroll
                for (int y = 0; y < 4; ++y) o[x][d][y] = float4_t{0, 0, 0, 0};
            }
        }

        for (int step = 0; tile < tend; tile += step) {
            const bool ok[2] = {(uint32_t)id0 < (uint32_t)pages && lo_key + tile * kTile < s.len,
                                (uint32_t)id1 < (uint32_t)pages && lo_key + tile * kTile + 16 < s.len};
            const int key = lo_key + tile * kTile;
            const bool edge = !ok[0] || !ok[1] || key + kTile > s.len || key < low_key;
            if (__builtin_expect(edge, 0)) {
                // Keys that no row sees may hold anything: scales and zeros of 0.
                asm volatile("");  // (a branch, not selects)
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    const int c = lane + 64 * d, in = c % (16 * ND), t = in >= 8 * ND, y = 2 * (in - t * 8 * ND);
                    const bool page_ok = t ? ok[1] : ok[0];
                    const int k0 = key + 16 * t + y / ND, k1 = key + 16 * t + (y + 1) / ND;
                    if (!page_ok || k0 >= s.len || k0 < low_key) T.par[d] &= 0xFFFF0000u;
                    if (!page_ok || k1 >= s.len || k1 < low_key) T.par[d] &= 0x0000FFFFu;
                }
            }
            // Value scales that are not within E (0 is: blocks of padded heads).
            bool odd = false;
#pragma unroll
            for (int d = 0; d < ND; ++d) odd = odd || (has_scales(d) && pk_max(pk_sub_but_0(T.par[d], low2), span2) != span2);
            const bool repeated = cut < 0x7C00u;
            bool again = false, grown = false;
            int next_E = E;
            if (__any(odd) || repeated) {
                asm volatile("");  // (a branch, not selects)
                uint32_t top = 0, low = 0;  // the largest of those that are left, 0x7C00 less the smallest
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int i = 0; i < 32; i += 16) {
                        const uint32_t v = has_scales(d) ? (T.par[d] >> i) & 0xFFFF : 0;
                        top = v < cut && v > top ? v : top;
                        low = v > 0 && v < cut && 0x7C00u - v > low ? 0x7C00u - v : low;
                        grown = grown || (v >= 0x7C00u && !repeated);
                    }
                top = wave_pk_max(top << 16 | low);
                low = 0x7C00u - (top & 0xFFFF);
                top >>= 16;
                if (top > 0 && (outside<kSplitSpan>(top, E) || outside<kSplitSpan>(low, E))) again = !fit<kSplitSpan>(top, low, &next_E);
                grown = grown || next_E != E;
                if (again || repeated) {
                    // No exponent holds for the tile: it is taken once for each
                    // that it needs, the largest first, with other scales 0.
                    const uint32_t lo = from<kSplitSpan>(next_E), hi = past(next_E) < cut ? past(next_E) : cut;
#pragma unroll
                    for (int d = 0; d < ND; ++d)
#pragma unroll
                        for (int i = 0; i < 32; i += 16) {
                            const uint32_t v = (T.par[d] >> i) & 0xFFFF;
                            if (has_scales(d) && !(v >= lo && v < hi) && (repeated || v < 0x7C00u)) T.par[d] &= ~(0xFFFFu << i);
                        }
                    if (repeated) {  // its weights are summed already
#pragma unroll
                        for (int x = 0; x < NT; ++x) {
                            sh.in.kept[wave][2 * x][lane] = l[x];
                            sh.in.kept[wave][2 * x + 1][lane] = nk[x];
                        }
                    }
                }
                cut = again ? from<kSplitSpan>(next_E) : 0x7C00u;
            }
            uint8_t *vl = sh.in.v[wave];
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                *reinterpret_cast<u32x4_t *>(vl + (lane + 64 * d) * 16) = T.v[d];
                par[lane + 64 * d] = T.par[d];
            }
            wave_fence();
            if (!again) {
                id0 = next0;
                id1 = next1;
            }
            const int to = again ? tile : later(1), then = again ? later(1) : later(2);
            rows_of(to, id0, id1, row);
            load_values(row, T);
            next0 = entry(lo_key + then * kTile);
            next1 = entry(lo_key + then * kTile + 16);

            // Scores.
            float S[NT][2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t ks[2 * ND], kz[2 * ND];
                read_par<ND>(par, kKeyScales, t, grp, ks);
                read_par<ND>(par, kKeyZeros, t, grp, kz);
#pragma unroll
                for (int d = 0; d < ND; ++d) {
                    const half8_t k0 = subnormals(T.k[t][d].x), k1 = subnormals(T.k[t][d].y);
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        float4_t acc = {0, 0, 0, 0};
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(k0, qf[x][d][0], acc, 0, 0, 0);
                        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(k1, qf[x][d][1], acc, 0, 0, 0);
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float u = fmaf(-half_at(kz, r * ND + d), qsum[x][d], acc[r]);
                            S[x][t][r] = d == 0 ? half_at(ks, r * ND) * u
                                                : fmaf(half_at(ks, r * ND + d), u, S[x][t][r]);
                        }
                    }
                }
            }
            load_keys(row, T);
            step = again ? 0 : kStep;
            const bool masked = key + kTile - 1 > all_to || key < all_from || !ok[0] || !ok[1];
            if (__builtin_expect(masked, 0)) {
                asm volatile("");  // (a branch, not selects)
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int k = key + 16 * t + 4 * grp + r;
#pragma unroll
                        for (int x = 0; x < NT; ++x)
                            if (!ok[t] || k > seen_to[x] || k < seen_from[x]) S[x][t][r] = -INFINITY;
                    }
            }
            // Whether a maximum has grown too far.
            float tmax[NT];
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                tmax[x] = fmaxf(fmaxf(fmaxf(S[x][0][0], S[x][0][1]), fmaxf(S[x][0][2], S[x][0][3])),
                                fmaxf(fmaxf(S[x][1][0], S[x][1][1]), fmaxf(S[x][1][2], S[x][1][3])));
                grown = grown || fmaf(tmax[x], kappa[x], ck[x]) > (float)(9 - E + kHeadroom);
            }
            if (__any(grown)) {
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    uint32_t vs[2 * ND];
                    read_par<ND>(par, kValueScales, t, grp, vs);
#pragma unroll
                    for (int y = 0; y < 4 * ND; ++y) {
                        const uint32_t v = (vs[y >> 1] >> (16 * (y & 1))) & 0xFFFF;
                        // A scale that is not finite makes the block NaN in the
                        // rows that see the key, and does not reach the others.
                        if (v >= 0x7C00u) {
                            uint16_t *at = reinterpret_cast<uint16_t *>(par + (kValueScales * 2 + t) * 8 * ND + grp * 2 * ND) + y;
                            at[0] = 0;
                            at[2 * 16 * ND] = 0;  // its zero, a plane further
#pragma unroll
                            for (int x = 0; x < NT; ++x)
                                if (S[x][t][y / ND] != -INFINITY) zs[x][y % ND] = NAN;
                        }
                    }
                }
                wave_fence();
                if (next_E != E) {
                    E = next_E;
                    low2 = from<kSplitSpan>(E) * 0x10001u;
                    span2 = (past(E) - 1 - from<kSplitSpan>(E)) * 0x10001u;
                }
                const float F = (float)(9 - E);
#pragma unroll
                for (int x = 0; x < NT; ++x) {
                    const float mn = fmaxf(m[x], max4(tmax[x]));
                    const float kn = mn == -INFINITY ? F : fmaf(-mn, kappa[x], F);
                    const float fade = m[x] == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(kn - nk[x]);
                    m[x] = mn;
                    nk[x] = kn;
                    ck[x] = mn == -INFINITY ? INFINITY : kn;
                    l[x] *= fade;
#pragma unroll
                    for (int d = 0; d < ND; ++d) {
                        zs[x][d] *= fade;
#pragma unroll
                        for (int y = 0; y < 4; ++y) o[x][d][y] *= fade;
                    }
                }
            }
            // Weights, and the operands of the second product.
            half8_t pf[NT][ND];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint32_t vs[2 * ND], vz[2 * ND];
                read_par<ND>(par, kValueScales, t, grp, vs);
                read_par<ND>(par, kValueZeros, t, grp, vz);
#pragma unroll
                for (int x = 0; x < NT; ++x)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const float p = __builtin_amdgcn_exp2f(fmaf(S[x][t][r], kappa[x], nk[x]));
                        l[x] += p;
#pragma unroll
                        for (int d = 0; d < ND; ++d) {
                            const _Float16 w16 = (_Float16)(p * half_at(vs, r * ND + d));
                            pf[x][d][2 * r + t] = w16;
                            zs[x][d] = fmaf((float)w16, half_at(vz, r * ND + d), zs[x][d]);
                        }
                    }
            }
            // Values: each group of 16 lanes turns its 8 keys (4 of each 16) by 32 dimensions.
            const int vkey = ((lane & 7) < 4 ? 0 : 16) + 4 * grp + (lane & 3);
            const uint8_t *vr = vl + vkey * (D / 2) + ((lane >> 3) & 1) * 8;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int2_t u = __builtin_amdgcn_ds_read_tr4_b64_v2i32(
                        (__attribute__((address_space(3))) int2_t *)(vr + 32 * d + 16 * y));
                    const half8_t v0 = subnormals((uint32_t)u.x), v1 = subnormals((uint32_t)u.y);
#pragma unroll
                    for (int x = 0; x < NT; ++x) {
                        o[x][d][2 * y] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v0, pf[x][d], o[x][d][2 * y], 0, 0, 0);
                        o[x][d][2 * y + 1] = __builtin_amdgcn_mfma_f32_16x16x32_f16(v1, pf[x][d], o[x][d][2 * y + 1], 0, 0, 0);
                    }
                }
            if (repeated) {
#pragma unroll
                for (int x = 0; x < NT; ++x)
                    l[x] = sh.in.kept[wave][2 * x][lane] * __builtin_amdgcn_exp2f(nk[x] - sh.in.kept[wave][2 * x + 1][lane]);
            }
        }

        // Results, 16 rows at a time.  A row's weights stand relative to 2^ref.
        const bool whole = t0 == 0 && t1 == nt;
        if (!DIRECT && t1 == nt && lane == 0) {
            g.pieces[b * heads + h] = Pieces{(int)(whole ? w : shares.at(row_start + kBegin)), (int)w};
        }
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            if (16 * x >= rows) break;
            float sum = sum4(l[x]), ref = -nk[x], z[ND];
#pragma unroll
            for (int d = 0; d < ND; ++d) z[d] = sum4(zs[x][d]);
            const int r = 16 * x + col, j = (int)(r * g.inv_G >> 16);
            const int64_t at_row = (int64_t)(s.first + j) * a.q_heads + (h * g.G + r - j * g.G);
            if constexpr (!DIRECT) {
                if (r >= rows) continue;
                const int64_t at_part = (2 * w + (t0 == 0 ? 1 : 0)) * g.max_rows + r;
                const float f = !whole ? 1.0f : sum == 0 ? 0.0f : 1.0f / sum;
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        float4_t v;
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = whole && sum == 0 ? 0.0f : fmaf(o[x][d][y][e], 0x1p20f, -z[d]) * f;
                        const int at_d = 64 * d + 16 * y + 4 * grp;
                        if (whole) store4(a, at_row * D + at_d, v);
                        else *reinterpret_cast<float4_t *>(g.part + at_part * D + at_d) = v;
                    }
                if (grp == 0) {
                    if (!whole) *reinterpret_cast<float2 *>(g.part_sums + at_part * 2) = make_float2(ref, sum);
                    else if (a.lse)
                        a.lse[at_row] = sum == 0 ? -INFINITY : (ref + __builtin_amdgcn_logf(sum)) * 0.693147180559945f;
                }
            } else {
                __syncthreads();
                if (grp == 0) {
                    sh.out.ref[wave][col] = ref;
                    sh.out.sum[wave][col] = sum;
                }
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        float4_t v;
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[e] = fmaf(o[x][d][y][e], 0x1p20f, -z[d]);
                        *reinterpret_cast<float4_t *>(&sh.out.o[wave][col][64 * d + 16 * y + 4 * grp]) = v;
                    }
                __syncthreads();
                for (int e = tid; e < 16 * D / 4; e += kSplitThreads) {
                    const int c = e / (D / 4), d = e % (D / 4) * 4, rr = 16 * x + c;
                    if (rr >= rows) break;
                    float top = -INFINITY;
#pragma unroll
                    for (int y = 0; y < kSplitWaves; ++y)
                        if (sh.out.sum[y][c] != 0) top = fmaxf(top, sh.out.ref[y][c]);
                    float lt = 0;
                    float4_t ot = {0, 0, 0, 0};
#pragma unroll
                    for (int y = 0; y < kSplitWaves; ++y) {
                        const float part = sh.out.sum[y][c];
                        const float4_t v = *reinterpret_cast<const float4_t *>(&sh.out.o[y][c][d]);
                        if (part != 0) {
                            const float f = __builtin_amdgcn_exp2f(sh.out.ref[y][c] - top);
                            lt = fmaf(f, part, lt);
#pragma unroll
                            for (int q = 0; q < 4; ++q) ot[q] = fmaf(f, v[q], ot[q]);
                        }
                    }
                    const int jj = (int)(rr * g.inv_G >> 16);
                    const int64_t to = (int64_t)(s.first + jj) * a.q_heads + (h * g.G + rr - jj * g.G);
                    const float f = lt == 0 ? 0.0f : 1.0f / lt;
#pragma unroll
                    for (int q = 0; q < 4; ++q) ot[q] = lt == 0 ? 0.0f : ot[q] * f;
                    store4(a, to * D + d, ot);
                    if (a.lse && d == 0) a.lse[to] = lt == 0 ? -INFINITY : (top + __builtin_amdgcn_logf(lt)) * 0.693147180559945f;
                }
            }
        }
        if (DIRECT) return;
    }
}

// Joins the pieces of a (sequence, key head): a workgroup per row and block of
// 64 dimensions, 16 lanes a piece, the pieces dealt to 16 groups of lanes.
// Bound by its launch and three loads one after the other: 4.5 us where there
// is nothing to join, 7 to 9 for 64 sequences of 8 heads.
__global__ __launch_bounds__(256) void attend_join_kernel(AttendArgs g) {
    constexpr int kLanes = 16, kGroups = 16;
    __shared__ float4_t so[kGroups][kLanes];
    __shared__ float ss[kGroups];
    const CacheAttend &a = g.a;
    const int r = (int)blockIdx.y, tid = (int)threadIdx.x, heads = (int)a.cache.heads, D = (int)a.cache.D;
    const int64_t b = blockIdx.x / heads;
    const int h = (int)(blockIdx.x - b * heads);
    const Sequence s = sequence_uniform(a, b);
    int lo_key;
    const int n = s.n < a.max_q ? s.n : (int)a.max_q;
    if (tiles_of(g, s, &lo_key) == 0 || r >= n * g.G) return;
    const Pieces e = g.pieces[blockIdx.x];
    if (e.first == e.last) return;
    const int pieces = e.last - e.first + 1;
    const float2 *sums = reinterpret_cast<const float2 *>(g.part_sums) + r;
    auto slot = [&](int p) { return (int64_t)(2 * (e.first + p) + (p == 0 ? 1 : 0)) * g.max_rows; };
    float top = -INFINITY;
    for (int p = tid & 63; p < pieces; p += 64) {
        const float2 q = sums[slot(p)];
        if (q.y != 0) top = fmaxf(top, q.x);
    }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
    const int c = tid % kLanes, gr = tid / kLanes, d = (int)blockIdx.z * 64 + 4 * c;
    float4_t ot = {0, 0, 0, 0};
    float lt = 0;
    const float *part = g.part + (int64_t)r * D + d;
#pragma unroll 4
    for (int p = gr; p < pieces; p += kGroups) {
        const int64_t x = slot(p);
        const float2 q = sums[x];
        const float4_t v = *reinterpret_cast<const float4_t *>(part + x * D);
        const bool any = q.y != 0;
        const float f = any ? __builtin_amdgcn_exp2f(q.x - top) : 0.0f;
        lt = any ? fmaf(f, q.y, lt) : lt;
#pragma unroll
        for (int i = 0; i < 4; ++i) ot[i] = any ? fmaf(f, v[i], ot[i]) : ot[i];
    }
    so[gr][c] = ot;
    if (c == 0) ss[gr] = lt;
    __syncthreads();
    if (tid >= kLanes) return;
#pragma unroll
    for (int p = 1; p < kGroups; ++p) {
        lt += ss[p];
        const float4_t v = so[p][c];
        ot += v;
    }
    const int j = (int)(r * g.inv_G >> 16);
    const int64_t at = (int64_t)(s.first + j) * a.q_heads + (h * g.G + r - j * g.G);
    float4_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = lt == 0 ? 0.0f : ot[i] / lt;
    store4(a, at * D + d, v);
    if (a.lse && d == 0) a.lse[at] = lt == 0 ? -INFINITY : (top + __builtin_amdgcn_logf(lt)) * 0.693147180559945f;
}

// ---------------------------------------------------------------------------
// Many rows a sequence (prompts and chunks of them): the tile kernel.
//
// Bound by the matrix cores and the exponentials.  A workgroup of 8 waves takes
// 256 rows of one key head (32 a wave) and walks the keys 64 at a time: they
// are decoded once, by all waves, into LDS as fp16, one buffer ahead of the one
// in use, so that a tile costs one barrier.  32 x 32 x 16 products: S^T = K Q^T,
// whose result is the operand of O^T = V^T P^T as it stands; V is turned by the
// transposing 16-bit LDS read.
// They become (c - zero) scale 2^-E, with 2^E for keys and one for values such
// that all scales are from 2^(E - 14) to 2^E: normal numbers in fp16, each rounded
// by 2^-11 of itself, whatever the largest scale of the tile is and whoever
// sees it (with 2^E above the largest scale alone, values of scale 0.0015 beside
// others of 65504, seen or not, were off by 0.8 of themselves, now by 3e-4).
// The sum of a row's weights is that of the fp32 weights: with the sum of the
// rounded ones, one instruction for two of them, lse was off by up to 2^-11.
//
// Where the rows are few for the card, the keys of a tile of rows are dealt to
// several workgroups, whose results a second launch joins.
// 512 tokens behind 32488, 40 + 8 heads of 128: 393 to 397 us, 865 TFLOP/s (a
// large library product makes 1153); prompts of 8191 tokens, 16 + 2 heads, 171 to
// 175, of which 9 are the kernels of few rows (calls in a replayed graph).  A
// tile of 64 keys cost about 5000 cycles while it told of its largest scales (3 in
// 100 more than now): QK 1190, PV 770, decoding 1230, maximum and softmax 1040,
// barrier and exponents 950, overlapped only in part by the two waves of a
// SIMD.  256 rows: with 128 the decoding would weigh twice.
// ---------------------------------------------------------------------------

constexpr int kRowTile = 256;
constexpr int kTileWaves = 8;
constexpr int kTileThreads = 64 * kTileWaves;
constexpr int kKeyTile = 64;     // keys that parts are counted in
constexpr int kMinKeyTiles = 8;  // tiles of keys a part should have
constexpr float kTop = 9;        // a weight of 1 is 2^9

struct RowTile {
    int64_t b;
    Sequence s;
    int row0, rows;   // first row, rows of the sequence
    int low, hi;      // keys that some row of the tile sees: low .. hi - 1
    int lo;           // low, down to a multiple of 64
    int parts;        // workgroups its keys are dealt to
};

__device__ __forceinline__ int row_tiles_of(const AttendArgs &g, const Sequence &s, int64_t *rows) {
    const int n = s.n < g.a.max_q ? s.n : (int)g.a.max_q;
    *rows = (int64_t)n * g.G;
    return n <= 0 || *rows <= g.limit ? 0 : (int)((*rows + kRowTile - 1) / kRowTile);
}

// The index-th tile of rows; false past the last.
template <int THREADS>
__device__ __forceinline__ bool find_row_tile(const AttendArgs &g, int64_t index, int64_t *sums, int64_t *found,
                                              int *longest, RowTile &r) {
    const CacheAttend &a = g.a;
    if (threadIdx.x == 0) {
        found[0] = -1;
        longest[0] = longest[1] = 0;
    }
    int most_keys = 0, most_before = 0;  // of the thread's sequences: keys that a tile of rows sees, and those before the new
    scan_sequences<THREADS>(
        a.B, sums,
        [&](int64_t b) {
            int64_t rows;
            const Sequence s = sequence_at(a, b);
            const uint32_t t = (uint32_t)row_tiles_of(g, s, &rows);
            if (t > 0) {
                const int seen = a.window > 0 ? (int)a.window + kRowTile / g.G : s.len;
                most_keys = max(most_keys, min(seen, s.len));
                most_before = max(most_before, min(seen, s.len - s.n));
            }
            return t;
        },
        [&](int64_t b, int64_t before, int64_t t) {
            if (index >= before && index < before + t) {
                found[0] = b;
                found[1] = index - before;
            }
        });
    if (g.parts > 1) {
        if (most_keys > 0) atomicMax(longest, most_keys);
        if (most_before > 0) atomicMax(longest + 1, most_before);
        __syncthreads();
    }
    r.b = uniform64(found[0]);
    if (r.b < 0) return false;
    r.s = sequence_at(a, r.b);
    int64_t rows;
    row_tiles_of(g, r.s, &rows);
    r.rows = (int)rows;
    r.row0 = (int)uniform64(found[1]) * kRowTile;
    const int last = r.row0 + kRowTile < r.rows ? r.row0 + kRowTile : r.rows;
    const int first_pos = r.s.len - r.s.n + r.row0 / g.G, last_pos = r.s.len - r.s.n + (last - 1) / g.G;
    r.hi = a.causal ? last_pos + 1 : r.s.len;
    if (r.hi < 0) r.hi = 0;
    const int64_t lo = a.window > 0 ? (int64_t)first_pos - a.window + 1 : 0;
    r.low = lo > 0 ? (int)(lo < r.hi ? lo : r.hi) : 0;
    r.lo = r.low & ~(kKeyTile - 1);
    const int nt = (r.hi - r.lo + kKeyTile - 1) / kKeyTile;
    r.parts = 1;
    if (g.parts > 1) {
        // In proportion to the keys, the most that any tile of rows sees in all:
        // by the lengths, since a table may be far wider (512 tokens behind
        // 32488 in a table for 131072 394 us as in one for 33000; in one part,
        // as by that width, 1031).
        const int keys = __builtin_amdgcn_readfirstlane(longest[0]), before = __builtin_amdgcn_readfirstlane(longest[1]);
        const int parts = before <= keys / 2 ? g.prompt_parts : g.prefix_parts;
        int each = (keys + kKeyTile * parts - 1) / (kKeyTile * parts);
        each = each < kMinKeyTiles ? kMinKeyTiles : each;
        const int most = (nt + each - 1) / each;
        r.parts = most < parts ? (most < 1 ? 1 : most) : parts;
    }
    return true;
}

// Where a piece of 16 bytes of a row of LDS lies: dealt so that neither 8 keys
// at one piece (reads of keys), nor 4 keys at two pieces (transposing reads of
// values), nor the c-th pieces of 4 neighbours of two keys (writes) meet in a
// bank.
__device__ __forceinline__ int key_turn(int key) { return key & 7; }
__device__ __forceinline__ int value_turn(int key) { return ((key & 1) << 2) | (key & 2) | ((key >> 2) & 1); }
__device__ __forceinline__ int place(int piece, int turn) { return piece ^ ((piece >> 2) & 3) ^ turn; }

typedef short short4_t __attribute__((ext_vector_type(4)));

// (code - zero) scale of 8 codes in fp16, in the order 0 4 1 5 2 6 3 7; `magic`
// in a register, since an instruction takes one constant.
__device__ __forceinline__ u32x4_t decode8(uint32_t w, half2_t off, half2_t s, uint32_t mask, uint32_t magic) {
    const uint32_t r[4] = {(w & mask) | magic, ((w >> 4) & mask) | magic, ((w >> 8) & mask) | magic, ((w >> 12) & mask) | magic};
    u32x4_t o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const half2_t h = (__builtin_bit_cast(half2_t, r[i]) + off) * s;
        o[i] = __builtin_bit_cast(uint32_t, h);
    }
    return o;
}

// A tile's scales from 2^(e - 14) to 2^e are normal in fp16 under 2^-e, so that
// keys and values are rounded by 2^-11 of themselves.
constexpr int kSpan = 14;

struct TileScales {
    uint32_t key_top, key_bottom, value_top, value_bottom;  // bits of the largest finite scale, 0x7C00 less the smallest but 0
    uint32_t wild;                                          // kWild, kHidden
};
// Some scale of a value is not finite; some page of the table is not one; some
// scale is outside of the exponents in use.
enum { kWild = 1, kHidden = 2, kOutside = 4 };

// KB: blocks of 32 keys a tile (with 192 and 256 dimensions one: the scores of
// two would not stay in registers beside the sums).
// EXACT: keys enter as c - zero and a score is multiplied behind each block of
// 64 by its scale over that of the next, so that it has the precision of fp32.
// For calls that ask for lse, which is fp32: from keys rounded to fp16 it was
// off by 3e-5 of itself, and is by 6e-8.  out, of weights and values in fp16,
// gains nothing that a bf16 shows, and EXACT costs (512 tokens behind 32488 484
// us instead of 394, prompts of 8191 214 instead of 173, with D = 64 141
// instead of 123, with 256 533 instead of 393).
// FAR: keys as in EXACT, and values in as many powers of two as a tile of keys
// needs (14 at a time), a tile after the other: right for whatever scales a
// cache may hold, and twice as slow (512 tokens behind 32488: 394 us; begun
// again under other powers of two, for one value scale 2^11 times the others,
// 490; FAR for one that is 2^18 times the others 783, for scales from 2^-20 to
// 1 everywhere 1055).
enum TileMode { kRounded, kExact, kFar };

template <int ND, int KB>
struct TileShared {
    uint16_t sk[2][32 * KB * ND * 64], sv[2][32 * KB * ND * 64];
    float key_scales[2][ND * 32 * KB];
    int64_t sums[kTileWaves], found[2];
    int longest[2];
    uint32_t news[3];  // of a tile: kWild, kHidden, kOutside
    TileScales scales;
};

// A tile of rows over its part of the keys.  Keys and values are under one
// power of two each: that of the first tile of keys, or of all.  kAgain, and
// nothing written, where the first tile's does not hold for a later one;
// kTooFar, where none does (FAR: neither).
enum TileEnd { kDone, kAgain, kTooFar };
template <int ND, int KB, TileMode MODE>
__device__ __forceinline__ TileEnd attend_tile(const AttendArgs &g, TileShared<ND, KB> &sh, const RowTile &rt, int64_t index, int h,
                                               int part, bool all, int tid) {
    constexpr int D = ND * 64, kKeys = 32 * KB;
    constexpr int kUnits = kKeys * 2 * ND;           // pieces of 16 bytes of codes of a tile of keys
    constexpr int kLoads = (2 * kUnits + kTileThreads - 1) / kTileThreads;
    constexpr bool EXACT = MODE != kRounded;
    auto &sk = sh.sk, &sv = sh.sv;
    auto &key_scales = sh.key_scales;
    auto &news = sh.news;
    auto &scales = sh.scales;
    const CacheAttend &a = g.a;
    const int lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 31, half = lane >> 5;
    const int heads = (int)a.cache.heads, page = (int)a.cache.page, pages = (int)a.cache.pages;
    const Sequence s = rt.s;
    const int nt_all = (rt.hi - rt.lo + kKeys - 1) / kKeys;
    const int t0 = (int)((int64_t)nt_all * part / rt.parts), t1 = (int)((int64_t)nt_all * (part + 1) / rt.parts);

    // Queries: the lane's row, 8 dimensions of every 16.
    const int r = rt.row0 + 32 * wave + col;
    const bool live = r < rt.rows;
    const int j = live ? r / g.G : 0, hq = h * g.G + (live ? r % g.G : 0);
    half8_t qf[ND * 4];
    float kappa;
    {
        const uint16_t *q = a.q + (int64_t)(s.first + j) * a.q_stride + (hq * D + 8 * half);
        u32x4_t raw[ND * 4];
        uint32_t most = 0;
#pragma unroll
        for (int d = 0; d < ND * 4; ++d) {
            raw[d] = *reinterpret_cast<const u32x4_t *>(q + 16 * d);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const uint32_t p = raw[d][y];
                most = pk_max(most, p & 0x7FFF7FFFu);
            }
        }
        most = half_max(pk_max(most, (uint32_t)__shfl_xor((int)most, 32)));
        const RowScale rs = row_scale<9, 0, -24, 16>(g.c, g.c_exp, most, live);  // (the keys' exponent is from -24 to 16)
        const int ex = rs.ex;
        kappa = rs.kappa;
#pragma unroll
        for (int d = 0; d < ND * 4; ++d)
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                // Codes come in the order 0 4 1 5 2 6 3 7.
                const uint32_t p = raw[d][y];
                const int to = 2 * y < 4 ? 4 * y : 4 * y - 7;
                qf[d][to] = (_Float16)ldexpf(__builtin_bit_cast(float, p << 16), ex);
                qf[d][to + 2] = (_Float16)ldexpf(__builtin_bit_cast(float, p & 0xFFFF0000u), ex);
            }
    }
    const int pos = s.len - s.n + j;
    const int seen_to = live ? (a.causal ? pos : s.len - 1) : -1;
    const int seen_from = a.window > 0 ? pos - (int)a.window + 1 : 0;
    // For the wave: keys that all its rows see, and that some row sees.
    const int wr0 = rt.row0 + 32 * wave, wr1 = wr0 + 31 < rt.rows ? wr0 + 31 : rt.rows - 1;
    const bool wave_live = wr0 < rt.rows;
    const int p0 = s.len - s.n + wr0 / g.G, p1 = s.len - s.n + (wave_live ? wr1 / g.G : 0);
    const int all_to = a.causal ? p0 : s.len - 1, some_to = wave_live ? (a.causal ? p1 : s.len - 1) : -1;
    const int64_t all_from = a.window > 0 ? (int64_t)p1 - a.window + 1 : 0;
    const int64_t some_from = a.window > 0 ? (int64_t)p0 - a.window + 1 : 0;

    const int32_t *table = a.table + rt.b * a.table_pages;
    auto page_at = [&](int key) -> int {
        if (key >= s.len) return -1;
        const int id = table[key >> g.page_shift];
        return id >= 0 && id < pages ? id : -1;
    };

    // What the thread decodes: pieces of 32 codes, keys' before values'.  Loads
    // are made without conditions, their values looked at where they are used:
    // a wait then never holds for loads that came after.
    struct Raw {
        u32x4_t codes;
        uint32_t scale, zero;
        uint32_t after;  // EXACT: the scale of a key's next block
        bool ok, hidden;
    };
    Raw raw[kLoads], coming[kLoads];  // of the tile to decode, and of the next
    int next_id[kLoads];              // the table's entries for the load after
    const int last_page = (s.len - 1) >> g.page_shift;
    auto is_value = [&](int i) { return wave * 64 + kTileThreads * i >= kUnits; };
    auto is_piece = [&](int i) { return wave * 64 + kTileThreads * i < 2 * kUnits; };
    auto key_of = [&](int i, int tile) {
        const int in = (tid + kTileThreads * i) % kUnits;
        return rt.lo + (tile < t1 ? tile : t1 - 1) * kKeys + in / (2 * ND);
    };
    auto ids = [&](int tile) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int p = key_of(i, tile) >> g.page_shift;
            next_id[i] = table[p < last_page ? p : last_page];
        }
    };
    auto load = [&](int tile) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int piece = (tid + kTileThreads * i) % (2 * ND), key = key_of(i, tile);
            const bool value = is_value(i), page_ok = (uint32_t)next_id[i] < (uint32_t)pages;
            Raw &c = coming[i];
            c.ok = page_ok && key >= rt.low && key < rt.hi;  // (others may hold anything)
            c.hidden = !page_ok && key < s.len;
            const int64_t row = ((int64_t)(page_ok ? next_id[i] : 0) * heads + h) * page + (key & (page - 1));
            c.codes = *reinterpret_cast<const u32x4_t *>((value ? a.cache.v_codes : a.cache.k_codes) + row * (D / 2) + piece * 16);
            c.scale = (value ? a.cache.v_scales : a.cache.k_scales)[row * ND + piece / 2];
            c.zero = (value ? a.cache.v_zeros : a.cache.k_zeros)[row * ND + piece / 2];
            if (EXACT && ND > 1) c.after = a.cache.k_scales[row * ND + (piece / 2 + 1 < ND ? piece / 2 + 1 : piece / 2)];
        }
    };
    auto take = [&] {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) raw[i] = coming[i];
    };
    // Tells of finite scales outside of the exponents in use, and of what is rare.
    auto publish = [&](int tile, int ek, int ev) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (!is_piece(i)) break;
            const Raw &c = coming[i];
            const bool value = is_value(i);
            const uint32_t bits = c.ok && (value || !EXACT) ? c.scale : 0;
            if (__any(outside<kSpan>(bits, value ? ev : ek) || c.hidden)) {
                const bool fin = bits < 0x7C00u;
                const uint32_t rare = (__any(fin && outside<kSpan>(bits, value ? ev : ek)) ? (uint32_t)kOutside : 0u) |
                                      (value && __any(!fin) ? (uint32_t)kWild : 0u) | (__any(c.hidden) ? (uint32_t)kHidden : 0u);
                if (lane == 0) atomicOr(&news[tile % 3], rare);
            }
        }
    };
    // The exponents that all finite scales of the tiles t .. end - 1 are within,
    // in the middle, so that larger and smaller ones later on are within
    // too; and what is rare in the last of them (which stays in `coming`).
    // False where one exponent is not enough.
    auto survey = [&](int t, int end, int &ek, int &ev, uint32_t &wild) -> bool {
        uint32_t top[kLoads] = {}, bottom[kLoads] = {}, rare = 0;
        if (tid == 0) scales = TileScales{0, 0, 0, 0, 0};
        for (; t < end; ++t) {
            ids(t);
            load(t);
            rare = 0;
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                if (!is_piece(i)) break;
                const Raw &c = coming[i];
                const bool value = is_value(i);
                const uint32_t bits = c.ok && (value || !EXACT) ? c.scale : 0;
                const bool fin = bits > 0 && bits < 0x7C00u;
                top[i] = max(top[i], fin ? bits : 0);
                bottom[i] = max(bottom[i], fin ? 0x7C00u - bits : 0);
                rare |= (value && bits >= 0x7C00u ? (uint32_t)kWild : 0u) | (c.hidden ? (uint32_t)kHidden : 0u);
            }
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (!is_piece(i)) break;
            const bool value = is_value(i);
            const uint32_t x = wave_max_u32(top[i]), y = wave_max_u32(bottom[i]);
            if (lane == 0) {
                atomicMax(value ? &scales.value_top : &scales.key_top, x);
                atomicMax(value ? &scales.value_bottom : &scales.key_bottom, y);
            }
        }
        if (rare) atomicOr(&scales.wild, rare);
        __syncthreads();
        const TileScales n = scales;
        wild = __builtin_amdgcn_readfirstlane(n.wild);
        auto bits = [](uint32_t x) { return (uint32_t)__builtin_amdgcn_readfirstlane(x); };
        const bool keys = fit<kSpan>(bits(n.key_top), 0x7C00u - bits(n.key_bottom), &ek);
        const bool values = fit<kSpan>(bits(n.value_top), 0x7C00u - bits(n.value_bottom), &ev);
        return keys && values;
    };
    uint32_t mask = 0x000F000Fu, magic = 0x64006400u;  // 1024 + code
    asm volatile("" : "+s"(mask), "+v"(magic));
    // 32 codes in fp16, times sc.
    auto put = [&](const Raw &c0, bool value, int buf, int key, int piece, _Float16 sc) {
        const _Float16 of = (_Float16)(-1024.0f - (c0.ok ? f16_bits_to_f32(c0.zero) : 0.0f));
        const half2_t s2 = {sc, sc}, o2 = {of, of};
        const uint32_t w[4] = {c0.codes.x, c0.codes.y, c0.codes.z, c0.codes.w};
        uint16_t *row = (value ? sv[buf] : sk[buf]) + key * D;
        const int turn = value ? value_turn(key) : key_turn(key);
#pragma unroll
        for (int c = 0; c < 4; ++c)
            *reinterpret_cast<u32x4_t *>(row + place(4 * piece + c, turn) * 8) = decode8(w[c], o2, s2, mask, magic);
    };
    auto decode = [&](int buf, int ek, int ev) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            if (!is_piece(i)) break;
            const int in = (tid + kTileThreads * i) % kUnits, piece = in % (2 * ND), key = in / (2 * ND);
            const bool value = is_value(i);
            const Raw &c0 = raw[i];
            uint32_t sb = c0.ok ? c0.scale : 0;
            if (EXACT && !value) {
                // A scale of 0 (codes of 0) as 2^-24: it divides the one before.
                const float own = f16_bits_to_f32(sb > 0 ? sb : 1u), after = f16_bits_to_f32(c0.ok && c0.after > 0 ? c0.after : 1u);
                if (!(piece & 1)) key_scales[buf][piece / 2 * kKeys + key] = piece / 2 + 1 < ND ? own * __builtin_amdgcn_rcpf(after) : own;
                sb = sb > 0 ? 0x3C00u : 0u;
            }
            if (value && sb >= 0x7C00u) sb = 0;  // (rows that see it are made NaN below)
            put(c0, value, buf, key, piece, (_Float16)ldexpf(f16_bits_to_f32(sb), -(value ? ev : EXACT ? 0 : ek)));
        }
    };

    float16_t o[2 * ND];
#pragma unroll
    for (int y = 0; y < 2 * ND; ++y)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[y][i] = 0;
    float top = -INFINITY, nk = kTop, ck = INFINITY, l = 0;
    int ek = -24, ev = -24;
    uint32_t wild = 0, wild_next = 0;

    // A tile in the buffers: its scores, their weights, and the values' sums.
    auto scores = [&](int buf, float16_t(&S)[KB]) {
        const uint16_t *kb = sk[buf];
#pragma unroll
        for (int x = 0; x < KB; ++x)
#pragma unroll
            for (int i = 0; i < 16; ++i) S[x][i] = 0;
#pragma unroll
        for (int d = 0; d < ND * 4; ++d) {
#pragma unroll
            for (int x = 0; x < KB; ++x) {
                const u32x4_t k = *reinterpret_cast<const u32x4_t *>(kb + (32 * x + col) * D + ((2 * d ^ ((d >> 1) & 3)) ^ half ^ key_turn(col)) * 8);
                S[x] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, k), qf[d], S[x], 0, 0, 0);
            }
            if (EXACT && (d & 3) == 3) {
                // Behind a block its scale, over that of the next block.
                const float *ks = key_scales[buf] + d / 4 * kKeys + 4 * half;
#pragma unroll
                for (int x = 0; x < KB; ++x)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const float4_t sc = *reinterpret_cast<const float4_t *>(ks + 32 * x + 8 * g);
#pragma unroll
                        for (int i = 0; i < 4; ++i) S[x][4 * g + i] *= sc[i];
                    }
            }
        }
    };
    auto weights = [&](int key0, float kap, float16_t(&S)[KB], half8_t(&pf)[KB][2]) {
        if (key0 + kKeys - 1 > all_to || key0 < all_from || (wild & kHidden)) {
            uint64_t shown = ~0ull;
            if (wild & kHidden) shown = __ballot(page_at(key0 + lane) >= 0);
#pragma unroll
            for (int x = 0; x < KB; ++x)
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int key = key0 + 32 * x + 8 * (i / 4) + 4 * half + (i & 3);
                    if (key > seen_to || key < seen_from || !(shown >> (key - key0) & 1)) S[x][i] = -INFINITY;
                }
        }
        float tm = S[0][0];
#pragma unroll
        for (int x = 0; x < KB; ++x)
#pragma unroll
            for (int i = 0; i < 16; ++i) tm = fmaxf(tm, S[x][i]);
        if (__any(fmaf(tm, kap, ck) > kTop + kHeadroom)) {
            const float m = fmaxf(top, fmaxf(tm, __shfl_xor(tm, 32)) * kap);
            const float kn = m == -INFINITY ? kTop : kTop - m;
            const float fade = top == -INFINITY ? 1.0f : __builtin_amdgcn_exp2f(kn - nk);
            top = m;
            nk = kn;
            ck = m == -INFINITY ? INFINITY : kn;
            l *= fade;
#pragma unroll
            for (int y = 0; y < 2 * ND; ++y) o[y] *= fade;
        }
#pragma unroll
        for (int x = 0; x < KB; ++x)
#pragma unroll
            for (int y = 0; y < 2; ++y) {
                u32x4_t w;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float pa = __builtin_amdgcn_exp2f(fmaf(S[x][8 * y + 2 * i], kap, nk));
                    const float pb = __builtin_amdgcn_exp2f(fmaf(S[x][8 * y + 2 * i + 1], kap, nk));
                    const half2_t p2 = {(_Float16)pa, (_Float16)pb};
                    l += pa + pb;
                    w[i] = __builtin_bit_cast(uint32_t, p2);
                }
                pf[x][y] = __builtin_bit_cast(half8_t, w);
            }
    };
    auto add_values = [&](int buf, const half8_t(&pf)[KB][2]) {
        const uint16_t *vb = sv[buf];
        const int gk = 4 * half + ((lane & 15) >> 2);               // the key of 8 that the lane's address names
        const int gd = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);   // its piece of a block of 32 dimensions
#pragma unroll
        for (int x = 0; x < KB; ++x)
#pragma unroll
            for (int z = 0; z < 2; ++z)
#pragma unroll
                for (int y = 0; y < 2 * ND; ++y) {
                    typedef __attribute__((address_space(3))) short4_t lds_short4;
                    typedef short short8_t __attribute__((ext_vector_type(8)));
                    const uint16_t *va = vb + gk * D + ((4 * y ^ (y & 3)) ^ gd ^ value_turn(gk)) * 8 + (lane & 1) * 4;
                    const short4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(va + (32 * x + 16 * z) * D));
                    const short4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_short4 *)(va + (32 * x + 16 * z + 8) * D));
                    const short8_t v8 = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
                    o[y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(half8_t, v8), pf[x][z], o[y], 0, 0, 0);
                }
    };
    // Rows that see a value whose scale is not finite.
    auto infect = [&](int key0) {
        for (int k = 0; k < kKeys; ++k) {
            const int key = key0 + k, id = page_at(key);
            if (id < 0) continue;
            const int64_t row = ((int64_t)id * heads + h) * page + (key & (page - 1));
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const float bad = a.cache.v_scales[row * ND + d] >= 0x7C00u && key <= seen_to && key >= seen_from ? NAN : 0.0f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    o[2 * d][i] += bad;
                    o[2 * d + 1][i] += bad;
                }
            }
        }
    };
    // o is in units of 2^ev.
    auto rescale = [&](int to) {
        const float f = exp2i(ev - to);
        ev = to;
#pragma unroll
        for (int y = 0; y < 2 * ND; ++y) o[y] *= f;
    };

    if constexpr (MODE != kFar) {
        if (t0 < t1) {
            if (tid < 3) news[tid] = 0;
            if (!survey(t0, all ? t1 : t0 + 1, ek, ev, wild_next)) return kTooFar;
            if (all) {
                ids(t0);
                load(t0);
                wild_next = kWild | kHidden;  // (of the last tile, not this one: looked for)
            }
            take();
            decode(t0 & 1, ek, ev);
            ids(t0 + 1);
            load(t0 + 1);
            ids(t0 + 2);
            publish(t0 + 1, ek, ev);
        }
        for (int tile = t0; tile < t1; ++tile) {
            __syncthreads();
            // This tile is in LDS, the next one in registers.
            wild = wild_next;
            wild_next = __builtin_amdgcn_readfirstlane(news[(tile + 1) % 3]);
            if (wild_next & kOutside) return kAgain;
            if (tid == 0) news[tile % 3] = 0;  // (read before this barrier, written after the next)
            take();
            load(tile + 2);
            ids(tile + 3);
            if (tile + 1 < t1) decode((tile + 1) & 1, ek, ev);
            const int key0 = rt.lo + tile * kKeys;
            if (key0 <= some_to && key0 + kKeys - 1 >= some_from) {
                float16_t S[KB];
                half8_t pf[KB][2];
                scores(tile & 1, S);
                weights(key0, EXACT ? kappa : ldexpf(kappa, ek), S, pf);
                add_values(tile & 1, pf);
                if (wild & kWild) infect(key0);
            }
            publish(tile + 2, ek, ev);
        }
    } else {
        for (int tile = t0; tile < t1; ++tile) {
            __syncthreads();
            int e;
            const bool one = survey(tile, tile + 1, ek, e, wild);
            if (!one) e = kSpan - 26;  // values below 2^-12, then 2^2, then 2^16
            const int key0 = rt.lo + tile * kKeys;
            const bool seen = key0 <= some_to && key0 + kKeys - 1 >= some_from;
            auto decode_values = [&](int e) {
#pragma unroll
                for (int i = 0; i < kLoads; ++i) {
                    if (!is_piece(i) || !is_value(i)) continue;
                    const int in = (tid + kTileThreads * i) % kUnits;
                    const uint32_t sb = coming[i].ok && coming[i].scale < 0x7C00u && !outside<kSpan>(coming[i].scale, e) ? coming[i].scale : 0;
                    put(coming[i], true, 0, in / (2 * ND), in % (2 * ND), (_Float16)ldexpf(f16_bits_to_f32(sb), -e));
                }
            };
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                if (!is_piece(i) || is_value(i)) continue;
                const int in = (tid + kTileThreads * i) % kUnits, piece = in % (2 * ND), key = in / (2 * ND);
                const uint32_t sb = coming[i].ok ? coming[i].scale : 0;
                if (!(piece & 1)) key_scales[1][piece / 2 * kKeys + key] = f16_bits_to_f32(sb > 0 ? sb : 1u);
                put(coming[i], false, 0, key, piece, (_Float16)(sb > 0 ? 1.0f : 0.0f));
            }
            decode_values(e);
            __syncthreads();
            for (int i = tid; i < ND * kKeys; i += kTileThreads)
                key_scales[0][i] = key_scales[1][i] / (i + kKeys < ND * kKeys ? key_scales[1][i + kKeys] : 1.0f);
            __syncthreads();
            half8_t pf[KB][2];
            if (seen) {
                float16_t S[KB];
                scores(0, S);
                weights(key0, kappa, S, pf);
            }
            for (;;) {
                rescale(e);
                if (seen) add_values(0, pf);
                e += kSpan;
                if (one || e > 16) break;
                __syncthreads();
                decode_values(e);
                __syncthreads();
            }
            if (seen && (wild & kWild)) infect(key0);
        }
    }

    // Results.  Of 8 dimensions the lane has 0 4 1 5 (2 6 3 7 in the other half
    // of the wave): exchanged, it has 0 1 2 3 (4 5 6 7).
    const float sum = l + __shfl_xor(l, 32), ref = -nk;
#pragma unroll
    for (int y = 0; y < 2 * ND; ++y)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a0 = o[y][4 * i], a1 = o[y][4 * i + 1], a2 = o[y][4 * i + 2], a3 = o[y][4 * i + 3];
            const float b0 = __shfl_xor(half ? a0 : a1, 32), b1 = __shfl_xor(half ? a2 : a3, 32);
            o[y][4 * i] = half ? b0 : a0;
            o[y][4 * i + 1] = half ? b1 : a2;
            o[y][4 * i + 2] = half ? a1 : b0;
            o[y][4 * i + 3] = half ? a3 : b1;
        }
    if (!live) return kDone;
    const int64_t t = s.first + j;
    if (rt.parts == 1) {
        const float f = sum == 0 ? 0.0f : exp2i(ev) / sum;
        const int64_t at = (t * a.q_heads + hq) * D + 4 * half;
#pragma unroll
        for (int y = 0; y < 2 * ND; ++y)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float4_t v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = sum == 0 ? 0.0f : o[y][4 * i + e] * f;
                store4(a, at + 32 * y + 8 * i, v);
            }
        if (a.lse && half == 0)
            a.lse[t * a.q_heads + hq] = sum == 0 ? -INFINITY : (ref + __builtin_amdgcn_logf(sum)) * 0.693147180559945f;
    } else {
        const float f = exp2i(ev);
        const int64_t slot = ((index * heads + h) * g.parts + part) * kRowTile + 32 * wave + col;
        float *p = g.part + slot * D + 4 * half;
#pragma unroll
        for (int y = 0; y < 2 * ND; ++y)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float4_t v;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[e] = o[y][4 * i + e] * f;
                *reinterpret_cast<float4_t *>(p + 32 * y + 8 * i) = v;
            }
        if (half == 0) {
            g.part_sums[slot * 2] = ref;
            g.part_sums[slot * 2 + 1] = sum;
        }
    }
    return kDone;
}

template <int ND, int KB, bool EXACT>
__global__ __launch_bounds__(kTileThreads, 1) void attend_tile_kernel(AttendArgs g) {
    __shared__ __attribute__((aligned(16))) TileShared<ND, KB> sh;
    int tid = (int)threadIdx.x;
    const int heads = (int)g.a.cache.heads;
    // The last tiles of rows see the most keys: they begin first, and all first
    // parts before the second ones (workgroups go to the card's dies and their
    // quarters strictly in turn: a tile's parts side by side, of which short
    // tiles have only the first, would leave some without work).
    const int64_t items = g.row_tiles * heads;
    const int part = (int)(blockIdx.x / items), h = (int)(blockIdx.x % heads);
    const int64_t index = g.row_tiles - 1 - (blockIdx.x - part * items) / heads;
    RowTile rt;
    const bool valid = find_row_tile<kTileThreads>(g, index, sh.sums, sh.found, sh.longest, rt);
    if (part == 0 && h == 0 && tid == 0)
        g.tile_rows[index] = valid ? TileRows{rt.s.first, rt.row0, rt.rows, rt.parts} : TileRows{0, 0, 0, 0};
    if (!valid || part >= rt.parts) return;
    // (What is made of an opaque tid is not kept in registers for the next run.)
    for (bool all = false;; all = true) {
        asm volatile("" : "+v"(tid));
        const TileEnd end = attend_tile<ND, KB, EXACT ? kExact : kRounded>(g, sh, rt, index, h, part, all, tid);
        if (end == kDone) return;
        __syncthreads();
        if (end == kTooFar || all) break;
    }
    // (As a call that is not inlined it took 612 MB of scratch memory where D = 256
    // instead of 109, for 376 us instead of 393.)
    asm volatile("" : "+v"(tid));
    attend_tile<ND, KB, kFar>(g, sh, rt, index, h, part, false, tid);
}

// Joins the parts of a tile of rows: 4 dimensions of a row a lane.
template <int ND>
__global__ __launch_bounds__(256) void attend_tile_join_kernel(AttendArgs g) {
    constexpr int D = ND * 64, kRows = 256 / (16 * ND);  // rows at a time, 4 times
    const CacheAttend &a = g.a;
    const int heads = (int)a.cache.heads, h = (int)(blockIdx.x % heads);
    const int64_t index = blockIdx.x / heads;
    const scalar_int *desc = (const scalar_int *)(g.tile_rows + index);
    const int first = desc[0], row0 = desc[1], rows = desc[2], parts = desc[3];
    if (parts < 2) return;
    const int c0 = (int)threadIdx.x / (D / 4), d = (int)threadIdx.x % (D / 4) * 4;
    if (c0 >= kRows) return;
    for (int c = (int)blockIdx.y * 4 * kRows + c0; c < ((int)blockIdx.y + 1) * 4 * kRows && c < kRowTile && row0 + c < rows; c += kRows) {
        const int r = row0 + c;
        const int64_t slot0 = (index * heads + h) * g.parts * kRowTile + c;
        const float2 *sums = reinterpret_cast<const float2 *>(g.part_sums) + slot0;
        const float *part = g.part + slot0 * D + d;
        float top = -INFINITY, lt = 0;
        float4_t ot = {0, 0, 0, 0};
        // Four parts at a time; one past the last counts for nothing.
        for (int p0 = 0; p0 < parts; p0 += 4) {
            float2 q[4];
            float4_t v[4];
            float most = top;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t p = (int64_t)(p0 + i < parts ? p0 + i : 0) * kRowTile;
                q[i] = sums[p];
                v[i] = *reinterpret_cast<const float4_t *>(part + p * D);
                if (p0 + i >= parts) q[i].y = 0;
                if (q[i].y != 0) most = fmaxf(most, q[i].x);
            }
            const float fade = top == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(top - most);
            if (top != -INFINITY) {
                lt *= fade;
#pragma unroll
                for (int e = 0; e < 4; ++e) ot[e] *= fade;
            }
            top = most;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (q[i].y == 0) continue;
                const float f = __builtin_amdgcn_exp2f(q[i].x - top);
                lt = fmaf(f, q[i].y, lt);
#pragma unroll
                for (int e = 0; e < 4; ++e) ot[e] = fmaf(f, v[i][e], ot[e]);
            }
        }
        const int64_t t = first + r / g.G, hq = (int64_t)h * g.G + r % g.G;
        float4_t v;
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = lt == 0 ? 0.0f : ot[i] / lt;
        store4(a, (t * a.q_heads + hq) * D + d, v);
        if (a.lse && d == 0) a.lse[t * a.q_heads + hq] = lt == 0 ? -INFINITY : (top + __builtin_amdgcn_logf(lt)) * 0.693147180559945f;
    }
}

// Rows of a sequence that the split kernel takes: its accumulators have to
// stay in registers (16 rows of 64 dimensions are 16 of them).
static int split_limit(int64_t D) { return D <= 128 ? 64 : 32; }

struct AttendPlan {
    int64_t split_rows;  // the most rows of a sequence in the split kernel
    int waves;           // its waves
    bool split, tiles;   // whether the split kernel runs, and the tile kernel
    int limit;           // the most rows of a sequence that are the split kernel's
    int64_t row_tiles;   // its tiles of rows at most
    int parts;           // workgroups the keys of one are dealt to
    int prompt_parts;    // the same where there is no long prefix
    size_t floats;       // workspace
};

// Tiles of 16 rows that the split kernel's accumulators are made for, and its
// waves: those that 256 compute units hold at once.
static int split_tiles(int nd, int64_t rows) { return rows <= 16 ? 1 : nd <= 2 && rows > 32 ? 4 : 2; }
static int split_waves(int nd, int64_t rows) { return 256 * kSplitWaves * split_occupancy(nd, split_tiles(nd, rows)); }

// Workgroups that the keys of each of n tiles of rows are dealt to, each one
// more costing 4 in 100 for the joining.  Behind a long prefix all tiles see
// about as many keys: as few rounds of the 256 compute units for each key as
// possible (512 tokens behind 32488 and 8 key heads: 3 parts 393 us, 5 parts
// 467; 64 tokens: 16 parts 97 us, 8 parts 154).  In a prompt they see half as
// many as the last one on average: the parts of that one should take no longer
// than the card does with all (4096 tokens and 2 key heads: 3 parts 150 us, 2
// parts 135).
static int key_parts(int64_t n, bool prompt) {
    int best_parts = 1;
    double best = 0;
    for (int parts = 1; parts <= 32 && (parts == 1 || n * parts <= 1024); ++parts) {
        double cost = (double)((n * parts + 255) / 256) / parts;
        if (prompt) cost = 1.0 / parts > n / 512.0 ? 1.0 / parts : n / 512.0;
        cost *= 1 + 0.04 * (parts - 1);
        if (parts == 1 || cost < best) {
            best = cost;
            best_parts = parts;
        }
    }
    return best_parts;
}

static AttendPlan attend_plan(int64_t T, int64_t q_heads, int64_t heads, int64_t D, int64_t B, int64_t max_q) {
    AttendPlan p = {};
    const int64_t G = q_heads / heads, limit = split_limit(D);
    const int64_t q = max_q < T ? max_q : T;
    p.tiles = q * G > limit;
    p.split = !p.tiles || B > 1;  // (one sequence that may be long: the tile kernel takes it as it comes)
    p.limit = p.split ? (int)limit : 0;
    p.split_rows = p.tiles ? limit : q * G;
    p.waves = split_waves((int)(D / 64), p.split_rows);
    if (p.split) p.floats = (size_t)(2 * p.waves) * p.split_rows * (D + 2) + (size_t)(B * heads) * (sizeof(Pieces) / sizeof(float));
    if (p.tiles) {
        // Sequences of more rows than the limit, and their tiles.
        const int64_t most = T * G / (p.limit + 1);
        p.row_tiles = (T * G + (B < most ? B : most) * (kRowTile - 1)) / kRowTile;
        const int64_t n = p.row_tiles * heads;
        p.parts = key_parts(n, false);
        p.prompt_parts = key_parts(n, true);
        const int64_t parts = p.parts > p.prompt_parts ? p.parts : p.prompt_parts;
        const size_t f = (size_t)p.row_tiles * (sizeof(TileRows) / sizeof(float)) +
                         (parts == 1 ? 0 : (size_t)(n * parts) * kRowTile * (D + 2));
        if (f > p.floats) p.floats = f;
    }
    return p;
}

size_t attend_ws_bytes(int64_t T, int64_t q_heads, int64_t heads, int64_t D, int64_t B, int64_t max_q) {
    return attend_plan(T, q_heads, heads, D, B, max_q).floats * sizeof(float);
}

template <int ND, bool DIRECT>
static const void *split_kernel(int64_t rows) {
    const int nt = split_tiles(ND, rows);
    if (nt == 1) return reinterpret_cast<const void *>(&attend_split_kernel<ND, 1, DIRECT>);
    if constexpr (ND <= 2) {
        if (nt == 4) return reinterpret_cast<const void *>(&attend_split_kernel<ND, 4, DIRECT>);
    }
    return reinterpret_cast<const void *>(&attend_split_kernel<ND, 2, DIRECT>);
}

// Where no token can see more keys than this (by the table, or the window): a
// workgroup for each (sequence, key head), which needs no plan and no joining.
// 64 sequences of up to 1000 keys and 8 heads 20 us instead of 31, of up to
// 2000 keys 30 instead of 36; 2 heads of one sequence on 1000 keys 13 instead
// of 18, but on 2000 21 instead of 16: there the keys need more waves.
static bool direct(int64_t keys, int64_t items) { return keys <= 1024 || (keys <= 2048 && items >= 512); }

template <int ND>
static hipError_t launch_attend(AttendArgs &g, const AttendPlan &p, float *workspace, hipStream_t stream) {
    const CacheAttend &a = g.a;
    void *args[] = {&g};
    hipError_t e = hipSuccess;
    if (p.split) {
        g.max_rows = (int)p.split_rows;
        g.part = workspace;
        g.part_sums = g.part + (size_t)(2 * p.waves) * p.split_rows * a.cache.D;
        g.pieces = reinterpret_cast<Pieces *>(g.part_sums + (size_t)(2 * p.waves) * p.split_rows * 2);
        g.waves = p.waves;
        int64_t most = a.table_pages * a.cache.page;
        if (a.window > 0 && a.window + a.max_q < most) most = a.window + a.max_q;
        if (direct(most, a.B * a.cache.heads)) {
            e = hipLaunchKernel(split_kernel<ND, true>(p.split_rows), dim3((unsigned)(a.B * a.cache.heads)), dim3(kSplitThreads), args,
                                0, stream);
        } else {
            e = hipLaunchKernel(split_kernel<ND, false>(p.split_rows), dim3((unsigned)(p.waves / kSplitWaves)), dim3(kSplitThreads),
                                args, 0, stream);
            if (e != hipSuccess) return e;
            e = hipLaunchKernel(reinterpret_cast<const void *>(&attend_join_kernel),
                                dim3((unsigned)(a.B * a.cache.heads), (unsigned)p.split_rows, ND), dim3(256), args, 0, stream);
        }
    }
    if (e != hipSuccess || !p.tiles) return e;
    g.row_tiles = p.row_tiles;
    const int64_t keys = a.table_pages * a.cache.page;
    // Whether there is a long prefix the lengths say, and sometimes the table.
    g.prompt_parts = a.causal ? p.prompt_parts : p.parts;
    g.prefix_parts = 2 * a.max_q >= keys ? g.prompt_parts : p.parts;
    const int parts = g.prompt_parts > g.prefix_parts ? g.prompt_parts : g.prefix_parts;
    g.parts = parts;
    const int64_t n = p.row_tiles * a.cache.heads;
    g.tile_rows = reinterpret_cast<TileRows *>(workspace);
    g.part = workspace + (size_t)p.row_tiles * (sizeof(TileRows) / sizeof(float));
    g.part_sums = g.part + (size_t)n * parts * kRowTile * a.cache.D;
    constexpr int KB = ND <= 2 ? 2 : 1;
    e = hipLaunchKernel(a.lse ? reinterpret_cast<const void *>(&attend_tile_kernel<ND, KB, true>)
                              : reinterpret_cast<const void *>(&attend_tile_kernel<ND, KB, false>),
                        dim3((unsigned)(n * parts)), dim3(kTileThreads), args, 0, stream);
    if (e != hipSuccess || parts == 1) return e;
    constexpr int kJoinRows = 4 * (256 / (16 * ND));
    return hipLaunchKernel(reinterpret_cast<const void *>(&attend_tile_join_kernel<ND>),
                           dim3((unsigned)n, (kRowTile + kJoinRows - 1) / kJoinRows), dim3(256), args, 0, stream);
}

hipError_t launch_cache_attend(const CacheAttend &a, void *workspace, hipStream_t stream) {
    AttendArgs g = {};
    g.a = a;
    if (a.cache.pages == 0) g.a.table_pages = 0;  // no key can be seen
    if (a.window > g.a.table_pages * a.cache.page) g.a.window = 0;  // it reaches past the first key everywhere
    g.page_shift = __builtin_ctzll((unsigned long long)a.cache.page);
    g.G = (int)(a.q_heads / a.cache.heads);
    g.inv_G = (65536 + g.G - 1) / g.G;
    const float c = a.scale * 1.44269504088896f;
    g.c = frexpf(c < FLT_MAX ? c : FLT_MAX, &g.c_exp);
    const AttendPlan p = attend_plan(a.T, a.q_heads, a.cache.heads, a.cache.D, a.B, a.max_q);
    g.limit = p.limit;
    float *ws = static_cast<float *>(workspace);
    switch (a.cache.D / 64) {
        case 1: return launch_attend<1>(g, p, ws, stream);
        case 2: return launch_attend<2>(g, p, ws, stream);
        case 3: return launch_attend<3>(g, p, ws, stream);
        default: return launch_attend<4>(g, p, ws, stream);
    }
}

}  // namespace q4
