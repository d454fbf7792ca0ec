// q4_attend.hip -- attention over the 4-bit key/value cache.
//
// For a row (a token's query head) with scores s_i = scale q . k_i over the
// keys it sees: out = sum p_i v_i / sum p_i, p_i = 2^(c (s_i - m)), c = log2 e.
// One pass over the keys, with the running maximum m; sums are fp32.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "q4_cache_internal.h"
#include "q4_device.h"

namespace q4 {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef int int2_t __attribute__((ext_vector_type(2)));

struct AttendArgs {
    CacheAttend a;
    int page_shift;
    int G;            // query heads a key head
    int limit;        // the split kernel takes sequences of at most this many rows
    int max_rows;     // rows a partial result is kept for
    float *part;      // partial results: [slot][max_rows][D], then (ref, sum) pairs
    float *part_sums;
};

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
// p' enters as fp16 (2^-11, random): scaled by 2^F so that the largest value
// scale of the keys so far, times a weight of 1, is 2^9; when the maximum
// grows by less than 2^6 nothing is rescaled.
//
// The work is the list of all tiles of 32 keys of all (sequence, key head),
// dealt evenly to a fixed number of workgroups, whatever the lengths: each
// finds its share from the lengths.  What a workgroup begins and does not end,
// or ends and did not begin, goes to the workspace, and a second launch joins
// the pieces in order (the same bits on every call).
// ---------------------------------------------------------------------------

constexpr int kTile = 32;        // keys a wave takes at a time
constexpr int kSplitWaves = 4;
constexpr int kSplitThreads = 64 * kSplitWaves;
constexpr int kSplitGroups = 512;  // workgroups: two a compute unit
constexpr int kMinTiles = 8;       // tiles a workgroup should have at least
constexpr int kHeadroom = 6;       // powers of two that weights may pass 1 by

struct Share {
    int64_t total, workers;
};

// Tiles of one key head of a sequence (one at least where it has rows, so
// that rows without keys are written).
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

__device__ __forceinline__ int64_t workers_of(int64_t total) {
    const int64_t w = (total + kMinTiles - 1) / kMinTiles;
    return w < 1 ? 1 : w > kSplitGroups ? kSplitGroups : w;
}
__device__ __forceinline__ int64_t share_start(int64_t total, int64_t workers, int64_t w) { return total * w / workers; }
// The worker that holds tile i.
__device__ __forceinline__ int64_t worker_at(int64_t total, int64_t workers, int64_t i) {
    int64_t w = (i * workers) / total;
    while (share_start(total, workers, w + 1) <= i) ++w;
    while (share_start(total, workers, w) > i) --w;
    return w;
}

// Prefix sums of the sequences' tiles by a workgroup of THREADS: the total,
// and for `find` (a sequence's index, or a position in the sum) where it lies.
template <int THREADS, class Found>
__device__ __forceinline__ int64_t scan_tiles(const AttendArgs &g, int64_t *sums, Found found) {
    const int tid = (int)threadIdx.x, wave = tid >> 6;
    int64_t before = 0;
    for (int64_t b0 = 0; b0 < g.a.B; b0 += THREADS) {
        const int64_t b = b0 + tid;
        int lo, t = 0;
        if (b < g.a.B) t = tiles_of(g, sequence_at(g.a, b), &lo);
        int64_t x = t;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int64_t y = __shfl_up(x, d);
            if ((tid & 63) >= d) x += y;
        }
        if ((tid & 63) == 63) sums[wave] = x;
        __syncthreads();
        int64_t off = before, all = 0;
#pragma unroll
        for (int w = 0; w < THREADS / 64; ++w) {
            if (w < wave) off += sums[w];
            all += sums[w];
        }
        if (b < g.a.B) found(b, off + x - t, t);
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

template <int ND, int NT>
struct SplitShared {
    static constexpr int kPad = 4;
    union {
        struct {
            uint8_t v[kSplitWaves][kTile * ND * 32];
            uint32_t par[kSplitWaves][64 * ND];
        } in;
        float o[kSplitWaves][16][ND * 64 + kPad];
    };
    float ref[kSplitWaves][16 * NT], sum[kSplitWaves][16 * NT];
    int64_t sums[kSplitWaves];
    int64_t start_b, start_at;
};

template <int ND, int NT>
__global__ __launch_bounds__(kSplitThreads, NT * ND > 4 ? 1 : 2) void attend_split_kernel(AttendArgs g) {
    constexpr int D = ND * 64;
    __shared__ __attribute__((aligned(16))) SplitShared<ND, NT> sh;
    const CacheAttend &a = g.a;
    const int tid = (int)threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int col = lane & 15, grp = lane >> 4;
    const int heads = (int)a.cache.heads, page = (int)a.cache.page, pages = (int)a.cache.pages;

    const int64_t tiles = scan_tiles<kSplitThreads>(g, sh.sums, [](int64_t, int64_t, int) {});
    const int64_t total = tiles * heads, workers = workers_of(total);
    const int64_t w = blockIdx.x;
    if (total == 0 || w >= workers) return;
    const int64_t begin = share_start(total, workers, w), end = share_start(total, workers, w + 1);
    scan_tiles<kSplitThreads>(g, sh.sums, [&](int64_t b, int64_t before, int t) {
        if (begin >= before * heads && begin < (before + t) * heads) {
            sh.start_b = b;
            sh.start_at = before * heads;
        }
    });
    int64_t b = uniform64(sh.start_b), at = uniform64(sh.start_at);  // tiles before sequence b

    int64_t i = begin;
    while (i < end) {
        const Sequence s = sequence_at(a, b);
        int lo_key;
        const int nt = tiles_of(g, s, &lo_key);
        if (i >= at + (int64_t)nt * heads) {
            at += (int64_t)nt * heads;
            ++b;
            continue;
        }
        const int h = (int)((i - at) / nt);
        const int64_t row_start = at + (int64_t)h * nt;
        const int t0 = (int)(i - row_start);
        const int t1 = (int)(end - row_start < nt ? end - row_start : nt);
        const int n = s.n < a.max_q ? s.n : (int)a.max_q;
        const int rows = n * g.G;

        // Queries: the lane's row of each tile of 16, its 8 dimensions of every 32.
        half8_t qf[NT][ND][2];
        float qsum[NT][ND], kappa[NT];
        int seen_to[NT], seen_from[NT];  // keys seen by the lane's row
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            const int r = 16 * x + col;
            const int j = r < rows ? r / g.G : 0, hq = h * g.G + (r < rows ? r % g.G : 0);
            const uint16_t *q = a.q + (int64_t)(s.first + j) * a.q_stride + (int64_t)hq * D + 16 * grp;
            float v[ND][16], top = 0;
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const u32x4_t u = *reinterpret_cast<const u32x4_t *>(q + 64 * d + 8 * e);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const uint32_t p = u[y];
                        v[d][8 * e + 2 * y] = __builtin_bit_cast(float, p << 16);
                        v[d][8 * e + 2 * y + 1] = __builtin_bit_cast(float, p & 0xFFFF0000u);
                    }
                }
#pragma unroll
            for (int d = 0; d < ND; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float m = fabsf(v[d][e]);
                    if (m < INFINITY) top = fmaxf(top, m);
                }
            top = max4(top);
            // The largest to 2^14 .. 2^15.
            int ex = 0;
            if (top > 0) ex = 15 - (int)__builtin_amdgcn_frexp_expf(top);
            kappa[x] = ldexpf(a.scale * 1.44269504088896f, 20 - ex);
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                float sum = 0;
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    half8_t f;
#pragma unroll
                    for (int y = 0; y < 8; ++y) {
                        // Codes come in the order 0 4 1 5 2 6 3 7.
                        const int src = 8 * e + (y & 1) * 4 + (y >> 1);
                        const float z = r < rows ? ldexpf(v[d][src], ex) : 0.0f;
                        f[y] = (_Float16)z;
                        sum += z;
                    }
                    qf[x][d][e] = f;
                }
                qsum[x][d] = sum4(sum) * 0x1p-20f;
            }
            const int pos = s.len - s.n + j;
            seen_to[x] = r < rows ? (a.causal ? pos : s.len - 1) : -1;
            seen_from[x] = a.window > 0 ? pos - (int)(a.window < 0x7fffffff ? a.window : 0x7fffffff) + 1 : 0;
        }
        // Keys that all rows see: tiles within need no mask.
        const int all_to = a.causal ? s.len - s.n : s.len - 1;
        const int64_t all_from = a.window > 0 ? (int64_t)s.len - s.n + (n - 1) - a.window + 1 : 0;

        float m[NT], l[NT], nk[NT], ck[NT], zs[NT][ND];
        float4_t o[NT][ND][4];
        int E = -24;                   // value scales so far are below 2^E
        uint32_t limit_bits = 0;       // the largest fp16 below
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

        const int32_t *table = a.table + b * a.table_pages;
        auto page_of = [&](int key) -> int {
            if (key >= s.len) return -1;
            const int id = table[key >> g.page_shift];
            return id >= 0 && id < pages ? id : -1;
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
                row[t] = ((int64_t)(id < 0 ? 0 : id) * heads + h) * page + ((key + 16 * t) & (page - 1));
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

        int tile = t0 + wave;
        Tile<ND> T;
        int id0 = -1, id1 = -1;
        int64_t row[2];
        uint32_t *const par = sh.in.par[wave];
        if (tile < t1) {
            id0 = page_of(lo_key + tile * kTile);
            id1 = page_of(lo_key + tile * kTile + 16);
            rows_of(tile, id0, id1, row);
            load_values(row, T);
            load_keys(row, T);
        }
        for (; tile < t1; tile += kSplitWaves) {
            const bool ok[2] = {id0 >= 0, id1 >= 0};
            const bool more = tile + kSplitWaves < t1;
            if (more) {
                id0 = page_of(lo_key + (tile + kSplitWaves) * kTile);
                id1 = page_of(lo_key + (tile + kSplitWaves) * kTile + 16);
            }
            const int key = lo_key + tile * kTile;
            uint8_t *vl = sh.in.v[wave];
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                *reinterpret_cast<u32x4_t *>(vl + (lane + 64 * d) * 16) = T.v[d];
                par[lane + 64 * d] = T.par[d];
            }
            wave_fence();
            if (more) {
                rows_of(tile + kSplitWaves, id0, id1, row);
                load_values(row, T);
            }

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
            if (more) load_keys(row, T);
            uint32_t vs[2][2 * ND], vz[2][2 * ND];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                read_par<ND>(par, kValueScales, t, grp, vs[t]);
                read_par<ND>(par, kValueZeros, t, grp, vz[t]);
            }
            const bool masked = key + kTile - 1 > all_to || key < all_from || !ok[0] || !ok[1];
            if (masked) {
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int k = key + 16 * t + 4 * grp + r;
#pragma unroll
                        for (int x = 0; x < NT; ++x)
                            if (!ok[t] || k > seen_to[x] || k < seen_from[x]) S[x][t][r] = -INFINITY;
                        // A key that no row sees may hold anything.
                        if (!ok[t] || k >= s.len) {
#pragma unroll
                            for (int d = 0; d < ND; ++d) {
                                const int y = r * ND + d;
                                const uint32_t keep = y & 1 ? 0x0000FFFFu : 0xFFFF0000u;
                                vs[t][y >> 1] &= keep;
                                vz[t][y >> 1] &= keep;
                            }
                        }
                    }
            }
            // Whether a maximum has grown too far, or a value scale.
            uint32_t top_bits = 0;
#pragma unroll
            for (int t = 0; t < 2; ++t)
#pragma unroll
                for (int y = 0; y < 2 * ND; ++y) {
                    const u16x2_t p = __builtin_bit_cast(u16x2_t, top_bits), c = __builtin_bit_cast(u16x2_t, vs[t][y]);
                    top_bits = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(p, c));
                }
            top_bits = (top_bits >> 16) > (top_bits & 0xFFFF) ? top_bits >> 16 : top_bits & 0xFFFF;
            bool grown = top_bits > limit_bits;
            float tmax[NT];
#pragma unroll
            for (int x = 0; x < NT; ++x) {
                tmax[x] = fmaxf(fmaxf(fmaxf(S[x][0][0], S[x][0][1]), fmaxf(S[x][0][2], S[x][0][3])),
                                fmaxf(fmaxf(S[x][1][0], S[x][1][1]), fmaxf(S[x][1][2], S[x][1][3])));
                grown = grown || fmaf(tmax[x], kappa[x], ck[x]) > (float)(9 - E + kHeadroom);
            }
            if (__any(grown)) {
                uint32_t fin = 0;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int y = 0; y < 4 * ND; ++y) {
                        const uint32_t v = (vs[t][y >> 1] >> (16 * (y & 1))) & 0xFFFF;
                        fin = v < 0x7C00u && v > fin ? v : fin;
                    }
                fin = wave_max_u32(fin);
                // Below 2^e: the exponent of the next power of two.
                const int e = (int)(fin >> 10) == 0 ? -14 : (int)(fin >> 10) - 14;
                if (fin > 0 && e > E) {
                    E = e;
                    limit_bits = (uint32_t)(e + 15) << 10;
                    limit_bits -= 1;
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
            for (int x = 0; x < NT; ++x) {
                float p[2][4];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        p[t][r] = __builtin_amdgcn_exp2f(fmaf(S[x][t][r], kappa[x], nk[x]));
                        l[x] += p[t][r];
                    }
#pragma unroll
                for (int d = 0; d < ND; ++d)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            _Float16 w16 = (_Float16)(p[t][r] * half_at(vs[t], r * ND + d));
                            if (masked && S[x][t][r] == -INFINITY) w16 = (_Float16)0.0f;
                            pf[x][d][2 * r + t] = w16;
                            zs[x][d] = fmaf((float)w16, half_at(vz[t], r * ND + d), zs[x][d]);
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
        }

        // The four waves' results, 16 rows at a time.  A row's weights stand
        // relative to 2^ref.
        const bool whole = t0 == 0 && t1 == nt;
        const int64_t slot = 2 * w + (i == begin ? 0 : 1);
#pragma unroll
        for (int x = 0; x < NT; ++x) {
            if (16 * x >= rows) break;
            const float sum = sum4(l[x]);
            const float ref = -nk[x];
            __syncthreads();
            if (grp == 0) {
                sh.ref[wave][col] = ref;
                sh.sum[wave][col] = sum;
            }
#pragma unroll
            for (int d = 0; d < ND; ++d) {
                const float z = sum4(zs[x][d]);
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    float4_t v;
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] = fmaf(o[x][d][y][r], 0x1p20f, -z);
                    *reinterpret_cast<float4_t *>(&sh.o[wave][col][64 * d + 16 * y + 4 * grp]) = v;
                }
            }
            __syncthreads();
            for (int e = tid; e < 16 * D; e += kSplitThreads) {
                const int c = e / D, d = e - c * D, r = 16 * x + c;
                if (r >= rows) break;
                float top = -INFINITY;
#pragma unroll
                for (int y = 0; y < kSplitWaves; ++y)
                    if (sh.sum[y][c] != 0) top = fmaxf(top, sh.ref[y][c]);
                float lt = 0, ot = 0;
#pragma unroll
                for (int y = 0; y < kSplitWaves; ++y)
                    if (sh.sum[y][c] != 0) {
                        const float f = __builtin_amdgcn_exp2f(sh.ref[y][c] - top);
                        lt = fmaf(f, sh.sum[y][c], lt);
                        ot = fmaf(f, sh.o[y][c][d], ot);
                    }
                if (whole) {
                    const int64_t t = s.first + r / g.G, hq = (int64_t)h * g.G + r % g.G;
                    const float out = lt == 0 ? 0.0f : ot / lt;
                    const int64_t at_out = (t * a.q_heads + hq) * D + d;
                    if (a.bf16) static_cast<__bf16 *>(a.out)[at_out] = (__bf16)out;
                    else static_cast<float *>(a.out)[at_out] = out;
                    if (a.lse && d == 0)
                        a.lse[t * a.q_heads + hq] = lt == 0 ? -INFINITY : (top + __builtin_amdgcn_logf(lt)) * 0.693147180559945f;
                } else {
                    g.part[(slot * g.max_rows + r) * D + d] = ot;
                    if (d == 0) {
                        g.part_sums[(slot * g.max_rows + r) * 2] = top;
                        g.part_sums[(slot * g.max_rows + r) * 2 + 1] = lt;
                    }
                }
            }
        }
        __syncthreads();
        i = row_start + t1;
    }
}

// Joins the pieces of one (sequence, key head), a workgroup per row.
template <int ND>
__global__ __launch_bounds__(64 * ND) void attend_join_kernel(AttendArgs g) {
    constexpr int D = ND * 64;
    __shared__ int64_t sums[ND];
    __shared__ int64_t found_at;
    const CacheAttend &a = g.a;
    const int64_t b = blockIdx.x / a.cache.heads;
    const int h = (int)(blockIdx.x % a.cache.heads), r = (int)blockIdx.y, heads = (int)a.cache.heads;
    const Sequence s = sequence_at(a, b);
    int lo_key;
    const int nt = tiles_of(g, s, &lo_key);
    const int n = s.n < a.max_q ? s.n : (int)a.max_q;
    if (nt < 2 || r >= n * g.G) return;
    const int64_t tiles = scan_tiles<64 * ND>(g, sums, [&](int64_t x, int64_t before, int) {
        if (x == b) found_at = before;
    });
    const int64_t total = tiles * heads, workers = workers_of(total);
    const int64_t start = found_at * heads + (int64_t)h * nt;
    const int64_t w0 = worker_at(total, workers, start), w1 = worker_at(total, workers, start + nt - 1);
    if (w0 == w1) return;
    float top = -INFINITY;
    for (int64_t w = w0; w <= w1; ++w) {
        const int64_t slot = 2 * w + (w == w0 && share_start(total, workers, w) != start ? 1 : 0);
        const float *p = g.part_sums + (slot * g.max_rows + r) * 2;
        if (p[1] != 0) top = fmaxf(top, p[0]);
    }
    float lt = 0, ot = 0;
    const int d = (int)threadIdx.x;
    for (int64_t w = w0; w <= w1; ++w) {
        const int64_t slot = 2 * w + (w == w0 && share_start(total, workers, w) != start ? 1 : 0);
        const float *p = g.part_sums + (slot * g.max_rows + r) * 2;
        if (p[1] != 0) {
            const float f = __builtin_amdgcn_exp2f(p[0] - top);
            lt = fmaf(f, p[1], lt);
            ot = fmaf(f, g.part[(slot * g.max_rows + r) * D + d], ot);
        }
    }
    const int64_t t = s.first + r / g.G, hq = (int64_t)h * g.G + r % g.G;
    const float out = lt == 0 ? 0.0f : ot / lt;
    const int64_t at = (t * a.q_heads + hq) * D + d;
    if (a.bf16) static_cast<__bf16 *>(a.out)[at] = (__bf16)out;
    else static_cast<float *>(a.out)[at] = out;
    if (a.lse && d == 0)
        a.lse[t * a.q_heads + hq] = lt == 0 ? -INFINITY : (top + __builtin_amdgcn_logf(lt)) * 0.693147180559945f;
}

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
        if ((n < a.max_q ? n : a.max_q) * g.G <= g.limit) return;
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


// Rows of a sequence that the split kernel takes: its accumulators have to
// stay in registers (16 rows of 64 dimensions are 16 of them).
static int split_limit(int64_t D) { return D <= 128 ? 64 : 32; }

size_t attend_ws_bytes(int64_t T, int64_t q_heads, int64_t heads, int64_t D, int64_t B, int64_t max_q) {
    (void)B;
    const int64_t q = max_q < T ? max_q : T, limit = split_limit(D);
    int64_t rows = q * (q_heads / heads);
    if (rows > limit) rows = limit;
    return (size_t)(2 * kSplitGroups) * rows * (D + 2) * sizeof(float);
}

template <int ND>
static const void *split_kernel(int64_t rows) {
    if (rows <= 16) return reinterpret_cast<const void *>(&attend_split_kernel<ND, 1>);
    if constexpr (ND <= 2) {
        if (rows > 32) return reinterpret_cast<const void *>(&attend_split_kernel<ND, 4>);
    }
    return reinterpret_cast<const void *>(&attend_split_kernel<ND, 2>);
}

hipError_t launch_cache_attend(const CacheAttend &a, void *workspace, hipStream_t stream) {
    AttendArgs g = {};
    g.a = a;
    if (a.cache.pages == 0) g.a.table_pages = 0;  // no key can be seen
    g.page_shift = __builtin_ctzll((unsigned long long)a.cache.page);
    g.G = (int)(a.q_heads / a.cache.heads);
    g.limit = split_limit(a.cache.D);
    int64_t rows = a.max_q * g.G;
    const bool longer = rows > g.limit;
    if (longer) rows = g.limit;
    g.max_rows = (int)rows;
    g.part = static_cast<float *>(workspace);
    g.part_sums = g.part + (size_t)(2 * kSplitGroups) * rows * a.cache.D;
    const int nd = (int)(a.cache.D / 64);
    void *args[] = {&g};
    const void *split = nd == 1 ? split_kernel<1>(rows) : nd == 2 ? split_kernel<2>(rows) : nd == 3 ? split_kernel<3>(rows) : split_kernel<4>(rows);
    hipError_t e = hipLaunchKernel(split, dim3(kSplitGroups), dim3(kSplitThreads), args, 0, stream);
    if (e != hipSuccess) return e;
    const void *join[4] = {reinterpret_cast<const void *>(&attend_join_kernel<1>), reinterpret_cast<const void *>(&attend_join_kernel<2>),
                           reinterpret_cast<const void *>(&attend_join_kernel<3>), reinterpret_cast<const void *>(&attend_join_kernel<4>)};
    e = hipLaunchKernel(join[nd - 1], dim3((unsigned)(a.B * a.cache.heads), (unsigned)rows), dim3(64 * nd), args, 0, stream);
    if (e != hipSuccess || !longer) return e;
    const void *row[4] = {reinterpret_cast<const void *>(&attend_row_kernel<1>), reinterpret_cast<const void *>(&attend_row_kernel<2>),
                          reinterpret_cast<const void *>(&attend_row_kernel<3>), reinterpret_cast<const void *>(&attend_row_kernel<4>)};
    return hipLaunchKernel(row[nd - 1], dim3((unsigned)(a.T * a.q_heads)), dim3(64), args, 0, stream);
}

}  // namespace q4
