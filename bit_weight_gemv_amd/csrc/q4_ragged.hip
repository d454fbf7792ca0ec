// q4_ragged.hip -- the packed product of ragged groups of rows:
//   Y[p][m] = sum_k What_e[m,k] x_p[k]            (plain)
//   Y[p][m] = silu(What_e x_p) * (Up_e x_p)       (gate and up together)
//   Y[p][m] = What x_p + sum_j t[p][j] B_a[m][j]  (beside an adapter)
// where e is the group of position p and x_p the row of X that it names.
// Two kernels: one for few rows a group (the weights' bytes bound it) and one
// for many (the matrix cores bound it).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_internal.h"
#include "q4_ragged.h"
#include "q4_ragged_device.h"

namespace q4 {

namespace {

struct Args {
    const uint8_t *codes[2];
    const uint16_t *scales[2];
    const int8_t *rowexp[2];   // tile kernel: exponent of each row's largest scale,
    const uint16_t *tscale[2]; // and the scales over 2^(exponent - 14) as fp16, [E][K/64][M]
    int M, K, E, R;
    const uint16_t *X;         // bf16 [T][K]; fp16 [T][tile_pitch(K)] (tile kernel) or [K/8][R][8] (chunk kernel, PRE) times 2^-xexp
    const int32_t *xexp;       // the power of two of each row of X (tile kernel) or slice and position (chunk kernel)
    int T;
    const int32_t *offsets, *rows;
    void *Y;
    int bf16;
    float *part;               // chunk kernel: partial planes [mats][ranges][R][M], or null
    int ranges, slices_each, slices_more;  // chunk kernel: ranges of K, slices of each, and how many have one more
    int rowtiles, chunks;      // tile kernel: grid shape
    const uint16_t *B;
    const float *t;
    const int32_t *ids;
    int r, L;
    const uint16_t *A;         // row kernel, beside adapters: what t is made of, by the workgroups from `wgs` on
    const float *scaling;
    float *tout;
    int wgs;
};

__device__ __forceinline__ int source_row(const Args &a, int p) {
    const int row = a.rows ? a.rows[p] : p;
    return row >= 0 && row < a.T ? row : -1;
}

// The part of adapter id in output (p, m), from rank j0 on.
__device__ __forceinline__ float adapter_term(const Args &a, int id, int p, int m, int j0 = 0) {
    if (id < 0 || id >= a.L) return 0.0f;
    const uint16_t *b = a.B + ((int64_t)id * a.M + m) * a.r;
    const float *t = a.t + (int64_t)p * a.r;
    float s = 0.0f;
#pragma unroll 4
    for (int j = j0; j < a.r; j += 8) {
        const uint4 v = *reinterpret_cast<const uint4 *>(b + j);
        const float4 t0 = *reinterpret_cast<const float4 *>(t + j), t1 = *reinterpret_cast<const float4 *>(t + j + 4);
        s = fmaf(bf16_lo(v.x), t0.x, s);
        s = fmaf(bf16_hi(v.x), t0.y, s);
        s = fmaf(bf16_lo(v.y), t0.z, s);
        s = fmaf(bf16_hi(v.y), t0.w, s);
        s = fmaf(bf16_lo(v.z), t1.x, s);
        s = fmaf(bf16_hi(v.z), t1.y, s);
        s = fmaf(bf16_lo(v.w), t1.z, s);
        s = fmaf(bf16_hi(v.w), t1.w, s);
    }
    return s;
}

// ---------------------------------------------------------------------------
// Few rows a group: chunks of at most 16 NT rows.
//
// K is cut into slices of four 64-blocks, and slices into ranges of at most
// 8.  A workgroup holds one chunk, one range and a few tiles of 32 rows
// (16 where NT is 2) of the matrix, with a wave for each slice; the wave's slice of the chunk's
// activations, in fp16 under a power of two a row, stays in registers.
// v_mfma_f32_16x16x32_f16 takes k in any order that both operands share: lane
// (r, g) holds the pieces g and 4 + g of 32 weights of row r, so that a load
// takes 64 neighbouring bytes of a row and a piece has one scale.  The weights
// are multiplied by the scale in fp16, under a power of two that brings the
// largest of the row's four scales to [2^14, 2^15): one more rounding of 2^-11
// than a scale applied to fp32 sums would cost, which the four blocks of a
// product do not allow.  Held exactly, in two fp16 and two products, they took
// 13.1 -> 13.9 us (32 tokens, 11008 x 2048), 34 -> 40 (512 rows in 64 groups of
// 2048 x 1408), for 2.2e-4 -> 1.6e-4 of the outputs' magnitude; a bf16 output's
// own rounding is 1.7e-3.  The waves' tiles are added through LDS.
//
// Such calls are bound by their waits and by the instructions of a wave (four
// cycles each) more than by their bytes: nothing is cleared that a clamped
// address or a scale of 0 makes harmless; the codes (and the adapters' rows)
// of the first two tiles are asked for before anything else, and a tile's
// registers take the tile after next.  PRE: the activations were converted by
// an earlier launch, and lie in the order of the loads.
//
// Measured (graph replay, whole calls): 74 rows in 16 groups of 2048 x 1408,
// 25 MB, 13.6 us; 32 tokens beside adapters of rank 16 on 11008 x 2048, 23 MB,
// 13.1 us (4.8 and 4.4 us at the rate of a large copy).  K = 1408 makes six
// slices: two of the eight waves have none.
// ---------------------------------------------------------------------------
constexpr int kChunkWaves = 8;
constexpr int kSliceK = 256;

template <int NT, int MATS, bool PART, bool LORA, bool PRE>
__global__ __launch_bounds__(kChunkWaves * 64, NT * MATS == 1 && !LORA ? 4 : 2) void ragged_chunk_kernel(const Args a) {
    constexpr int CAP = 16 * NT;
    constexpr int H = NT == 2 ? 1 : 2;  // 16-row pieces of a tile
    constexpr int ROWS = 16 * H;
    constexpr int D = 2;                // tiles whose codes are held or on their way
    static_assert(CAP * ROWS == kChunkWaves * 64, "an output a thread");
    __shared__ uint32_t lut[kLutDwords];
    __shared__ float red[MATS][kChunkWaves][CAP * ROWS];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;

    const Share share = find_share(a.offsets, a.E, a.R, CAP, blockIdx.x, gridDim.x);
    const Chunk ck = share.chunk;
    const int nb = a.K >> 6;
    // Ranges take slices dealt evenly, the longer ones first.
    const int z = blockIdx.y;
    const int s0 = z * a.slices_each + min(z, a.slices_more), ns = a.slices_each + (z < a.slices_more ? 1 : 0);
    // This lane's two pieces of 32 k, and whether they lie within the row.
    const int pc[2] = {8 * (s0 + wave) + g, 8 * (s0 + wave) + 4 + g};
    const bool live[2] = {pc[0] < 2 * nb, pc[1] < 2 * nb};
    const bool whole = 8 * (s0 + wave) + 8 <= 2 * nb;
    const int at[2] = {min(pc[0], 2 * nb - 1), min(pc[1], 2 * nb - 1)};
    const int ntiles = (a.M + ROWS - 1) / ROWS;
    const int t0 = (int)((uint32_t)ntiles * share.part / share.nparts);
    const int t1 = (int)((uint32_t)ntiles * (share.part + 1) / share.nparts);
    if (ck.count == 0 || t0 == t1) return;
    // This thread's output of each tile: row p of Y, packed row `om` of the tile.
    const int orow = threadIdx.x / ROWS, om = threadIdx.x % ROWS, p = ck.start + min(orow, ck.count - 1);

    u32x4_t cw[D][MATS][H][2];          // [matrix][16 rows][piece]
    uint32_t sc[D][MATS][H][2];
    u32x4_t bw[D][2];                   // the first 16 ranks of B for this thread's output
    int id = -1;
    const uint16_t *brow = nullptr;
    if constexpr (LORA) {
        id = a.ids[p];
        if (id >= a.L) id = -1;
        brow = a.B + (int64_t)max(id, 0) * a.M * a.r;
    }
    auto load_tile = [&](int u, int t) {
#pragma unroll
        for (int q = 0; q < MATS; ++q) {
            const int64_t m0 = (int64_t)ck.e * a.M + t * ROWS;
            const uint8_t *cbase = a.codes[q] + m0 * (a.K >> 1);
            const uint16_t *sbase = a.scales[q] + m0 * nb;
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const uint32_t m = min(16 * h + col, a.M - 1 - t * ROWS);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    cw[u][q][h][j] = *reinterpret_cast<const u32x4_t *>(cbase + (m * (uint32_t)(a.K >> 1) + 16 * at[j]));
                    sc[u][q][h][j] = sbase[m * (uint32_t)nb + (at[j] >> 1)];
                }
            }
        }
        if constexpr (LORA) {
            const uint16_t *b = brow + (int64_t)min(t * ROWS + om, a.M - 1) * a.r;
            bw[u][0] = *reinterpret_cast<const u32x4_t *>(b);
            bw[u][1] = *reinterpret_cast<const u32x4_t *>(b + (a.r > 8 ? 8 : 0));
        }
    };
    u32x4_t x[NT][8];
    int back[NT][4];                    // the inverse power of two of each register's row, less 14
    // Pieces past the row have scales of 0, and zeros for x: the values that
    // their clamped addresses read could be infinite.
    auto cut = [&]() {
        if (whole) return;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int s = 0; s < 8; ++s)
                if (!live[s >> 2]) x[n][s] = u32x4_t{0u, 0u, 0u, 0u};
    };
    if constexpr (PRE) {
        // [piece of 8 k][position]: 16 lanes read 256 neighbouring bytes.
        const u32x4_t *src = reinterpret_cast<const u32x4_t *>(a.X) + ck.start;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = min(16 * n + col, ck.count - 1);
#pragma unroll
            for (int s = 0; s < 8; ++s) x[n][s] = src[(int64_t)(4 * at[s >> 2] + (s & 3)) * a.R + row];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                back[n][i] = a.xexp[(int64_t)(at[0] >> 3) * a.R + ck.start + min(16 * n + 4 * g + i, ck.count - 1)] - 14;
        }
#pragma unroll
        for (int u = 0; u < D; ++u) load_tile(u, min(t0 + u, t1 - 1));
        fill_lut(lut);
        cut();
    } else {
        int row[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) row[n] = max(source_row(a, ck.start + min(16 * n + col, ck.count - 1)), 0);
        load_tile(0, t0);
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int s = 0; s < 8; ++s) x[n][s] = u32x4_t{0u, 0u, 0u, 0u};
        if (a.T > 0) {
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const u32x4_t *src = reinterpret_cast<const u32x4_t *>(a.X + (int64_t)row[n] * a.K);
#pragma unroll
                for (int s = 0; s < 8; ++s) x[n][s] = src[4 * at[s >> 2] + (s & 3)];
            }
        }
#pragma unroll
        for (int u = 1; u < D; ++u) load_tile(u, min(t0 + u, t1 - 1));
        fill_lut(lut);
        cut();
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            u16x2_t mx = {0, 0};
#pragma unroll
            for (int s = 0; s < 8; ++s)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    mx = __builtin_elementwise_max(mx, __builtin_bit_cast(u16x2_t, x[n][s][c] & 0x7FFF7FFFu));
            int m = max((int)mx.x, (int)mx.y);
            m = max(m, __shfl_xor(m, 16));
            m = max(m, __shfl_xor(m, 32));
            const int shift = fp16_shift((uint32_t)m);
            const float f = exp2i(shift);
#pragma unroll
            for (int s = 0; s < 8; ++s)
#pragma unroll
                for (int c = 0; c < 4; ++c) x[n][s][c] = bf16x2_to_f16x2(x[n][s][c], f);
#pragma unroll
            for (int i = 0; i < 4; ++i) back[n][i] = -14 - __shfl(shift, 4 * g + i);
        }
    }
    float tv[16];                       // the first 16 of t for this thread's row
    if constexpr (LORA) {
#pragma unroll
        for (int i = 0; i < 16; ++i) tv[i] = id >= 0 && i < a.r ? a.t[(int64_t)p * a.r + i] : 0.0f;
    }
    __syncthreads();

    const uint32_t laneoff = (uint32_t)lane << 2;
    auto tile = [&](int u, int t) {
        float4_t d[MATS][H][NT];
        if (wave < ns) {
            int e[MATS][H];
            half2_t s2[MATS][H][2];
#pragma unroll
            for (int q = 0; q < MATS; ++q)
#pragma unroll
                for (int h = 0; h < H; ++h) {
                    const uint32_t bits[2] = {live[0] ? sc[u][q][h][0] : 0, live[1] ? sc[u][q][h][1] : 0};
                    int m = (int)max(bits[0] & 0x7FFFu, bits[1] & 0x7FFFu);
                    m = max(m, __shfl_xor(m, 16));
                    m = max(m, __shfl_xor(m, 32));
                    e[q][h] = m ? (int)(__builtin_bit_cast(uint32_t, f16_bits_to_f32((uint32_t)m)) >> 23) - 127 : 0;
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const _Float16 sh = (_Float16)ldexpf(f16_bits_to_f32(bits[j]), 14 - e[q][h]);
                        s2[q][h][j] = half2_t{sh, sh};
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) d[q][h][n] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
                }
            // A step of all matrices and pieces together: their lookups are
            // in flight at once, and their products are chains of their own.
#pragma unroll
            for (int s = 0; s < 8; ++s) {
                half2_t w[MATS][H][4];
#pragma unroll
                for (int q = 0; q < MATS; ++q)
#pragma unroll
                    for (int h = 0; h < H; ++h) lut8(lut, cw[u][q][h][s >> 2][s & 3], laneoff, w[q][h]);
#pragma unroll
                for (int q = 0; q < MATS; ++q)
#pragma unroll
                    for (int h = 0; h < H; ++h) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) w[q][h][c] *= s2[q][h][s >> 2];
#pragma unroll
                        for (int n = 0; n < NT; ++n)
                            d[q][h][n] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                                __builtin_bit_cast(half8_t, x[n][s]), join8(w[q][h]), d[q][h][n], 0, 0, 0);
                    }
            }
            // Register i of row tile n: row 16 n + 4 g + i, column 16 h + col.
#pragma unroll
            for (int q = 0; q < MATS; ++q)
#pragma unroll
                for (int h = 0; h < H; ++h)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            red[q][wave][(16 * n + 4 * g + i) * ROWS + 16 * h + col] =
                                ldexpf(d[q][h][n][i], e[q][h] + back[n][i]);
        }
        float term = 0.0f;
        if constexpr (LORA) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                if (h == 1 && a.r == 8) break;  // (8 ranks: the second half is the first again)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    term = fmaf(bf16_lo(bw[u][h][c]), tv[8 * h + 2 * c], term);
                    term = fmaf(bf16_hi(bw[u][h][c]), tv[8 * h + 2 * c + 1], term);
                }
            }
        }
        if (t + D < t1) load_tile(u, t + D);
        __syncthreads();
        const int mo = t * ROWS + om;
        if (orow < ck.count && mo < a.M) {
            float v[MATS];
#pragma unroll
            for (int q = 0; q < MATS; ++q) {
                v[q] = red[q][0][threadIdx.x];
#pragma unroll
                for (int w = 1; w < kChunkWaves; ++w)
                    if (w < ns) v[q] += red[q][w][threadIdx.x];
            }
            if (!PRE && source_row(a, p) < 0) {
#pragma unroll
                for (int q = 0; q < MATS; ++q) v[q] = 0.0f;
            }
            const int64_t o = (int64_t)p * a.M + mo;
            if constexpr (PART) {
#pragma unroll
                for (int q = 0; q < MATS; ++q) a.part[((int64_t)q * a.ranges + z) * a.R * a.M + o] = v[q];
            } else {
                float y = MATS == 2 ? swiglu(v[0], v[MATS - 1]) : v[0];
                if constexpr (LORA) {
                    if (id >= 0) y += term + adapter_term(a, id, p, mo, 16);
                }
                store_out(a.Y, a.bf16, o, y);
            }
        }
        __syncthreads();
    };
    for (int t = t0; t < t1; t += D) {
#pragma unroll
        for (int u = 0; u < D; ++u)
            if (t + u < t1) tile(u, t + u);
    }
}

// ---------------------------------------------------------------------------
// One row a group, mostly: every row of X by itself.
//
// A wave takes tiles of 8 packed rows (with MATS == 2 four of the gate and the
// same four of the up matrix) of one range of at most 2048 weights; a lane
// holds one piece of 32 weights of each row (1 KB of a row in one load) and
// the same 32 activations, in fp16 under a power of two a range, in registers.
// Table lookups feed v_dot2_f32_f16, the piece's scale multiplies its fp32
// sum, and the 8 rows' sums are added over the lanes together.  Waves do not
// wait for each other after the table is filled, and a row's registers take
// the next tile's row as soon as it is used: bound by the bytes of the codes,
// or by the launch and the waits before the first of them.  One token's 8
// experts of 1408 x 2048, gate and up, 24.5 MB: 9.0 us (2.7 TB/s; the chunk
// kernel 16.7).
// ---------------------------------------------------------------------------
constexpr int kRowTile = 8;
constexpr int kRowRangeK = 2048;

// Beside adapters (LORA) the last workgroups make t = s A x meanwhile, a wave
// a rank, and the launch that adds the planes has both.
template <int MATS, bool PART, bool LORA>
__global__ __launch_bounds__(512, 4) void ragged_row_kernel(const Args a) {
    constexpr int ROWS = kRowTile / MATS;
    static_assert(!LORA || PART, "t is made by the same launch");
    if constexpr (LORA) {
        if ((int)blockIdx.x >= a.wgs) {
            const int n = ((int)blockIdx.x - a.wgs) * ((int)blockDim.x >> 6) + ((int)threadIdx.x >> 6);
            if (blockIdx.y == 0) shrink_row(a.X, a.A, a.scaling, a.ids, a.K, a.K, a.r, a.L, n / a.r, n % a.r, a.R, a.tout);
            return;
        }
    }
    __shared__ uint32_t lut[kLutDwords];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int waves = blockDim.x >> 6;
    const int nb = a.K >> 6;
    const int z = blockIdx.y;
    const int first = z * (kRowRangeK / 32) + lane;
    const bool live = first < 2 * nb;
    const int piece = min(first, 2 * nb - 1);
    const int ntiles = (a.M * MATS + kRowTile - 1) / kRowTile;
    const Share share = find_share(a.offsets, a.E, a.R, 1, blockIdx.x, LORA ? a.wgs : (int)gridDim.x);
    const Chunk ck = share.chunk;
    int t = share.part * waves + wave;
    const int tstep = share.nparts * waves;
    if (ck.count == 0) return;

    u32x4_t cw[kRowTile];
    uint32_t sc[kRowTile];
    auto load = [&](int tile, int r) {
        const int q = r / ROWS, m = min(tile * ROWS + r % ROWS, a.M - 1);
        const int64_t mrow = (int64_t)ck.e * a.M + m;
        cw[r] = *reinterpret_cast<const u32x4_t *>(a.codes[q] + mrow * (a.K >> 1) + 16 * (uint32_t)piece);
        sc[r] = a.scales[q][mrow * nb + (piece >> 1)];
    };
    const int p = ck.start, row = source_row(a, p);
#pragma unroll
    for (int r = 0; r < kRowTile; ++r) load(min(t, ntiles - 1), r);
    u32x4_t xr[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
        xr[s] = u32x4_t{0u, 0u, 0u, 0u};
        if (row >= 0) xr[s] = reinterpret_cast<const u32x4_t *>(a.X + (int64_t)row * a.K + 32 * piece)[s];
    }
    fill_lut(lut);
    half2_t x[16];
    u16x2_t mx = {0, 0};
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int c = 0; c < 4; ++c)
            mx = __builtin_elementwise_max(mx, __builtin_bit_cast(u16x2_t, xr[s][c] & 0x7FFF7FFFu));
    const int shift = fp16_shift(wave_max_u32(mx.x > mx.y ? mx.x : mx.y));
    const float f = exp2i(shift);
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
        for (int c = 0; c < 4; ++c) x[4 * s + c] = __builtin_bit_cast(half2_t, bf16x2_to_f16x2(xr[s][c], f));
    __syncthreads();

    const uint32_t laneoff = (uint32_t)lane << 2;
    for (; t < ntiles; t += tstep) {
        const int mo = t * ROWS + (lane & (ROWS - 1));
        float v[kRowTile];
#pragma unroll
        for (int r = 0; r < kRowTile; ++r) {
            float d0 = 0.0f, d1 = 0.0f;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                half2_t w[4];
                lut8(lut, cw[r][c], laneoff, w);
                d0 = __builtin_amdgcn_fdot2(w[0], x[4 * c], d0, false);
                d1 = __builtin_amdgcn_fdot2(w[1], x[4 * c + 1], d1, false);
                d0 = __builtin_amdgcn_fdot2(w[2], x[4 * c + 2], d0, false);
                d1 = __builtin_amdgcn_fdot2(w[3], x[4 * c + 3], d1, false);
            }
            v[r] = live ? f16_bits_to_f32(sc[r]) * (d0 + d1) : 0.0f;
            if (t + tstep < ntiles) load(t + tstep, r);
        }
        float total = ldexpf(reduce_rows<kRowTile>(v), -shift);  // of row lane % 8
        const int64_t at = (int64_t)p * a.M + mo;
        if constexpr (PART) {
            const int q = (lane & (kRowTile - 1)) / ROWS;
            if (lane < kRowTile && mo < a.M) a.part[((int64_t)q * a.ranges + z) * a.R * a.M + at] = total;
        } else {
            if constexpr (MATS == 2) total = swiglu(total, __shfl_xor(total, ROWS));
            if (lane < ROWS && mo < a.M) store_out(a.Y, a.bf16, at, total);
        }
    }
}

__global__ __launch_bounds__(256) void ragged_pieces_kernel(const uint16_t *__restrict__ X,
                                                            const int32_t *__restrict__ rows, int K, int T, int R,
                                                            Pieces out) {
    write_pieces(X, rows, K, T, R, out, blockIdx.x);
}

// Adds the partial planes in range order and finishes the outputs.
template <int MATS, bool LORA>
__global__ __launch_bounds__(256) void ragged_finish_kernel(const Args a) {
    const int per = (a.M + 255) >> 8;
    const int p = blockIdx.x / per, m = (blockIdx.x % per) * 256 + threadIdx.x;
    if (a.offsets) {
        // A position outside every group has no planes, and keeps its row.
        bool in = false;
        for (int e = threadIdx.x & 63; e < a.E; e += 64)
            in = in || (p >= min(max(a.offsets[e], 0), a.R) && p < min(max(a.offsets[e + 1], 0), a.R));
        if (__builtin_amdgcn_ballot_w64(in) == 0) return;
    }
    if (m >= a.M) return;
    const int64_t at = (int64_t)p * a.M + m, plane = (int64_t)a.R * a.M;
    float v[MATS];
#pragma unroll
    for (int q = 0; q < MATS; ++q) {
        const float *s = a.part + (int64_t)q * a.ranges * plane + at;
        v[q] = s[0];
        for (int z = 1; z < a.ranges; ++z) v[q] += s[z * plane];
    }
    float y = MATS == 2 ? swiglu(v[0], v[MATS - 1]) : v[0];
    if constexpr (LORA) y += adapter_term(a, a.ids[p], p, m);
    store_out(a.Y, a.bf16, at, y);
}

// ---------------------------------------------------------------------------
// Many rows a group.
// ---------------------------------------------------------------------------

// The tile kernel takes two 64-blocks at a time: its rows of X are padded to
// that with zeros, so that the step past an odd row adds zeros (what it met in
// place of them, times a scale of 0, would make NaN of an infinity).
__host__ __device__ constexpr int64_t tile_pitch(int64_t K) { return (K + 127) & ~(int64_t)127; }

// One workgroup a row of X: fp16 under a power of two (the row's largest
// magnitude goes to [2^14, 2^15)), and that power of two.  The workgroups
// behind them take 16 packed rows each: the exponent of a row's largest scale,
// and its scales under it, so that the lanes of a tile, which hold neighbouring
// rows, read neighbouring scales (from rows of K / 64 they would take a line
// each, 13% of the time of 4096 x 8192 x 8192).
__global__ __launch_bounds__(256) void ragged_prepare_kernel(const uint16_t *__restrict__ X, int T, int K,
                                                             uint16_t *__restrict__ x16, int32_t *__restrict__ xexp,
                                                             const uint16_t *__restrict__ s0,
                                                             const uint16_t *__restrict__ s1, int M, int64_t nrows,
                                                             int8_t *__restrict__ e0, int8_t *__restrict__ e1,
                                                             uint16_t *__restrict__ t0, uint16_t *__restrict__ t1) {
    __shared__ uint32_t wmax[4];
    if ((int)blockIdx.x < T) {
        const u32x4_t *src = reinterpret_cast<const u32x4_t *>(X + (int64_t)blockIdx.x * K);
        u32x4_t *dst = reinterpret_cast<u32x4_t *>(x16 + (int64_t)blockIdx.x * tile_pitch(K));
        const int n = K / 8;
        u16x2_t mx = {0, 0};
        for (int i = threadIdx.x; i < n; i += 256) {
            const u32x4_t v = src[i];
#pragma unroll
            for (int c = 0; c < 4; ++c)
                mx = __builtin_elementwise_max(mx, __builtin_bit_cast(u16x2_t, v[c] & 0x7FFF7FFFu));
        }
        const uint32_t m = wave_max_u32(mx.x > mx.y ? mx.x : mx.y);
        if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
        __syncthreads();
        const int shift = fp16_shift(max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3])));
        const float f = exp2i(shift);
        for (int i = threadIdx.x; i < n; i += 256) {
            u32x4_t v = src[i];
#pragma unroll
            for (int c = 0; c < 4; ++c) v[c] = bf16x2_to_f16x2(v[c], f);
            dst[i] = v;
        }
        if (threadIdx.x < (uint32_t)(tile_pitch(K) - K) / 8) dst[n + threadIdx.x] = u32x4_t{0u, 0u, 0u, 0u};
        if (threadIdx.x == 0) xexp[blockIdx.x] = -shift;
        return;
    }
    const int64_t row0 = ((int64_t)blockIdx.x - T) * 16;
#pragma unroll
    for (int q = 0; q < 2; ++q)
        if (q ? s1 : s0) prepare_scales<0>(q ? s1 : s0, row0, nrows, M, K >> 6, q ? e1 : e0, q ? t1 : t0);
}

constexpr int kTileWaves = 8;

// A workgroup computes 64 MT rows of X (2 waves of MT tiles of 32) by 256
// packed rows (4 waves of two 32-row tiles; with MATS == 2 each wave's tiles
// are the gate's and the up's same 32 rows), 64 k a step.  X goes through LDS
// in two buffers; each wave looks its own weights up and multiplies them by
// the block's scale in fp16.
//
// The matrix cores bound it where nothing of a step is waited for: a step's
// rows of X go from registers to the free buffer while the step before it is
// multiplied, the loads of the step after take their place, and the lookups of
// a quarter step (16 k a lane group) are under way during the products of the
// quarter before, the last quarter's across the barrier.
//
// Measured (cards differ): 4093 tokens beside adapters of rank 64 on 11008 x
// 2048 264-277 us, of which 251 here (191 GFLOP: 760 TFLOP/s; a library fp16
// product of 8192^3 reaches 1450); 32768 rows in 64 groups of 1408 x 2048, gate
// and up, 526-550 us (690-720 TFLOP/s, ragged last pieces among them).  What is
// left is the lookups'
// and scalings' instructions beside the products, and the clock that the
// power of both allows, and in ragged last pieces the rows that are not there:
// all 32-row tiles are multiplied.  The scaled weights are rounded to fp16 as in
// the chunk kernel; held exactly, in two products, the same calls took 381 and
// 807 us.  Not faster: 16 waves a workgroup (310 us where 8 took
// 278), waves of other corners of the tile (618 against 555), codes through
// LDS (spills), 16-bit results of two rows stored together (+35 us).
template <int MT, bool LORA>
struct TileShared {
    uint32_t lut[kLutDwords];  // first: its address is 0, and a lookup's the code byte and the lane
    u32x4_t xs[2][64 * MT * 8];
    int xe[64 * MT];
    int sid[LORA ? 64 * MT : 1];
};

// PART: a workgroup takes one of a.ranges runs of 64-blocks (blockIdx.y) and
// writes fp32 sums to that run's plane, the adapters' term with the first.
template <int MT, int MATS, bool LORA, bool PART>
__global__ __launch_bounds__(kTileWaves * 64) void ragged_tile_kernel(const Args a) {
    constexpr int TM = 64 * MT;
    constexpr int kRowsWg = MATS == 2 ? 128 : 256;
    constexpr int kPieces = TM * 8 / (kTileWaves * 64);  // 16-byte pieces of X a thread stages
    __shared__ TileShared<MT, LORA> sm;
    int (&xe)[TM] = sm.xe;
    auto &sid = sm.sid;
    const uint32_t *lut = sm.lut;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, g = lane >> 5;
    const int wt = wave & 1, wr = wave >> 1;

    // Workgroups go round the 8 XCDs; each XCD takes a run of the (chunk, row
    // tile) pairs, so that a chunk's rows stay in one L2.
    const int total = __builtin_amdgcn_readfirstlane(count_chunks(a.offsets, a.E, a.R, TM)) * a.rowtiles;
    const int each = (total + 7) >> 3, at = (int)(blockIdx.x & 7) * each + (int)(blockIdx.x >> 3);
    if ((int)(blockIdx.x >> 3) >= each || at >= total) return;
    const int rt0 = at % a.rowtiles;
    const Chunk ck = find_chunk(a.offsets, a.E, a.R, at / a.rowtiles, TM);

    // A row outside [0, T) reads row 0 and is put out as zeros (kNoRow).
    constexpr int kNoRow = -1000000;
    for (int i = threadIdx.x; i < TM; i += kTileWaves * 64) {
        const int row = i < ck.count ? source_row(a, ck.start + i) : -1;
        xe[i] = row >= 0 ? a.xexp[row] : kNoRow;
        if constexpr (LORA) {
            const int id = i < ck.count ? a.ids[ck.start + i] : -1;
            sid[i] = id >= 0 && id < a.L ? id : -1;
        }
    }
    // Staging of X: piece j of this thread is row threadIdx / 8 + 64 j, slot
    // threadIdx % 8, which holds the row's 16-byte piece slot ^ (row / 2 % 8): the
    // 16 rows that LDS serves at once then meet all 64 banks.
    const u32x4_t *xsrc[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        const int i = (threadIdx.x >> 3) + 64 * j;
        const int row = max(source_row(a, ck.start + min(i, ck.count - 1)), 0);
        const int piece = (threadIdx.x & 7) ^ ((i >> 1) & 7);
        xsrc[j] = reinterpret_cast<const u32x4_t *>(a.X + row * tile_pitch(a.K)) + piece;
    }

    int m[2];
    const u32x4_t *csrc[2];
    const uint16_t *ssrc[2];
    int e[2];
    // Runs of pairs of blocks: only the last may end in an odd one.
    const int pairs = (a.K + 127) >> 7;
    const int b0 = PART ? 2 * (pairs * (int)blockIdx.y / a.ranges) : 0;  // the first block
    const int nb = (PART ? min(2 * (pairs * ((int)blockIdx.y + 1) / a.ranges), a.K >> 6) : a.K >> 6) - b0;
    const int nbx = (nb + 1) & ~1;                                       // with the padding of X
    if constexpr (PART) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) xsrc[j] += 8 * b0;
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int mat = MATS == 2 ? q : 0;
        m[q] = rt0 * kRowsWg + (MATS == 2 ? wr * 32 : wr * 64 + q * 32) + col;
        const int64_t mrow = (int64_t)ck.e * a.M + min(m[q], a.M - 1);
        csrc[q] = reinterpret_cast<const u32x4_t *>(a.codes[mat] + mrow * (a.K >> 1)) + g + 2 * b0;
        ssrc[q] = a.tscale[mat] + ((int64_t)ck.e * (a.K >> 6) + b0) * a.M + min(m[q], a.M - 1);
        e[q] = a.rowexp[mat][mrow];
    }

    // Codes and scales of even and of odd steps: a set is loaded for the step
    // after next as soon as it is used up (and never copied, which would wait
    // for the loads).
    u32x4_t xv[kPieces], c0[2], c1[2];
    uint32_t v0[2], v1[2];
    auto load_x = [&](int b) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) xv[j] = __builtin_nontemporal_load(xsrc[j] + 8 * b);  // (read once)
    };
    auto load_codes = [&](int b, u32x4_t (&cd)[2], uint32_t (&sd)[2]) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            cd[q] = csrc[q][2 * b];
            sd[q] = ssrc[q][(int64_t)b * a.M];
        }
    };
    auto stage = [&](int b) {
        u32x4_t *buf = sm.xs[b & 1];
#pragma unroll
        for (int j = 0; j < kPieces; ++j) buf[threadIdx.x + 512 * j] = xv[j];
    };
    load_x(0);
    load_codes(0, c0, v0);
    load_codes(min(1, nb - 1), c1, v1);
    fill_lut(sm.lut);
    stage(0);
    load_x(1);

    float16_t acc[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q) acc[i][q] = float16_t{};
    const uint32_t laneoff = (uint32_t)lane << 2;

    // A quarter step's weights (lookups, then the scale) and its rows of X.
    half2_t raw[2][4];
    half2_t s2[2];
    u32x4_t xa[2][MT];
    auto look = [&](const u32x4_t (&cd)[2], int s) {
#pragma unroll
        for (int q = 0; q < 2; ++q) lut8(lut, cd[q][s], laneoff, raw[q]);
    };
    auto scale = [&](int b, const uint32_t (&sd)[2]) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t h = b < nb ? sd[q] : 0;
            s2[q] = __builtin_bit_cast(half2_t, h | h << 16);
        }
    };
    auto rows = [&](int b, int s) {
        const u32x4_t *buf = sm.xs[b & 1] + (wt * 32 * MT + col) * 8 + ((4 * g + s) ^ ((col >> 1) & 7));
#pragma unroll
        for (int i = 0; i < MT; ++i) xa[s & 1][i] = buf[32 * 8 * i];
    };
    half8_t w[2];
    auto weigh = [&]() {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
#pragma unroll
            for (int i = 0; i < 4; ++i) raw[q][i] *= s2[q];
            w[q] = join8(raw[q]);
        }
    };
    // Step b on the codes `cd`, with those of the next in `cnext`; its first
    // weights and rows were made by the step before.
    auto step = [&](int b, u32x4_t (&cd)[2], uint32_t (&sd)[2], const u32x4_t (&cnext)[2],
                    const uint32_t (&snext)[2]) {
        // (The last steps stage and load what is there already.)
        stage(b + 1);
        load_x(min(b + 2, nbx - 1));
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            const half8_t wn[2] = {w[0], w[1]};
            if (s < 3) {
                look(cd, s + 1);
                rows(b, s + 1);
            } else {
                // Every wave has staged step b + 1, and has this step's last rows.
                __syncthreads();
                load_codes(min(b + 2, nb - 1), cd, sd);
                scale(b + 1, snext);
                look(cnext, 0);
                rows(b + 1, 0);
            }
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const half8_t x = __builtin_bit_cast(half8_t, xa[s & 1][i]);
                acc[i][0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, wn[0], acc[i][0], 0, 0, 0);
                acc[i][1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(x, wn[1], acc[i][1], 0, 0, 0);
            }
            weigh();
            // In the shadow of each product: lookups and rows of the next
            // quarter beside the first half of them, their scales beside the
            // second.
#pragma unroll
            for (int k = 0; k < MT; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);            // a product
                __builtin_amdgcn_sched_group_barrier(0x002, 8 / MT, 0);       // addresses
                __builtin_amdgcn_sched_group_barrier(0x100, 8 / MT + 1, 0);   // LDS reads
                if (s == 0) {
                    __builtin_amdgcn_sched_group_barrier(0x200, 1, 0);        // staging
                    __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
                }
            }
#pragma unroll
            for (int k = 0; k < MT; ++k) {
                __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                if (s == 3) __builtin_amdgcn_sched_group_barrier(0x002, 8 / MT + 2, 0);
                else __builtin_amdgcn_sched_group_barrier(0x002, 8 / MT, 0);
            }
        }
    };
    __syncthreads();
    scale(0, v0);
    look(c0, 0);
    rows(0, 0);
    weigh();
    // (The step past an odd last one has scales of 0, and zeros for X.)
    for (int b = 0; b < nb; b += 2) {
        step(b, c0, v0, c1, v1);
        step(b + 1, c1, v1, c0, v0);
    }
    __syncthreads();

#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int x = xe[wt * 32 * MT + 32 * i + tile_row(j, lane)];
            acc[i][0][j] = x == kNoRow ? 0.0f : ldexpf(acc[i][0][j], x - 14 + e[0]);
            acc[i][1][j] = x == kNoRow ? 0.0f : ldexpf(acc[i][1][j], x - 14 + e[1]);
        }

    bool wild = false;  // an adapter of this wave's rows holds a value that is not finite
    if constexpr (LORA) {
        // The adapters among this wave's rows, one after the other; the rows
        // of others enter as zeros.
        int mine[2] = {-1, -1};
        const int w0 = wt * 32 * MT;
        if (lane < 32 * MT) mine[0] = sid[w0 + lane];
        if (MT == 4) mine[1] = sid[w0 + 64 + lane];
        while (!PART || blockIdx.y == 0) {
            const uint64_t p0 = __builtin_amdgcn_ballot_w64(mine[0] >= 0);
            const uint64_t p1 = __builtin_amdgcn_ballot_w64(mine[1] >= 0);
            if (!(p0 | p1)) break;
            const int id = p0 ? __builtin_amdgcn_readlane(mine[0], __builtin_ctzll(p0))
                              : __builtin_amdgcn_readlane(mine[1], __builtin_ctzll(p1));
            if (mine[0] == id) mine[0] = -1;
            if (mine[1] == id) mine[1] = -1;
            for (int j0 = 0; j0 < a.r; j0 += 16) {
                const bool live = j0 + 8 * g < a.r;
                u32x4_t bb[2];
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    bb[q] = u32x4_t{0u, 0u, 0u, 0u};
                    if (live && m[q] < a.M)
                        bb[q] = *reinterpret_cast<const u32x4_t *>(a.B + ((int64_t)id * a.M + m[q]) * a.r + j0 + 8 * g);
                }
                if (__builtin_amdgcn_ballot_w64(not_finite8(bb[0]) || not_finite8(bb[1]))) {
                    wild = true;
                    bb[0] = finite8(bb[0]);
                    bb[1] = finite8(bb[1]);
                }
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const int row = w0 + 32 * i + col;
                    const bool use = sid[row] == id;
                    if (__builtin_amdgcn_ballot_w64(use) == 0) continue;
                    float t[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) t[x] = 0.0f;
                    if (use && live) {
                        const float *src = a.t + (int64_t)(ck.start + row) * a.r + j0 + 8 * g;
#pragma unroll
                        for (int x = 0; x < 8; ++x) t[x] = src[x];
                    }
                    bf16x8_t hi, lo;
                    split2(t, hi, lo);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const bf16x8_t b = __builtin_bit_cast(bf16x8_t, bb[q]);
                        acc[i][q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(hi, b, acc[i][q], 0, 0, 0);
                        acc[i][q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(lo, b, acc[i][q], 0, 0, 0);
                    }
                }
            }
        }
    }

#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int row = wt * 32 * MT + 32 * i + tile_row(j, lane);
            if (row >= ck.count) continue;
            const int64_t at = (int64_t)(ck.start + row) * a.M;
            if constexpr (PART) {
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const int64_t plane = (MATS == 2 ? q * a.ranges : 0) + (int)blockIdx.y;
                    if (m[q] < a.M) a.part[plane * a.R * a.M + at + m[q]] = acc[i][q][j];
                }
            } else if constexpr (MATS == 2) {
                if (m[0] < a.M) store_out(a.Y, a.bf16, at + m[0], swiglu(acc[i][0][j], acc[i][1][j]));
            } else {
                if (m[0] < a.M) store_out(a.Y, a.bf16, at + m[0], acc[i][0][j]);
                if (m[1] < a.M) store_out(a.Y, a.bf16, at + m[1], acc[i][1][j]);
            }
        }
    if constexpr (LORA) {
        if (!wild) return;
        // (Every lane adds to the outputs that it has stored.)
        const int w0 = wt * 32 * MT;
        for (int i = 0; i < 16 * MT; ++i) {
            const int row = w0 + 32 * (i >> 4) + tile_row(i & 15, lane);
            if (row >= ck.count || sid[row] < 0) continue;
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if (m[q] >= a.M) continue;
                const float y = wild_term(a.t + (int64_t)(ck.start + row) * a.r,
                                          a.B + ((int64_t)sid[row] * a.M + m[q]) * a.r, 1, a.r);
                if (y == 0.0f) continue;
                const int64_t at = (int64_t)(ck.start + row) * a.M + m[q];
                if constexpr (PART) a.part[at] += y;  // (the first plane)
                else store_out(a.Y, a.bf16, at, load_out(a.Y, a.bf16, at) + y);
            }
        }
    }
}

int64_t slices_of(int64_t K) { return (K + kSliceK - 1) / kSliceK; }

// How a call runs.
struct Plan {
    bool single;  // row kernel
    bool tiles;   // tile kernel (else chunk kernel)
    int mt;       // tile kernel: 32-row tiles a wave
    int cap;      // chunk kernel: rows a chunk
    bool pre;     // chunk kernel: the activations are converted by a launch before
    int ranges;   // ranges of K, each with planes of partial sums (1: none but beside the row kernel's adapters)
};

// Chunks of `most` rows that R rows in E groups can make at most.
int64_t chunk_bound(int64_t E, int64_t R, int64_t most) {
    const int64_t a = E == 1 ? (R + most - 1) / most : R / most + E;
    return a < R ? a : R;
}

// The rules, with what both sides take in us: E x M x K, "up" where there is
// an up matrix; r ranks of adapters, 0 without.  Their costs were measured on
// the 256 compute units of an MI355X and count those; a size of a workspace
// has to follow from the shape alone.
Plan plan_of(int64_t E, int64_t M, int64_t K, int64_t R, bool up, int64_t r) {
    Plan p = {};
    const int64_t groups = E < R ? E : R;
    const int64_t avg = groups ? (R + groups - 1) / groups : 0;  // rows a group, were all in use equally full
    // Chunks of `most` rows that are likely: half a chunk a group is empty.
    auto chunks = [&](int64_t most) {
        const int64_t n = E == 1 ? (R + most - 1) / most : (2 * R + groups * most) / (2 * most);
        return n > groups ? n : groups;
    };
    // The row kernel reads a group's codes for each row, but waits for less:
    // row | chunk for 64 x 1408 x 2048 up, R = 8 9.1 | 16.7, 32 23.1 | 34.5,
    // 64 36.1 | 45.1, 80 44.6 | 45.1, 96 51.9 | 44.6, 192 108 | 56; 16 x 2048 x
    // 4096 up, R = 16 32.7 | 36.2, 24 45.7 | 47.0, 32 53.8 | 51.8; 8 x 1408 x 2048
    // up, R = 8 8.9 | 16.8, 16 14.7 | 16.9; 64 x 2048 x 1408, R = 16 9.3 | 12.9, 32
    // 16.2 | 18.6, 40 20.4 | 18.4, 48 21.8 | 18.4; 16 x 2048 x 4096, R = 8 13.2 |
    // 17.3, 12 19.7 | 18.3; 8 x 2048 x 4096, R = 4 9.4 | 14.8, 16 21.4 | 17.6;
    // 1 x 4096 x 4096, R = 2 10.4 | 11.0, 8 20.6 | 11.4.  (The sides meet between
    // E and 2 E with an up matrix, between E / 2 and E without.)
    p.single = R <= 2 || R <= (up ? E : E / 2);
    // Chunks of 16 rows | 32: with two matrices, 64 x 1408 x 2048 up, R = 256
    // (4 a group) 56.2 | 58.8, 512 86.8 | 76.0, 1024 125 | 101.  With one, a
    // compute unit holds two workgroups of 16 and one of 32, which pays where
    // one group's codes would be read twice: 1 x 4096 x 4096, R = 32
    // 17.2 | 13.4, 16 10.9 | 11.6; 64 x 2048 x 1408, R = 512 32 | 46, 2048 62 | 83.
    p.cap = (up ? avg < 8 : E > 1 || R <= 16) ? 16 : 32;
    // The chunk kernel's time goes with chunks x M, the tile kernel's (with 64
    // or 128 rows for each of two waves, mt 2 or 4) with the times that its
    // workgroups fill the 256 compute units, each a walk along K: in units of
    // 1.8 ps for 64 weights of K (a us is 35.8e6 / K of them).  Chunk | mt 2 |
    // mt 4 for 1 x 11008 x 2048, R = 128 30 | 51 | 67, 256 52 | 53 | 71, 512 93 | 55 | 72, 1024 - | 101 | 78,
    // 4096 - | 290 | 228; 64 x 1408 x 2048 up, R = 1024 101 | - | -, 2048 146 | 149 |
    // 205, 4096 285 | 191 | 217, 16384 809 | 340 | 355, 32768 - | 615 | 524.
    const int64_t mats = up ? 2 : 1, rowtiles = (M * mats + 255) / 256;
    const int64_t full2 = (chunks(128) * rowtiles + 255) / 256, full4 = (chunks(256) * rowtiles + 255) / 256;
    p.mt = 3 * full4 <= 2 * full2 ? 4 : 2;
    int64_t tile_cost = 392000 * (2 * full2 < 3 * full4 ? 2 * full2 : 3 * full4) + 143000000 / K;
    // Workgroups that leave half of the compute units empty share the walk
    // along K, at the price of the planes' bytes and of the launch that adds
    // them (8 us more).  Chunk | 1 run | 2 | 4 | 8 for 1 x 2048 x 11008, R = 256
    // 54 | 207 | 120 | 77 | 56, 1024 219 | 220 | 142 | 111 | -; 1 x 4096 x 4096
    // of rank 64, R = 128 34 | 96 | 67 | 51 | 44, 512 104 | 105 | 79 | 69 | -;
    // 1 x 2048 x 2048, R = 512 25 | 50 | 41 | 36 | 36; 1 x 11008 x 2048, R = 256
    // 52 | 53 | 44 | - | -.
    const int64_t wgs = chunks(128) * rowtiles;
    int splits = 1;
    for (int64_t s = 2; s <= 16 && wgs * s <= 256 && K / 64 >= 4 * s; ++s) {
        const int64_t cost = 700000 / s + (R * M * mats * s * 60 + 430000000) / K;
        if (cost < tile_cost) {
            tile_cost = cost;
            splits = (int)s;
        }
    }
    // (Ranks past 16 are products on the vector units in the chunk kernel, and
    // on the matrix units in the tile kernel: 1 x 11008 x 2048 of rank 64, R =
    // 192 84 | 60.)
    const int64_t chunk_cost =
        chunks(p.cap) * M * mats * (p.cap == 16 ? 4 : 9) + (r > 16 ? R * M * (r - 16) * 15 / K : 0);
    p.tiles = !p.single && avg > 32 &&
              (avg > 1024 || chunk_cost > tile_cost || (M + 255) / 256 * R >= INT64_C(1) << 24);
    // A launch that converts the activations first, against a conversion in
    // every workgroup: not | first for chunks of 32, 64 x 1408 x 2048 up, R =
    // 512 79.0 | 76.0, 1024 105 | 101, 1 x 4096 x 4096, R = 32 14.3 | 13.4; of
    // 16, 64 x 2048 x 1408, R = 48 17.5 | 19.6, 512 32.0 | 34.2.  Adapters
    // have a launch before the product anyhow, and it does both.
    p.pre = !p.single && !p.tiles && (r > 0 || p.cap == 32);
    p.ranges = p.tiles    ? splits
               : p.single ? (int)((K + kRowRangeK - 1) / kRowRangeK)
                          : (int)((slices_of(K) + kChunkWaves - 1) / kChunkWaves);
    if (p.tiles && splits > 1) p.mt = 2;
    return p;
}

// The tile kernel's rows of X in fp16: one at least, which rows outside [0, T) read.
size_t tile_rows_bytes(int64_t T, int64_t K) { return (size_t)(T > 0 ? T : 1) * tile_pitch(K) * 2; }

}  // namespace

int compute_units() {
    int dev = 0, n = 0;
    if (hipGetDevice(&dev) != hipSuccess ||
        hipDeviceGetAttribute(&n, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || n < 1)
        return 256;
    return n;
}

bool ragged_fits(int64_t E, int64_t M, int64_t K, int64_t T, int64_t R, bool up) {
    const Plan p = plan_of(E, M, K, R, up, 0);
    const int64_t most = INT64_C(1) << 32;  // threads of one launch
    if (p.tiles) {
        const int64_t rowtiles = (M + (up ? 127 : 255)) / (up ? 128 : 256);
        return (T + (E * M + 15) / 16) * 256 < most && rowtiles * chunk_bound(E, R, 64 * p.mt) * 512 < most;
    }
    return ((M + 255) / 256) * R * 256 < most && chunk_bound(E, R, p.single ? 1 : p.cap) < 65536 &&
           (!p.pre || pieces_blocks(K, R) * 256 < most);
}

size_t ragged_ws_bytes(int64_t E, int64_t M, int64_t K, int64_t T, int64_t R, bool up, int64_t r) {
    const Plan p = plan_of(E, M, K, R, up, r);
    const size_t mats = up ? 2 : 1;
    if (p.tiles)
        return tile_rows_bytes(T, K) + round16((size_t)T * 4) +
               mats * (round16((size_t)E * M) + round16((size_t)E * M * (K / 64) * 2)) +
               (p.ranges > 1 ? mats * p.ranges * (size_t)R * M * 4 : 0);
    return (p.pre ? pieces_bytes(K, R) : 0) + (p.ranges > 1 || (p.single && r > 0) ? mats * p.ranges * (size_t)R * M * 4 : 0);
}

bool ragged_takes_pieces(int64_t E, int64_t M, int64_t K, int64_t R, int64_t r) {
    return plan_of(E, M, K, R, false, r).pre;
}

bool ragged_shrinks(int64_t E, int64_t M, int64_t K, int64_t R, int64_t r) {
    return plan_of(E, M, K, R, false, r).single;
}

template <int MT, bool PART>
static const void *tile_fn(bool up, bool lora) {
    if (up) return reinterpret_cast<const void *>(&ragged_tile_kernel<MT, 2, false, PART>);
    return lora ? reinterpret_cast<const void *>(&ragged_tile_kernel<MT, 1, true, PART>)
                : reinterpret_cast<const void *>(&ragged_tile_kernel<MT, 1, false, PART>);
}

static const void *row_fn(bool up, bool part, bool lora) {
    if (up)
        return part ? reinterpret_cast<const void *>(&ragged_row_kernel<2, true, false>)
                    : reinterpret_cast<const void *>(&ragged_row_kernel<2, false, false>);
    if (lora) return reinterpret_cast<const void *>(&ragged_row_kernel<1, true, true>);
    return part ? reinterpret_cast<const void *>(&ragged_row_kernel<1, true, false>)
                : reinterpret_cast<const void *>(&ragged_row_kernel<1, false, false>);
}

template <int NT, bool PRE>
static const void *chunk_fn(bool up, bool part, bool lora) {
    // Chunks of 16 rows converted before are those beside adapters, and have one matrix.
    if constexpr (NT == 2 || !PRE)
        if (up)
            return part ? reinterpret_cast<const void *>(&ragged_chunk_kernel<NT, 2, true, false, PRE>)
                        : reinterpret_cast<const void *>(&ragged_chunk_kernel<NT, 2, false, false, PRE>);
    if (part) return reinterpret_cast<const void *>(&ragged_chunk_kernel<NT, 1, true, false, PRE>);
    if constexpr (PRE)
        if (NT == 1 || lora) return reinterpret_cast<const void *>(&ragged_chunk_kernel<NT, 1, false, true, true>);
    if constexpr (NT == 2 || !PRE) return reinterpret_cast<const void *>(&ragged_chunk_kernel<NT, 1, false, false, PRE>);
}

// Adds the planes (and, with lora, the adapters' terms).
static hipError_t launch_finish(Args a, bool up, bool lora, hipStream_t stream) {
    const void *fin = up     ? reinterpret_cast<const void *>(&ragged_finish_kernel<2, false>)
                      : lora ? reinterpret_cast<const void *>(&ragged_finish_kernel<1, true>)
                             : reinterpret_cast<const void *>(&ragged_finish_kernel<1, false>);
    void *args[] = {&a};
    return hipLaunchKernel(fin, dim3((unsigned)(((int64_t)a.M + 255) / 256 * a.R)), dim3(256), args, 0, stream);
}

hipError_t launch_ragged(const RaggedProduct &p, void *workspace, hipStream_t stream) {
    const bool up = p.up_codes != nullptr, lora = p.B != nullptr;
    const Plan pl = plan_of(p.E, p.M, p.K, p.R, up, lora ? p.r : 0);
    Args a = {};
    a.codes[0] = p.codes;
    a.codes[1] = p.up_codes;
    a.scales[0] = p.scales;
    a.scales[1] = p.up_scales;
    a.M = (int)p.M;
    a.K = (int)p.K;
    a.E = (int)p.E;
    a.R = (int)p.R;
    a.X = p.X;
    a.T = (int)p.T;
    a.offsets = p.offsets;
    a.rows = p.rows;
    a.Y = p.Y;
    a.bf16 = p.bf16;
    a.B = p.B;
    a.t = p.t;
    a.ids = p.ids;
    a.r = (int)p.r;
    a.L = (int)p.L;
    a.A = p.A;
    a.scaling = p.scaling;
    a.tout = const_cast<float *>(p.t);
    void *args[] = {&a};
    if (pl.tiles) {
        char *w = static_cast<char *>(workspace);
        uint16_t *x16 = reinterpret_cast<uint16_t *>(w);
        w += tile_rows_bytes(p.T, p.K);
        int32_t *xexp = reinterpret_cast<int32_t *>(w);
        w += round16((size_t)p.T * 4);
        const size_t eb = round16((size_t)p.E * p.M), sb = round16((size_t)p.E * p.M * (p.K / 64) * 2);
        int8_t *re0 = reinterpret_cast<int8_t *>(w), *re1 = up ? re0 + eb : nullptr;
        w += eb * (up ? 2 : 1);
        uint16_t *ts0 = reinterpret_cast<uint16_t *>(w), *ts1 = up ? reinterpret_cast<uint16_t *>(w + sb) : nullptr;
        int64_t nrows = p.E * p.M;
        int T = a.T, K = a.K, M = a.M;
        const uint16_t *X = p.X, *s0 = p.scales, *s1 = p.up_scales;
        void *pargs[] = {&X, &T, &K, &x16, &xexp, &s0, &s1, &M, &nrows, &re0, &re1, &ts0, &ts1};
        const int64_t blocks = p.T + (nrows + 15) / 16;
        hipError_t e = hipLaunchKernel(reinterpret_cast<const void *>(&ragged_prepare_kernel), dim3((unsigned)blocks),
                                       dim3(256), pargs, 0, stream);
        if (e != hipSuccess) return e;
        a.X = x16;
        a.xexp = xexp;
        a.rowexp[0] = re0;
        a.rowexp[1] = re1;
        a.tscale[0] = ts0;
        a.tscale[1] = ts1;
        const int rows_wg = up ? 128 : 256;
        a.rowtiles = (int)((p.M + rows_wg - 1) / rows_wg);
        a.chunks = (int)chunk_bound(p.E, p.R, 64 * pl.mt);
        const bool part = pl.ranges > 1;
        a.ranges = pl.ranges;
        a.part = part ? reinterpret_cast<float *>(w + sb * (up ? 2 : 1)) : nullptr;
        const void *fn = part         ? tile_fn<2, true>(up, lora)
                         : pl.mt == 4 ? tile_fn<4, false>(up, lora)
                                      : tile_fn<2, false>(up, lora);
        e = hipLaunchKernel(fn, dim3((unsigned)(((int64_t)a.rowtiles * a.chunks + 7) / 8 * 8), (unsigned)pl.ranges),
                            dim3(kTileWaves * 64), args, 0, stream);
        return e != hipSuccess || !part ? e : launch_finish(a, up, false, stream);
    }
    a.ranges = pl.ranges;
    a.slices_each = (int)(slices_of(p.K) / pl.ranges);
    a.slices_more = (int)(slices_of(p.K) % pl.ranges);
    hipError_t e;
    char *w = static_cast<char *>(workspace);
    if (pl.pre) {
        Pieces pc = pieces_at(p.K, p.R, w);
        w += pieces_bytes(p.K, p.R);
        if (!lora) {  // (the adapters' first launch writes them)
            const uint16_t *X = p.X;
            const int32_t *rows = p.rows;
            int K = a.K, T = a.T, R = a.R;
            void *pargs[] = {&X, &rows, &K, &T, &R, &pc};
            e = hipLaunchKernel(reinterpret_cast<const void *>(&ragged_pieces_kernel), dim3((unsigned)pieces_blocks(p.K, p.R)),
                                dim3(256), pargs, 0, stream);
            if (e != hipSuccess) return e;
        }
        a.X = pc.x16;
        a.xexp = pc.exps;
    }
    const bool part = pl.ranges > 1 || (pl.single && lora);
    a.part = part ? reinterpret_cast<float *>(w) : nullptr;
    const int64_t chunks = chunk_bound(p.E, p.R, pl.single ? 1 : pl.cap);
    // The workgroups that the compute units hold at once (two of 128 registers
    // each, or one), the tiles dealt evenly over them.
    const int at_once = pl.single || (pl.cap == 16 && !up && (!lora || pl.ranges > 1)) ? 2 : 1;
    int64_t wgs = at_once * compute_units() / pl.ranges;
    if (pl.single) {
        const int64_t ntiles = (p.M * (up ? 2 : 1) + kRowTile - 1) / kRowTile * chunks;
        // 4 waves a workgroup while 8 would leave compute units empty.
        const int waves = ntiles * pl.ranges < 8 * compute_units() ? 4 : 8;
        if (wgs * waves > ntiles) wgs = (ntiles + waves - 1) / waves;
        if (wgs < chunks) wgs = chunks;
        a.wgs = (int)wgs;
        if (lora) wgs += (p.R * p.r + waves - 1) / waves;
        e = hipLaunchKernel(row_fn(up, part, lora), dim3((unsigned)wgs, (unsigned)pl.ranges), dim3(64 * waves), args, 0,
                            stream);
    } else {
        const int tile_rows = pl.cap == 16 ? 32 : 16;
        const int64_t ntiles = (p.M + tile_rows - 1) / tile_rows * chunks;
        if (wgs > ntiles) wgs = ntiles;
        if (wgs < chunks) wgs = chunks;
        const void *fn = pl.cap == 32 ? chunk_fn<2, true>(up, part, lora)
                         : pl.pre     ? chunk_fn<1, true>(up, part, lora)
                                      : chunk_fn<1, false>(up, part, lora);
        e = hipLaunchKernel(fn, dim3((unsigned)wgs, (unsigned)pl.ranges), dim3(kChunkWaves * 64), args, 0, stream);
    }
    return e != hipSuccess || !part ? e : launch_finish(a, up, lora, stream);
}

}  // namespace q4
