// q4_lora.hip -- low-rank adapters beside a packed projection: the first
// product t = s A x, and the backward pass.
//
// Forward: t[n] = s_a A_a X[n] here, then the packed product with the term
// sum_j t[n][j] B_a[m][j] in its epilogue (q4_ragged.hip).
// Backward, with the packed matrix frozen:
//   u[n]  = s_a B_a^T dY[n]                            (the first product, on B transposed)
//   dX[n] = What^T dY[n] + A_a^T u[n]
//   dA_a  = sum u[n] x[n]^T,  dB_a = sum dY[n] t[n]^T  over the tokens of a
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "q4_lora.h"
#include "q4_ragged.h"
#include "q4_ragged_device.h"

namespace q4 {

namespace {

// ---------------------------------------------------------------------------
// t[n][j] = scaling[a] * sum_k Z[a][j][k] x[n][k], a = ids[n]; rows of tokens
// without an adapter are not written.  Z is bf16 [L][r][pitch].
// ---------------------------------------------------------------------------
struct ShrinkArgs {
    const uint16_t *X, *Z;
    const float *scaling;
    const int32_t *ids;
    int N, K, pitch, r, L;
    float *t;
};

constexpr int kTokens = 1024;  // tokens on their own at most; products that take pieces have no more

// Few tokens: a workgroup takes one token and 4 ranks, a wave a rank.  The
// workgroups behind those write the packed product's activations as pieces.
template <bool VEC>
__global__ __launch_bounds__(256) void lora_shrink_token_kernel(const ShrinkArgs a, const Pieces pieces, int shrinks) {
    if ((int)blockIdx.x >= shrinks) {
        write_pieces(a.X, nullptr, a.K, a.N, a.N, pieces, blockIdx.x - shrinks);
        return;
    }
    shrink_row<VEC>(a.X, a.Z, a.scaling, a.ids, a.K, a.pitch, a.r, a.L, blockIdx.x % a.N,
                    blockIdx.x / a.N * 4 + (threadIdx.x >> 6), a.N, a.t);
}

// Many tokens: a workgroup takes 16, its W waves split K in 64-blocks dealt
// round; the adapters among the 16 tokens come AD at a time.  Lane (row, g) of
// v_mfma_f32_16x16x32_bf16 holds k = 64 b + 32 s + 8 g + (0..7) of a block
// in step s, so a row's four lanes read 64 neighbouring bytes.  Bound by the
// bytes of X: an adapter's rows stay in the cache.  4096 rows of 11008 (90 MB)
// with rank 16: 32 us (2.8 TB/s; 41 with 8 waves and an adapter at a time).
template <bool VEC, int JT>
__global__ __launch_bounds__(JT >= 8 ? 512 : 1024) void lora_shrink_kernel(const ShrinkArgs a) {
    constexpr int AD = JT == 1 ? 2 : 1, W = JT >= 8 ? 8 : 16;
    __shared__ float red[W][AD][16 * 16 * JT];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 15, g = lane >> 4;
    const int n0 = blockIdx.x * 16, n = n0 + col;
    int id = n < a.N ? a.ids[n] : -1;
    if (id >= a.L) id = -1;
    const uint16_t *x = a.X + (int64_t)min(n, a.N - 1) * a.K;
    const int nb = (a.K + 63) >> 6;
    int pending = id;
    while (true) {
        int now[AD];
#pragma unroll
        for (int p = 0; p < AD; ++p) {
            const uint64_t left = __builtin_amdgcn_ballot_w64(pending >= 0);
            if (p == 0 && !left) return;
            now[p] = left ? __builtin_amdgcn_readlane(pending, __builtin_ctzll(left)) : -1;
            if (pending == now[p]) pending = -1;
        }
        float4_t acc[AD][JT];
#pragma unroll
        for (int p = 0; p < AD; ++p)
#pragma unroll
            for (int q = 0; q < JT; ++q) acc[p][q] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
        // U blocks' loads go together; blocks past the row are zeros.
        constexpr int U = JT >= 4 ? 2 : 4;
        for (int b = wave; b < nb; b += W * U) {
            u32x4_t xv[U][2], zv[U][AD][JT][2];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int k = 64 * (b + W * u) + 8 * g;
#pragma unroll
                for (int s = 0; s < 2; ++s) xv[u][s] = row_piece<VEC>(x, k + 32 * s, a.K);
#pragma unroll
                for (int p = 0; p < AD; ++p)
#pragma unroll
                    for (int q = 0; q < JT; ++q)
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            zv[u][p][q][s] = u32x4_t{0u, 0u, 0u, 0u};
                            if (now[p] >= 0 && 16 * q + col < a.r && k < a.pitch)
                                zv[u][p][q][s] = *reinterpret_cast<const u32x4_t *>(
                                    a.Z + ((int64_t)now[p] * a.r + 16 * q + col) * a.pitch + k + 32 * s);
                        }
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int s = 0; s < 2; ++s)
#pragma unroll
                    for (int p = 0; p < AD; ++p)
#pragma unroll
                        for (int q = 0; q < JT; ++q)
                            acc[p][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(bf16x8_t, xv[u][s]), __builtin_bit_cast(bf16x8_t, zv[u][p][q][s]),
                                acc[p][q], 0, 0, 0);
        }
        // Register i: token 4 g + i, rank 16 q + col.
#pragma unroll
        for (int p = 0; p < AD; ++p)
#pragma unroll
            for (int q = 0; q < JT; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i) red[wave][p][(4 * g + i) * 16 * JT + 16 * q + col] = acc[p][q][i];
        __syncthreads();
        for (int o = threadIdx.x; o < AD * 256 * JT; o += 64 * W) {
            const int p = o / (256 * JT), at = o % (256 * JT), row = at / (16 * JT), j = at % (16 * JT);
            const int adapter = p == 0 ? now[0] : now[AD - 1];
            if (n0 + row < a.N && j < a.r && adapter >= 0 && a.ids[n0 + row] == adapter) {
                float s = red[0][p][at];
#pragma unroll
                for (int w = 1; w < W; ++w) s += red[w][p][at];
                a.t[(int64_t)(n0 + row) * a.r + j] = s * a.scaling[adapter];
            }
        }
        __syncthreads();
    }
}

hipError_t launch_shrink(const ShrinkArgs &s, Pieces pieces, hipStream_t stream) {
    ShrinkArgs a = s;
    void *args[] = {&a};
    const bool vec = a.K % 8 == 0;
    // A token of its own workgroups reads its adapter alone: many short waits
    // at once, but an adapter's bytes for every token; 16 tokens that share a
    // workgroup read it once for all that use it.  With the product, in us
    // (tokens alone | 16 together): K = 2048, 512 tokens of rank 16 71.9 |
    // 75.2, 4096 82.8 | 76.8, 512 of rank 64 85.9 | 96.1, 2048 108 | 103; K =
    // 11008, 256 of rank 64 76 | 150, 1024 303 | 316.
    if (a.N <= kTokens) {
        int shrinks = a.N * ((a.r + 3) / 4);
        void *targs[] = {&a, &pieces, &shrinks};
        return hipLaunchKernel(vec ? reinterpret_cast<const void *>(&lora_shrink_token_kernel<true>)
                                   : reinterpret_cast<const void *>(&lora_shrink_token_kernel<false>),
                               dim3((unsigned)(shrinks + (pieces.x16 ? pieces_blocks(a.K, a.N) : 0))), dim3(256),
                               targs, 0, stream);
    }
    const void *fn;
    if (a.r <= 16)
        fn = vec ? reinterpret_cast<const void *>(&lora_shrink_kernel<true, 1>)
                 : reinterpret_cast<const void *>(&lora_shrink_kernel<false, 1>);
    else if (a.r <= 32)
        fn = vec ? reinterpret_cast<const void *>(&lora_shrink_kernel<true, 2>)
                 : reinterpret_cast<const void *>(&lora_shrink_kernel<false, 2>);
    else if (a.r <= 64)
        fn = vec ? reinterpret_cast<const void *>(&lora_shrink_kernel<true, 4>)
                 : reinterpret_cast<const void *>(&lora_shrink_kernel<false, 4>);
    else
        fn = vec ? reinterpret_cast<const void *>(&lora_shrink_kernel<true, 8>)
                 : reinterpret_cast<const void *>(&lora_shrink_kernel<false, 8>);
    return hipLaunchKernel(fn, dim3((unsigned)((a.N + 15) / 16)), dim3(a.r > 64 ? 512 : 1024), args, 0, stream);
}

// ---------------------------------------------------------------------------
// Backward: what is prepared.
// ---------------------------------------------------------------------------

// The exponent of a packed row of zeros: its dY then counts as nothing, in the
// choice of a token's power of two too.
constexpr int kZeroRow = -4096;

// The packed rows' exponents and scales (16 rows a workgroup), and behind those
// workgroups B transposed: bt[a][j][m], rows of `pitch` with zeros past M (a
// workgroup takes 64 m of one adapter).
__global__ __launch_bounds__(256) void lora_rows_kernel(const uint16_t *__restrict__ scales, int M, int nb,
                                                        int16_t *__restrict__ rowexp, uint16_t *__restrict__ tscale,
                                                        int rowblocks, const uint16_t *__restrict__ B, int r,
                                                        int pitch, uint16_t *__restrict__ bt) {
    __shared__ uint16_t tile[64][130];
    if ((int)blockIdx.x < rowblocks) {
        prepare_scales<kZeroRow>(scales, (int64_t)blockIdx.x * 16, M, M, nb, rowexp, tscale);
        return;
    }
    const int per = pitch / 64, w = blockIdx.x - rowblocks;
    const int l = w / per, m0 = (w % per) * 64;
    for (int i = threadIdx.x; i < 64 * r; i += 256) {
        const int m = m0 + i / r, j = i % r;
        tile[i / r][j] = m < M ? B[((int64_t)l * M + m) * r + j] : 0;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 64 * r; i += 256)
        bt[((int64_t)l * r + i / 64) * pitch + m0 + i % 64] = tile[i % 64][i / 64];
}

// dY[n][m] 2^(rowexp[m] + shift[n]) as fp16, rows of `pitch` with zeros past
// M: the power of two of each packed row goes to this side, so that the
// weights' fp16 values keep their full precision, and the token's brings the
// largest to [2^14, 2^15).
// The exponents of two values are found at once in 16-bit halves; the first
// kDyHeld pieces of a thread stay in registers between the two passes.  4096 x
// 11008: 180 MB read and written in 30 us (6 TB/s, in part to the Infinity
// Cache).
typedef short s16x2_t __attribute__((ext_vector_type(2)));
constexpr int kDyHeld = 6;

template <bool VEC>
__global__ __launch_bounds__(256) void lora_dy_kernel(const uint16_t *__restrict__ dY, int M, int pitch,
                                                      const int16_t *__restrict__ rowexp, uint16_t *__restrict__ out,
                                                      int32_t *__restrict__ exps) {
    __shared__ int wmax[4];
    const int n = blockIdx.x;
    const uint16_t *src = dY + (int64_t)n * M;
    s16x2_t best2 = {0, 0};
    u32x4_t held[kDyHeld];
    auto look = [&](const u32x4_t &v, int m) {
        const u32x4_t e = *reinterpret_cast<const u32x4_t *>(rowexp + m);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const u16x2_t mag = __builtin_bit_cast(u16x2_t, v[c] & 0x7FFF7FFFu);
            u16x2_t ex = mag >> 7;
            ex = __builtin_elementwise_min(ex, u16x2_t{254, 254});
            // 2048 more than the exponent, 0 for a zero (whatever stands in the
            // exponents behind the last packed row), below 0 for kZeroRow.
            const s16x2_t nz = __builtin_bit_cast(s16x2_t, __builtin_elementwise_min(mag, u16x2_t{1, 1}));
            // (Copied first: a bit cast of a vector's element itself reads element 0.)
            const uint32_t pair = e[c];
            const s16x2_t key = __builtin_bit_cast(s16x2_t, ex) + __builtin_bit_cast(s16x2_t, pair) + s16x2_t{2048, 2048};
            best2 = __builtin_elementwise_max(best2, key & -nz);
        }
    };
    auto put = [&](const u32x4_t &v, int m, int shift) {
        const u32x4_t e = *reinterpret_cast<const u32x4_t *>(rowexp + m);
        u32x4_t h;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int el = (int)(e[c] << 16) >> 16, eh = (int)e[c] >> 16;
            h[c] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(ldexpf(bf16_lo(v[c]), shift + el),
                                                                           ldexpf(bf16_hi(v[c]), shift + eh)));
        }
        *reinterpret_cast<u32x4_t *>(out + (int64_t)n * pitch + m) = h;
    };
#pragma unroll
    for (int i = 0; i < kDyHeld; ++i) {
        const int m = threadIdx.x * 8 + 2048 * i;
        held[i] = m < M ? row_piece<VEC>(src, m, M) : u32x4_t{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int i = 0; i < kDyHeld; ++i) {
        const int m = threadIdx.x * 8 + 2048 * i;
        if (m < M) look(held[i], m);
    }
    for (int m = threadIdx.x * 8 + 2048 * kDyHeld; m < M; m += 2048) look(row_piece<VEC>(src, m, M), m);
    int best = max((int)best2.x, (int)best2.y);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) best = max(best, __shfl_xor(best, d));
    if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = best;
    __syncthreads();
    best = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3])) - 2048;
    const int shift = best < -1024 ? 0 : 141 - best;  // (a row of zeros)
#pragma unroll
    for (int i = 0; i < kDyHeld; ++i) {
        const int m = threadIdx.x * 8 + 2048 * i;
        if (m < pitch) put(held[i], m, shift);
    }
    for (int m = threadIdx.x * 8 + 2048 * kDyHeld; m < pitch; m += 2048)
        put(m < M ? row_piece<VEC>(src, m, M) : u32x4_t{0u, 0u, 0u, 0u}, m, shift);
    if (threadIdx.x == 0) exps[n] = -shift;
}

// ---------------------------------------------------------------------------
// dX[n][k] = sum_m What[m,k] dY[n][m] + sum_j u[n][j] A_a[j][k].
// ---------------------------------------------------------------------------
struct DxArgs {
    const uint16_t *dy16;   // fp16 [N][pitch]
    const int32_t *exps;
    const uint8_t *codes;
    const uint16_t *tscale; // the scales under each packed row's power of two, [K/64][M]
    int N, M, K, pitch, ktiles, splits;
    float *part;            // [splits][N][K], or null
    uint16_t *dX;
    const uint16_t *A;
    const float *u;
    const int32_t *ids;
    int r, L;
};

// A workgroup computes 64 MT tokens (2 waves of MT tiles of 32) by 256 k (4
// waves of 64: one block of the packed rows, whose 32 code bytes are the 32
// lanes' columns; a lane's two weights of a byte are the columns 2c and 2c+1
// of two tiles).  The contraction runs over 64 packed rows a step: their code
// bytes are transposed into LDS so that a lane reads its column's bytes of 32
// rows as two 16-byte pieces.  The scaled weights are rounded to fp16 as in the
// forward kernels.  4096 tokens, 11008 x 2048 take 245 us (750 TFLOP/s) in two
// parts of the packed rows, and 13 to add them: bound by the lookups beside the
// matrix cores, which are busy 0.40 of the time, and by dY, which is read eight
// times (736 MB: workgroups go round the XCDs by column tile, so each XCD's L2
// takes in all of it).  Few tokens are bound by the walk along the packed rows,
// which is split over workgroups.
template <int MT>
__global__ __launch_bounds__(512) void lora_dx_kernel(const DxArgs a) {
    constexpr int TM = 64 * MT;
    constexpr int kPieces = TM * 8 / 512;
    __shared__ uint32_t lut[kLutDwords];
    __shared__ uint4 ys[2][TM * 8];
    __shared__ uint32_t ct[2][128 * 16];  // [column slot][64 rows' bytes]
    __shared__ uint4 sl[2][4 * 8];        // [block of 64 k][64 rows] fp16 scales
    __shared__ int xe[TM];
    __shared__ int sid[TM];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = lane & 31, g = lane >> 5;
    const int wt = wave & 1, wk = wave >> 1;
    const int tile = blockIdx.x / a.ktiles, kt = blockIdx.x % a.ktiles;
    const int n0 = tile * TM, count = min(TM, a.N - n0);
    const int nb = a.K >> 6;
    const int steps = a.pitch >> 6;
    const int st0 = (int)((int64_t)steps * blockIdx.y / a.splits), st1 = (int)((int64_t)steps * (blockIdx.y + 1) / a.splits);

    for (int i = threadIdx.x; i < TM; i += 512) {
        xe[i] = i < count ? a.exps[n0 + i] : 0;
        const int id = a.L > 0 && i < count ? a.ids[n0 + i] : -1;
        sid[i] = id >= 0 && id < a.L ? id : -1;
    }
    const uint4 *ysrc[kPieces];
#pragma unroll
    for (int j = 0; j < kPieces; ++j) {
        const int i = (threadIdx.x >> 3) + 64 * j;
        const int piece = (threadIdx.x & 7) ^ ((i >> 1) & 7);
        ysrc[j] = i < count ? reinterpret_cast<const uint4 *>(a.dy16 + (int64_t)(n0 + i) * a.pitch) + piece : nullptr;
    }
    // Codes: lane bits 0..3 pick four rows, the rest a dword of the 128 bytes.
    const int m4 = threadIdx.x & 15, dc = threadIdx.x >> 4;
    const int dbyte = kt * 128 + dc * 4;
    const bool dlive = dbyte < (a.K >> 1);
    const int skb = threadIdx.x >> 6, sm = threadIdx.x & 63;  // scales: first 256 threads

    uint4 yv[kPieces];
    uint32_t cv[4];
    uint32_t sv = 0;
    auto load = [&](int st) {
#pragma unroll
        for (int j = 0; j < kPieces; ++j) yv[j] = ysrc[j] ? ysrc[j][8 * st] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int m = min(64 * st + 4 * m4 + i, a.M - 1);
            cv[i] = dlive ? *reinterpret_cast<const uint32_t *>(a.codes + (int64_t)m * (a.K >> 1) + dbyte) : 0;
        }
        if (threadIdx.x < 256) {
            const int m = 64 * st + sm, kb = kt * 4 + skb;
            sv = m < a.M && kb < nb ? a.tscale[(int64_t)kb * a.M + m] : 0;
        }
    };
    load(st0);
    fill_lut(lut);

    float16_t acc[MT][2];
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int q = 0; q < 2; ++q) acc[i][q] = float16_t{};
    const uint32_t laneoff = (uint32_t)lane << 2;
    // Column slot of byte 4 d + j: j * 32 + d, so that both the transposing
    // writes and the reads meet every bank; 16-byte pieces under an exchange
    // by j.
    const int mycol = (col & 3) * 32 + wk * 8 + (col >> 2);

    for (int st = st0; st < st1; ++st) {
        const int bi = st & 1;
#pragma unroll
        for (int j = 0; j < kPieces; ++j) ys[bi][threadIdx.x + 512 * j] = yv[j];
        {
            const uint32_t p0 = __builtin_amdgcn_perm(cv[1], cv[0], 0x05010400u);  // r0.b0 r1.b0 r0.b1 r1.b1
            const uint32_t p1 = __builtin_amdgcn_perm(cv[1], cv[0], 0x07030602u);  // r0.b2 r1.b2 r0.b3 r1.b3
            const uint32_t p2 = __builtin_amdgcn_perm(cv[3], cv[2], 0x05010400u);
            const uint32_t p3 = __builtin_amdgcn_perm(cv[3], cv[2], 0x07030602u);
            const uint32_t o[4] = {__builtin_amdgcn_perm(p2, p0, 0x05040100u), __builtin_amdgcn_perm(p2, p0, 0x07060302u),
                                   __builtin_amdgcn_perm(p3, p1, 0x05040100u), __builtin_amdgcn_perm(p3, p1, 0x07060302u)};
#pragma unroll
            for (int j = 0; j < 4; ++j) ct[bi][(j * 32 + dc) * 16 + (((m4 >> 2) ^ j) << 2) + (m4 & 3)] = o[j];
        }
        if (threadIdx.x < 256)
            reinterpret_cast<uint16_t *>(sl[bi])[skb * 64 + sm] = (uint16_t)sv;
        __syncthreads();
        if (st + 1 < st1) load(st + 1);

        // This lane's column: the bytes of rows 32 g .. 32 g + 31.
        u32x4_t by[2];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            by[h] = *reinterpret_cast<const u32x4_t *>(&ct[bi][mycol * 16 + (((2 * g + h) ^ (col & 3)) << 2)]);
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            // Rows 32 g + 8 s + (0..7): two dwords of bytes, eight scales.
            const uint32_t w0 = by[s >> 1][2 * (s & 1)], w1 = by[s >> 1][2 * (s & 1) + 1];
            half2_t v[8];
            v[0] = lut_pair<0>(lut, w0, laneoff);
            v[1] = lut_pair<1>(lut, w0, laneoff);
            v[2] = lut_pair<2>(lut, w0, laneoff);
            v[3] = lut_pair<3>(lut, w0, laneoff);
            v[4] = lut_pair<0>(lut, w1, laneoff);
            v[5] = lut_pair<1>(lut, w1, laneoff);
            v[6] = lut_pair<2>(lut, w1, laneoff);
            v[7] = lut_pair<3>(lut, w1, laneoff);
            const uint4 sc = sl[bi][wk * 8 + 4 * g + s];
            const uint32_t scd[4] = {sc.x, sc.y, sc.z, sc.w};
            half2_t even[4], odd[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t x = __builtin_bit_cast(uint32_t, v[2 * i]), y = __builtin_bit_cast(uint32_t, v[2 * i + 1]);
                const half2_t s2 = __builtin_bit_cast(half2_t, scd[i]);
                even[i] = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(y, x, 0x05040100u)) * s2;
                odd[i] = __builtin_bit_cast(half2_t, __builtin_amdgcn_perm(y, x, 0x07060302u)) * s2;
            }
            const half8_t b0 = join8(even), b1 = join8(odd);
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                const int row = wt * 32 * MT + 32 * i + col;
                const half8_t ya = __builtin_bit_cast(half8_t, ys[bi][row * 8 + ((4 * g + s) ^ ((row >> 1) & 7))]);
                acc[i][0] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ya, b0, acc[i][0], 0, 0, 0);
                acc[i][1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(ya, b1, acc[i][1], 0, 0, 0);
            }
        }
    }

#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int x = xe[wt * 32 * MT + 32 * i + tile_row(j, lane)] - 14;
            acc[i][0][j] = ldexpf(acc[i][0][j], x);
            acc[i][1][j] = ldexpf(acc[i][1][j], x);
        }
    const int k = kt * 256 + wk * 64 + 2 * col;  // this lane's two columns
    bool wild = false;  // an adapter of this wave's rows holds a value that is not finite

    // With planes the first of them takes the adapters' term; with few tokens,
    // each of which may have an adapter of its own, the launch that adds the
    // planes makes it for all tokens at once (4096 tokens in that launch: 38 us,
    // here 13).
    if (!a.part || (MT > 1 && blockIdx.y == 0)) {
        int mine[2] = {-1, -1};
        const int w0 = wt * 32 * MT;
        mine[0] = sid[w0 + (lane & (32 * MT - 1))];
        if (MT == 4) mine[1] = sid[w0 + 64 + lane];
        while (true) {
            const uint64_t p0 = __builtin_amdgcn_ballot_w64(mine[0] >= 0);
            const uint64_t p1 = __builtin_amdgcn_ballot_w64(mine[1] >= 0);
            if (!(p0 | p1)) break;
            const int id = p0 ? __builtin_amdgcn_readlane(mine[0], __builtin_ctzll(p0))
                              : __builtin_amdgcn_readlane(mine[1], __builtin_ctzll(p1));
            if (mine[0] == id) mine[0] = -1;
            if (mine[1] == id) mine[1] = -1;
            for (int j0 = 0; j0 < a.r; j0 += 16) {
                const bool live = j0 + 8 * g < a.r;
                uint32_t d[8];
#pragma unroll
                for (int x = 0; x < 8; ++x)
                    d[x] = live && k < a.K ? *reinterpret_cast<const uint32_t *>(
                                                 a.A + ((int64_t)id * a.r + j0 + 8 * g + x) * a.K + k)
                                           : 0;
                u32x4_t e, o;
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    e[x] = __builtin_amdgcn_perm(d[2 * x + 1], d[2 * x], 0x05040100u);
                    o[x] = __builtin_amdgcn_perm(d[2 * x + 1], d[2 * x], 0x07060302u);
                }
                if (__builtin_amdgcn_ballot_w64(not_finite8(e) || not_finite8(o))) {
                    wild = true;
                    e = finite8(e);
                    o = finite8(o);
                }
                const bf16x8_t be = __builtin_bit_cast(bf16x8_t, e), bo = __builtin_bit_cast(bf16x8_t, o);
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                    const int row = w0 + 32 * i + col;
                    const bool use = sid[row] == id;
                    if (__builtin_amdgcn_ballot_w64(use) == 0) continue;
                    float t[8];
#pragma unroll
                    for (int x = 0; x < 8; ++x) t[x] = 0.0f;
                    if (use && live) {
                        const float *src = a.u + (int64_t)(n0 + row) * a.r + j0 + 8 * g;
#pragma unroll
                        for (int x = 0; x < 8; ++x) t[x] = src[x];
                    }
                    bf16x8_t hi, lo;
                    split2(t, hi, lo);
                    acc[i][0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(hi, be, acc[i][0], 0, 0, 0);
                    acc[i][0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(lo, be, acc[i][0], 0, 0, 0);
                    acc[i][1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(hi, bo, acc[i][1], 0, 0, 0);
                    acc[i][1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(lo, bo, acc[i][1], 0, 0, 0);
                }
            }
        }
    }
    if (k >= a.K) return;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            const int row = wt * 32 * MT + 32 * i + tile_row(j, lane);
            if (row >= count) continue;
            const int64_t at = (int64_t)(n0 + row) * a.K + k;
            if (a.part) {
                float2 *o = reinterpret_cast<float2 *>(a.part + (int64_t)blockIdx.y * a.N * a.K + at);
                *o = make_float2(acc[i][0][j], acc[i][1][j]);
            } else {
                *reinterpret_cast<uint32_t *>(a.dX + at) =
                    (uint32_t)f32_bf16(acc[i][0][j]) | (uint32_t)f32_bf16(acc[i][1][j]) << 16;
            }
        }
    if (!wild) return;
    // (Every lane adds to the outputs that it has stored.)
    for (int i = 0; i < 32 * MT; ++i) {
        const int row = wt * 32 * MT + 32 * (i >> 5) + tile_row(i >> 1 & 15, lane);
        if (row >= count || sid[row] < 0) continue;
        const float y = wild_term(a.u + (int64_t)(n0 + row) * a.r, a.A + (int64_t)sid[row] * a.r * a.K + k + (i & 1), a.K,
                                  a.r);
        if (y == 0.0f) continue;
        const int64_t at = (int64_t)(n0 + row) * a.K + k + (i & 1);
        if (a.part) a.part[at] += y;  // (the first plane)
        else a.dX[at] = f32_bf16(bf16_f32(a.dX[at]) + y);
    }
}

// Adds the partial planes in order, and the adapter's term where there are few
// tokens (L is 0 elsewhere); four columns a lane.
__global__ __launch_bounds__(256) void lora_dx_finish_kernel(const DxArgs a) {
    const int per = (a.K + 1023) >> 10;
    const int n = blockIdx.x / per, k = ((blockIdx.x % per) * 256 + threadIdx.x) * 4;
    if (k >= a.K) return;
    const int64_t at = (int64_t)n * a.K + k, plane = (int64_t)a.N * a.K;
    float4_t v = *reinterpret_cast<const float4_t *>(a.part + at);
#pragma unroll 4
    for (int z = 1; z < a.splits; ++z) v += *reinterpret_cast<const float4_t *>(a.part + z * plane + at);
    const int id = a.L > 0 ? a.ids[n] : -1;
    if (id >= 0 && id < a.L) {
        float4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
        for (int j = 0; j < a.r; ++j) {
            const uint2 d = *reinterpret_cast<const uint2 *>(a.A + ((int64_t)id * a.r + j) * a.K + k);
            const float t = a.u[(int64_t)n * a.r + j];
            s[0] = fmaf(t, bf16_lo(d.x), s[0]);
            s[1] = fmaf(t, bf16_hi(d.x), s[1]);
            s[2] = fmaf(t, bf16_lo(d.y), s[2]);
            s[3] = fmaf(t, bf16_hi(d.y), s[3]);
        }
        v += s;
    }
    *reinterpret_cast<uint2 *>(a.dX + at) = make_uint2((uint32_t)f32_bf16(v[0]) | (uint32_t)f32_bf16(v[1]) << 16,
                                                       (uint32_t)f32_bf16(v[2]) | (uint32_t)f32_bf16(v[3]) << 16);
}

// ---------------------------------------------------------------------------
// Gradients of the adapters: for pieces of at most kPieceTokens tokens of one
// adapter (in the order of the tokens), g[j][c] = sum_n t[n][j] Z[n][c].
//
// v_mfma_f32_16x16x4_f32 adds four tokens' products of 16 ranks and 16
// columns, exact products of fp32 operands: lane (i, g) holds t[n + g][j0 + i]
// and one column of Z's row n + g, both as they lie in memory, so nothing is
// transposed and nothing rounded.  A lane's 16 bytes of a row are 8 columns,
// one for each of 8 such products.  A wave takes 128 columns.  4096 tokens,
// rank 16, 2048 and 11008 columns (107 MB): 34 us (3.1 TB/s), and 12 for the
// sum of the pieces; bound by the waits for the rows.
// ---------------------------------------------------------------------------
constexpr int kPieceTokens = 128;

struct GradArgs {
    const uint16_t *Z[2];    // X [N][K] and dY [N][M]
    const float *t[2];       // u and t
    int cols[2];
    float *part[2];          // [pieces][r][cols]
    float *out[2];           // dA [L][r][K], dB [L][M][r]
    const int32_t *offsets, *rows;
    int N, L, r, blocks0;
};

// VEC: both matrices' rows start on 16 bytes.  JT: tiles of 16 ranks at once.
template <bool VEC, int JT>
__global__ __launch_bounds__(256) void lora_grad_kernel(const GradArgs a) {
    constexpr int U = JT == 1 ? 8 : 4;  // steps of four tokens whose loads go together
    const int q = (int)blockIdx.x >= a.blocks0 ? 1 : 0;
    const Chunk ck = find_chunk(a.offsets, a.L, a.N, blockIdx.y, kPieceTokens);
    if (ck.count == 0) return;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, i16 = lane & 15, g = lane >> 4;
    const int cols = a.cols[q];
    const int c = (int)(blockIdx.x - (q ? a.blocks0 : 0)) * 512 + wave * 128 + 8 * i16;
    const int j0 = blockIdx.z * 16 * JT;
    const uint16_t *Z = a.Z[q];
    const float *T = a.t[q];
    // The piece's tokens: two of them in a lane.
    static_assert(kPieceTokens == 128, "two rows a lane");
    int tok[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) tok[h] = a.rows[ck.start + min(64 * h + lane, ck.count - 1)];
    float4_t acc[JT][8];
#pragma unroll
    for (int p = 0; p < JT; ++p)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[p][i] = float4_t{0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; s < ck.count; s += 4 * U) {
        u32x4_t z[U];
        float t[U][JT];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = s + 4 * u + g;
            const int n = __shfl(s < 64 ? tok[0] : tok[1], at & 63);
            z[u] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
            for (int p = 0; p < JT; ++p) t[u][p] = 0.0f;
            if (at < ck.count) {
                z[u] = row_piece<VEC>(Z + (int64_t)n * cols, c, cols);
#pragma unroll
                for (int p = 0; p < JT; ++p)
                    if (j0 + 16 * p + i16 < a.r) t[u][p] = T[(int64_t)n * a.r + j0 + 16 * p + i16];
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float v = i & 1 ? bf16_hi(z[u][i >> 1]) : bf16_lo(z[u][i >> 1]);
#pragma unroll
                for (int p = 0; p < JT; ++p)
                    acc[p][i] = __builtin_amdgcn_mfma_f32_16x16x4f32(t[u][p], v, acc[p][i], 0, 0, 0);
            }
    }
    // Register x of tile (p, i): rank j0 + 16 p + 4 g + x, column c + i.
#pragma unroll
    for (int p = 0; p < JT; ++p)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
            const int j = j0 + 16 * p + 4 * g + x;
            if (j >= a.r) continue;
            float *o = a.part[q] + ((int64_t)blockIdx.y * a.r + j) * cols + c;
            if (VEC) {
                if (c < cols) {
                    *reinterpret_cast<float4 *>(o) = make_float4(acc[p][0][x], acc[p][1][x], acc[p][2][x], acc[p][3][x]);
                    *reinterpret_cast<float4 *>(o + 4) = make_float4(acc[p][4][x], acc[p][5][x], acc[p][6][x], acc[p][7][x]);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + i < cols) o[i] = acc[p][i][x];
            }
        }
}

// Adds the pieces of each adapter in order (none: zeros).
__global__ __launch_bounds__(256) void lora_grad_sum_kernel(const GradArgs a) {
    const int q = (int)blockIdx.x >= a.blocks0 ? 1 : 0;
    const int l = blockIdx.y, j = blockIdx.z;
    const int cols = a.cols[q];
    const int c = (int)(blockIdx.x - (q ? a.blocks0 : 0)) * 256 + threadIdx.x;
    // The pieces before those of adapter l, and its own.
    int first = 0;
    for (int e0 = 0; e0 < l; e0 += 64) {
        const int e = e0 + (threadIdx.x & 63);
        int n = 0;
        if (e < l) n = (a.offsets[e + 1] - a.offsets[e] + kPieceTokens - 1) / kPieceTokens;
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) n += __shfl_xor(n, d);
        first += n;
    }
    const int n = (a.offsets[l + 1] - a.offsets[l] + kPieceTokens - 1) / kPieceTokens;
    if (c >= cols) return;
    float s = 0.0f;
    for (int i = 0; i < n; ++i) s += a.part[q][((int64_t)(first + i) * a.r + j) * cols + c];
    if (q == 0) a.out[0][((int64_t)l * a.r + j) * cols + c] = s;
    else a.out[1][((int64_t)l * cols + c) * a.r + j] = s;
}

int64_t pieces_bound(int64_t N, int64_t L) {
    const int64_t p = N / kPieceTokens + L;
    return p < N ? p : N;
}

struct DxPlan {
    int mt, ktiles, splits;
    int64_t tiles;
};

DxPlan dx_plan(int64_t M, int64_t K, int64_t N) {
    DxPlan p = {};
    // 1 | 2 | 4 tiles a wave, the whole call in us: 2048 x 2048, N = 64 40.3 |
    // 41.7 | 44.2, 512 64.5 | 64.1 | 72.4; 11008 x 2048, N = 512 146 | 125 |
    // 126, 2048 341 | 262 | 244.
    p.mt = N > 1024 ? 4 : N > 256 ? 2 : 1;
    p.tiles = (N + 64 * p.mt - 1) / (64 * p.mt);
    p.ktiles = (int)((K + 255) / 256);
    // Packed rows are split while there are fewer workgroups than compute
    // units, into parts of 256 rows at least: 2048 x 2048, N = 64 in 1, 4, 8,
    // 16 parts 71.5, 42.2, 38.5, 40.4 us; N = 128 in 4, 8, 16 48.3, 47.1, 52.9.
    // (256: an MI355X's; the workspace's size follows from the shape alone.)
    const int64_t steps = (M + 63) / 64, have = p.tiles * p.ktiles, cus = 256;
    int64_t s = have >= cus || have == 0 ? 1 : (cus + have - 1) / have;
    if (s > (steps + 3) / 4) s = (steps + 3) / 4;
    p.splits = (int)(s < 1 ? 1 : s);
    return p;
}

struct BackwardLayout {
    size_t t, u, bt, dy16, exps, rowexp, tscale, offsets, rows, sort, part, grad[2], total;
    int64_t pitch;
};

BackwardLayout backward_layout(int64_t M, int64_t K, int64_t N, int64_t r, int64_t L) {
    BackwardLayout b = {};
    size_t at = 0;
    auto take = [&](size_t n) {
        const size_t was = at;
        at += round16(n);
        return was;
    };
    b.pitch = (M + 63) / 64 * 64;
    const DxPlan p = dx_plan(M, K, N);
    b.t = take((size_t)N * r * 4);
    b.u = take((size_t)N * r * 4);
    b.bt = take((size_t)L * r * b.pitch * 2);
    b.dy16 = take((size_t)N * b.pitch * 2);
    b.exps = take((size_t)N * 4);
    b.rowexp = take((size_t)b.pitch * 2);
    b.tscale = take((size_t)M * (K / 64) * 2);
    b.offsets = take((size_t)(L + 1) * 4);
    b.rows = take((size_t)N * 4);
    b.sort = take(sort_ws_bytes(N, L));
    b.part = take(p.splits > 1 ? (size_t)p.splits * N * K * 4 : 0);
    b.grad[0] = take((size_t)pieces_bound(N, L) * r * K * 4);
    b.grad[1] = take((size_t)pieces_bound(N, L) * r * M * 4);
    b.total = at;
    return b;
}

}  // namespace

bool lora_backward_fits(int64_t M, int64_t K, int64_t N, int64_t L) {
    const DxPlan p = dx_plan(M, K, N);
    const int64_t most = INT64_C(1) << 32;  // threads of one launch
    return ((M + 15) / 16 + L * ((M + 63) / 64)) * 256 < most && p.tiles * p.ktiles * 512 < most &&
           pieces_bound(N, L) < 65536;
}

size_t lora_ws_bytes(int64_t M, int64_t K, int64_t N, int64_t r, int64_t L) {
    return (L > 0 ? round16((size_t)N * r * 4) : 0) + ragged_ws_bytes(1, M, K, N, N, false, L > 0 ? r : 0);
}

hipError_t launch_lora(const LoraCall &c, bool bf16, void *Y, void *workspace, hipStream_t stream) {
    RaggedProduct p = {};
    p.codes = c.codes;
    p.scales = c.scales;
    p.E = 1;
    p.M = c.M;
    p.K = c.K;
    p.X = c.X;
    p.T = p.R = c.N;
    p.bf16 = bf16;
    p.Y = Y;
    char *w = static_cast<char *>(workspace);
    if (c.L > 0 && ragged_shrinks(1, c.M, c.K, c.N, c.r)) {
        p.A = c.A;
        p.scaling = c.scaling;
        p.t = reinterpret_cast<float *>(w);
    } else if (c.L > 0) {
        ShrinkArgs s = {c.X,      c.A, c.scaling, c.ids, (int)c.N, (int)c.K, (int)c.K, (int)c.r, (int)c.L,
                        reinterpret_cast<float *>(w)};
        Pieces pieces = {};
        if (ragged_takes_pieces(1, c.M, c.K, c.N, c.r))
            pieces = pieces_at(c.K, c.N, w + round16((size_t)c.N * c.r * 4));
        const hipError_t e = launch_shrink(s, pieces, stream);
        if (e != hipSuccess) return e;
        p.t = s.t;
    }
    if (c.L > 0) {
        p.B = c.B;
        p.ids = c.ids;
        p.r = c.r;
        p.L = c.L;
        w += round16((size_t)c.N * c.r * 4);
    }
    return launch_ragged(p, w, stream);
}

size_t lora_backward_ws_bytes(int64_t M, int64_t K, int64_t N, int64_t r, int64_t L) {
    return backward_layout(M, K, N, r, L).total;
}

hipError_t launch_lora_backward(const LoraCall &c, const uint16_t *dY, uint16_t *dX, float *dA, float *dB,
                                void *workspace, hipStream_t stream) {
    const BackwardLayout b = backward_layout(c.M, c.K, c.N, c.r, c.L);
    char *w = static_cast<char *>(workspace);
    float *t = reinterpret_cast<float *>(w + b.t), *u = reinterpret_cast<float *>(w + b.u);
    uint16_t *bt = reinterpret_cast<uint16_t *>(w + b.bt), *dy16 = reinterpret_cast<uint16_t *>(w + b.dy16);
    int32_t *exps = reinterpret_cast<int32_t *>(w + b.exps);
    int16_t *rowexp = reinterpret_cast<int16_t *>(w + b.rowexp);
    uint16_t *tscale = reinterpret_cast<uint16_t *>(w + b.tscale);
    int32_t *offsets = reinterpret_cast<int32_t *>(w + b.offsets), *rows = reinterpret_cast<int32_t *>(w + b.rows);
    hipError_t e;
    if (c.N > 0) {
        const uint16_t *scales = c.scales, *B = c.B;
        int M = (int)c.M, nb = (int)(c.K / 64), rowblocks = dX ? (int)((c.M + 15) / 16) : 0, r = (int)c.r;
        int pitch = (int)b.pitch;
        void *rargs[] = {&scales, &M, &nb, &rowexp, &tscale, &rowblocks, &B, &r, &pitch, &bt};
        e = hipLaunchKernel(reinterpret_cast<const void *>(&lora_rows_kernel),
                            dim3((unsigned)(rowblocks + c.L * (b.pitch / 64))), dim3(256), rargs, 0, stream);
        if (e != hipSuccess) return e;
        if (c.L > 0) {
            ShrinkArgs su = {dY, bt, c.scaling, c.ids, (int)c.N, (int)c.M, (int)b.pitch, (int)c.r, (int)c.L, u};
            if ((e = launch_shrink(su, Pieces{}, stream)) != hipSuccess) return e;
        }
        if (dX) {
            void *yargs[] = {&dY, &M, &pitch, &rowexp, &dy16, &exps};
            e = hipLaunchKernel(c.M % 8 == 0 ? reinterpret_cast<const void *>(&lora_dy_kernel<true>)
                                             : reinterpret_cast<const void *>(&lora_dy_kernel<false>),
                                dim3((unsigned)c.N), dim3(256), yargs, 0, stream);
            if (e != hipSuccess) return e;
            const DxPlan p = dx_plan(c.M, c.K, c.N);
            DxArgs d = {};
            d.dy16 = dy16;
            d.exps = exps;
            d.codes = c.codes;
            d.tscale = tscale;
            d.N = (int)c.N;
            d.M = M;
            d.K = (int)c.K;
            d.pitch = pitch;
            d.ktiles = p.ktiles;
            d.splits = p.splits;
            d.part = p.splits > 1 ? reinterpret_cast<float *>(w + b.part) : nullptr;
            d.dX = dX;
            d.A = c.A;
            d.u = u;
            d.ids = c.ids;
            d.r = r;
            d.L = (int)c.L;
            void *dargs[] = {&d};
            const void *fn = p.mt == 4   ? reinterpret_cast<const void *>(&lora_dx_kernel<4>)
                             : p.mt == 2 ? reinterpret_cast<const void *>(&lora_dx_kernel<2>)
                                         : reinterpret_cast<const void *>(&lora_dx_kernel<1>);
            e = hipLaunchKernel(fn, dim3((unsigned)(p.tiles * p.ktiles), (unsigned)p.splits), dim3(512), dargs, 0,
                                stream);
            if (e != hipSuccess) return e;
            if (p.splits > 1) {
                if (p.mt > 1) d.L = 0;
                e = hipLaunchKernel(reinterpret_cast<const void *>(&lora_dx_finish_kernel),
                                    dim3((unsigned)(c.N * ((c.K + 1023) / 1024))), dim3(256), dargs, 0, stream);
                if (e != hipSuccess) return e;
            }
        }
    }
    if (!dA || c.L == 0) return hipSuccess;
    if (c.N > 0) {
        ShrinkArgs st = {c.X, c.A, c.scaling, c.ids, (int)c.N, (int)c.K, (int)c.K, (int)c.r, (int)c.L, t};
        if ((e = launch_shrink(st, Pieces{}, stream)) != hipSuccess) return e;
    }
    if ((e = launch_sort(c.ids, c.N, c.L, 1, offsets, rows, nullptr, w + b.sort, stream)) != hipSuccess) return e;
    GradArgs g = {};
    g.Z[0] = c.X;
    g.Z[1] = dY;
    g.t[0] = u;
    g.t[1] = t;
    g.cols[0] = (int)c.K;
    g.cols[1] = (int)c.M;
    g.part[0] = reinterpret_cast<float *>(w + b.grad[0]);
    g.part[1] = reinterpret_cast<float *>(w + b.grad[1]);
    g.out[0] = dA;
    g.out[1] = dB;
    g.offsets = offsets;
    g.rows = rows;
    g.N = (int)c.N;
    g.L = (int)c.L;
    g.r = (int)c.r;
    void *gargs[] = {&g};
    if (c.N > 0) {
        g.blocks0 = (int)((c.K + 511) / 512);
        const bool vec = c.M % 8 == 0;
        const int jt = c.r > 16 ? 2 : 1;
        const void *fn = vec ? jt == 2 ? reinterpret_cast<const void *>(&lora_grad_kernel<true, 2>)
                                       : reinterpret_cast<const void *>(&lora_grad_kernel<true, 1>)
                             : jt == 2 ? reinterpret_cast<const void *>(&lora_grad_kernel<false, 2>)
                                       : reinterpret_cast<const void *>(&lora_grad_kernel<false, 1>);
        e = hipLaunchKernel(fn,
                            dim3((unsigned)(g.blocks0 + (c.M + 511) / 512), (unsigned)pieces_bound(c.N, c.L),
                                 (unsigned)((c.r + 16 * jt - 1) / (16 * jt))),
                            dim3(256), gargs, 0, stream);
        if (e != hipSuccess) return e;
    }
    g.blocks0 = (int)((c.K + 255) / 256);
    return hipLaunchKernel(reinterpret_cast<const void *>(&lora_grad_sum_kernel),
                           dim3((unsigned)(g.blocks0 + (c.M + 255) / 256), (unsigned)c.L, (unsigned)c.r), dim3(256),
                           gargs, 0, stream);
}

}  // namespace q4
