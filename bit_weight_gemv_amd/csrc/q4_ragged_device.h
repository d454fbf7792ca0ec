// q4_ragged_device.h -- pieces shared by the ragged products, the router and
// the adapters' kernels (gfx950).
#pragma once

#include "q4_device.h"
#include "q4_lut.h"
#include "q4_ragged.h"

namespace q4 {

typedef _Float16 half8_t __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float bf16_lo(uint32_t d) { return __builtin_bit_cast(float, d << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t d) { return __builtin_bit_cast(float, d & 0xFFFF0000u); }
__device__ __forceinline__ float bf16_f32(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }
// Nearest even.
__device__ __forceinline__ uint16_t f32_bf16(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

__device__ __forceinline__ void store_out(void *Y, bool bf16, int64_t at, float v) {
    if (bf16) static_cast<uint16_t *>(Y)[at] = f32_bf16(v);
    else static_cast<float *>(Y)[at] = v;
}

__device__ __forceinline__ float load_out(const void *Y, bool bf16, int64_t at) {
    return bf16 ? bf16_f32(static_cast<const uint16_t *>(Y)[at]) : static_cast<const float *>(Y)[at];
}

// silu(g) * u; for g below -88 e^-g overflows to infinity and the quotient is -0.
__device__ __forceinline__ float swiglu(float g, float u) { return g / (1.0f + __expf(-g)) * u; }

// A piece of at most `most` rows of one group.
struct Chunk {
    int e;      // group
    int start;  // first position
    int count;  // rows (0: no such chunk)
};

// Rows of group e, its offsets held to 0 .. R.
__device__ __forceinline__ int group_rows(const int32_t *__restrict__ offsets, int E, int R, int e, int &lo) {
    lo = 0;
    if (e >= E) return 0;
    lo = min(max(offsets[e], 0), R);
    return max(min(max(offsets[e + 1], 0), R) - lo, 0);
}

// Chunk c of the groups cut into pieces of `most` rows, in order.  Every lane
// of the wave returns the same values.
__device__ __forceinline__ Chunk find_chunk(const int32_t *__restrict__ offsets, int E, int R, int c, int most) {
    if (!offsets) {
        const int64_t s = (int64_t)c * most;
        if (s >= R) return {0, 0, 0};
        return {0, (int)s, min(most, R - (int)s)};
    }
    const int lane = threadIdx.x & 63;
    int base = 0;
    for (int e0 = 0; e0 < E; e0 += 64) {
        const int e = e0 + lane;
        int lo;
        const int n = group_rows(offsets, E, R, e, lo);
        const int pieces = (n + most - 1) / most;
        int incl = pieces;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int o = __shfl_up(incl, d);
            if (lane >= d) incl += o;
        }
        const int first = base + incl - pieces;
        const uint64_t hit = __builtin_amdgcn_ballot_w64(c >= first && c < first + pieces);
        if (hit) {
            const int src = __builtin_ctzll(hit);
            const int s = (c - first) * most;
            Chunk k;
            k.e = __builtin_amdgcn_readlane(e, src);
            k.start = __builtin_amdgcn_readlane(lo + s, src);
            k.count = __builtin_amdgcn_readlane(min(most, n - s), src);
            return k;
        }
        base += __builtin_amdgcn_readlane(incl, 63);
    }
    return {0, 0, 0};
}

// Number of chunks of at most `most` rows.
__device__ __forceinline__ int count_chunks(const int32_t *__restrict__ offsets, int E, int R, int most) {
    if (!offsets) return (R + most - 1) / most;
    int total = 0;
    for (int e = threadIdx.x & 63; e < E + 63; e += 64) {
        int lo;
        total += (group_rows(offsets, E, R, e, lo) + most - 1) / most;
        if (e - (int)(threadIdx.x & 63) + 64 >= E) break;
    }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) total += __shfl_xor(total, d);
    return total;
}

// The share of workgroup `w` of `wgs` (at least as many as there are chunks):
// a chunk, and the part'th of the nparts that its row tiles are dealt to.
struct Share {
    Chunk chunk;  // count 0: nothing
    int part, nparts;
};
__device__ __forceinline__ Share find_share(const int32_t *__restrict__ offsets, int E, int R, int most, int w,
                                            int wgs) {
    const int n = __builtin_amdgcn_readfirstlane(count_chunks(offsets, E, R, most));
    if (n == 0) return {{0, 0, 0}, 0, 1};
    const int c = w % n;
    return {find_chunk(offsets, E, R, c, most), w / n, (wgs - c - 1) / n + 1};
}

// Shift that puts a bf16 row's largest magnitude (given as its bits) into
// fp16's upper range [2^14, 2^15); held to what one fp32 power of two can do
// (a row below 2^-113 then stays smaller), and taken as for the largest
// finite exponent where the row holds an infinity or a NaN.
__device__ __forceinline__ int fp16_shift(uint32_t maxbits) {
    const int E = min((int)(maxbits >> 7), 254);
    return min(141 - E, 127);
}

// Two bf16 of a dword, each times 2^shift (f), as two fp16.  Exact where the
// result is an fp16 normal number, towards zero below that.
__device__ __forceinline__ uint32_t bf16x2_to_f16x2(uint32_t d, float f) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_pkrtz(bf16_lo(d) * f, bf16_hi(d) * f));
}

// Workgroup `block` (of 256) of those that write the rows of X (bf16 [T][K];
// position p takes rows[p], or row p; one outside [0, T): zeros) as pieces: a
// lane converts one piece, the 32 lanes of a half-wave a slice of a position.
__device__ __forceinline__ void write_pieces(const uint16_t *__restrict__ X, const int32_t *__restrict__ rows, int K,
                                             int T, int R, const Pieces &out, int block) {
    const int pairs = (R + 1) >> 1, slices = (K + 255) >> 8;
    const int w = block * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    const int slice = w / pairs, p = (w % pairs) * 2 + (lane >> 5), piece = slice * 32 + (lane & 31);
    const bool live = slice < slices && p < R && piece < K / 8;
    u32x4_t v = {0u, 0u, 0u, 0u};
    if (live) {
        const int row = rows ? rows[p] : p;
        if (row >= 0 && row < T) v = reinterpret_cast<const u32x4_t *>(X + (int64_t)row * K)[piece];
    }
    u16x2_t mx = {0, 0};
#pragma unroll
    for (int c = 0; c < 4; ++c) mx = __builtin_elementwise_max(mx, __builtin_bit_cast(u16x2_t, v[c] & 0x7FFF7FFFu));
    int m = max((int)mx.x, (int)mx.y);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = max(m, __shfl_xor(m, d));
    const int shift = fp16_shift((uint32_t)m);
    const float f = exp2i(shift);
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = bf16x2_to_f16x2(v[c], f);
    if (live) {
        reinterpret_cast<u32x4_t *>(out.x16)[(int64_t)piece * R + p] = v;
        if ((lane & 31) == 0) out.exps[(int64_t)slice * R + p] = -shift;
    }
}

// A workgroup of 256 takes the 16 packed rows from row0 (below nrows; matrices
// of M rows, nb blocks a row, one after the other): the exponent of each row's
// largest scale (ZERO in a row of zeros), and scale 2^(14 - exponent) as fp16 at
// [matrix][block][row].
template <int ZERO, typename E>
__device__ __forceinline__ void prepare_scales(const uint16_t *__restrict__ scales, int64_t row0, int64_t nrows, int M,
                                               int nb, E *__restrict__ rowexp, uint16_t *__restrict__ out) {
    __shared__ int16_t exps[16];
    __syncthreads();
    {
        const int64_t row = row0 + (threadIdx.x >> 4);
        int m = 0;
        if (row < nrows)
            for (int b = threadIdx.x & 15; b < nb; b += 16) m = max(m, (int)(scales[row * nb + b] & 0x7FFF));
#pragma unroll
        for (int d = 8; d >= 1; d >>= 1) m = max(m, __shfl_xor(m, d));
        const float f = f16_bits_to_f32((uint32_t)m);
        const int e = m == 0 ? ZERO : min((int)(__builtin_bit_cast(uint32_t, f) >> 23) - 127, 16);
        if ((threadIdx.x & 15) == 0) {
            exps[threadIdx.x >> 4] = (int16_t)e;
            if (row < nrows) rowexp[row] = (E)e;
        }
    }
    __syncthreads();
    const int64_t row = row0 + (threadIdx.x & 15);
    if (row >= nrows) return;
    const int e = exps[threadIdx.x & 15];
    const int64_t mat = row / M;
    for (int b = threadIdx.x >> 4; b < nb; b += 16)
        out[(mat * nb + b) * M + (row - mat * M)] =
            __builtin_bit_cast(uint16_t, (_Float16)ldexpf(f16_bits_to_f32(scales[row * nb + b]), 14 - e));
}

// Eight bf16 of a row at column k; zeros past its end.  VEC: rows start on 16
// bytes and have whole pieces.
template <bool VEC>
__device__ __forceinline__ u32x4_t row_piece(const uint16_t *row, int k, int K) {
    u32x4_t v = {0u, 0u, 0u, 0u};
    if constexpr (VEC) {
        if (k < K) v = *reinterpret_cast<const u32x4_t *>(row + k);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i < K) v[i >> 1] |= (uint32_t)row[k + i] << (16 * (i & 1));
    }
    return v;
}

__device__ __forceinline__ float dot8(const u32x4_t &x, const u32x4_t &z, float s) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        s = fmaf(bf16_lo(x[c]), bf16_lo(z[c]), s);
        s = fmaf(bf16_hi(x[c]), bf16_hi(z[c]), s);
    }
    return s;
}

// t[n][j] = scaling[a] * sum_k Z[a][j][k] x[n][k], a = ids[n], by one wave
// (nothing where the token has no adapter).
template <bool VEC = true>
__device__ __forceinline__ void shrink_row(const uint16_t *X, const uint16_t *Z, const float *scaling,
                                           const int32_t *ids, int K, int pitch, int r, int L, int n, int j, int N,
                                           float *t) {
    if (n >= N || j >= r) return;
    const int id = ids[n];
    if (id < 0 || id >= L) return;
    const int lane = threadIdx.x & 63;
    const uint16_t *x = X + (int64_t)n * K, *z = Z + ((int64_t)id * r + j) * pitch;
    float s = 0.0f;
#pragma unroll 4
    for (int k = lane * 8; k < K; k += 512)
        s = dot8(row_piece<VEC>(x, k, K), *reinterpret_cast<const u32x4_t *>(z + k), s);
    s = wave_sum(s);
    if (lane == 0) t[(int64_t)n * r + j] = s * scaling[id];
}

// Eight weights of four code bytes, as fp16 table entries.
__device__ __forceinline__ void lut8(const uint32_t *lut, uint32_t word, uint32_t laneoff, half2_t (&w)[4]) {
    w[0] = lut_pair<0>(lut, word, laneoff);
    w[1] = lut_pair<1>(lut, word, laneoff);
    w[2] = lut_pair<2>(lut, word, laneoff);
    w[3] = lut_pair<3>(lut, word, laneoff);
}

__device__ __forceinline__ half8_t join8(const half2_t (&w)[4]) {
    const u32x4_t v = {__builtin_bit_cast(uint32_t, w[0]), __builtin_bit_cast(uint32_t, w[1]),
                       __builtin_bit_cast(uint32_t, w[2]), __builtin_bit_cast(uint32_t, w[3])};
    return __builtin_bit_cast(half8_t, v);
}

// A 32 x 32 tile of v_mfma_f32_32x32x16: lane l holds column l % 32 and, in
// register i, row 8 (i / 4) + 4 (l / 32) + i % 4.
__device__ __forceinline__ int tile_row(int i, int lane) { return 8 * (i >> 2) + 4 * (lane >> 5) + (i & 3); }

// v as the sum of two bf16: the nearest one and the nearest to what it leaves
// (2^-17 of v at most is lost).  An infinity or a NaN stands alone.
__device__ __forceinline__ void split2(const float (&v)[8], bf16x8_t &hi, bf16x8_t &lo) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const __bf16 h = (__bf16)v[i];
        const float rest = v[i] - (float)h;
        hi[i] = h;
        lo[i] = (__bf16)(fabsf(rest) < __builtin_inff() ? rest : 0.0f);
    }
}

// An adapter's term is added to a tile of tokens by matrix cores, with zeros in
// the rows of tokens that do not use it.  Those zeros times an infinity or a NaN
// of the adapter would be NaN, so such values enter the tile as 1 of their sign
// (an infinity of the token's own stays one), and what they add is added to the
// finished outputs of the adapter's tokens alone.  Held beside the tile, as
// products of their own, they took 14 us of the 267 of 4093 tokens.
__device__ __forceinline__ bool not_finite8(const u32x4_t &v) {
    u16x2_t mx = {0, 0};
#pragma unroll
    for (int c = 0; c < 4; ++c) mx = __builtin_elementwise_max(mx, __builtin_bit_cast(u16x2_t, v[c] & 0x7FFF7FFFu));
    return max((int)mx.x, (int)mx.y) >= 0x7F80;
}
__device__ __forceinline__ u32x4_t finite8(u32x4_t v) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if ((v[c] & 0x7F80u) == 0x7F80u) v[c] = (v[c] & 0xFFFF8000u) | 0x3F80u;
        if ((v[c] & 0x7F800000u) == 0x7F800000u) v[c] = (v[c] & 0x8000FFFFu) | 0x3F800000u;
    }
    return v;
}
// sum_j t[j] b[j pitch] over the values of b that are not finite; 0 where all are.
__device__ __forceinline__ float wild_term(const float *t, const uint16_t *b, int64_t pitch, int r) {
    float s = 0.0f;
    for (int j = 0; j < r; ++j) {
        const uint16_t v = b[j * pitch];
        if ((v & 0x7F80u) == 0x7F80u) s += t[j] * bf16_f32(v);
    }
    return s;
}

}  // namespace q4
