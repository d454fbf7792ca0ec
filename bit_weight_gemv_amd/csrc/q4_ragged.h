// q4_ragged.h -- the packed product of ragged groups of rows (host side):
// what the experts' and the adapters' entry points share.  Not exported.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace q4 {

// Y[p] = What_e X[row(p)] for the positions p of group e, or, with up_codes,
// silu(What_e x) * (Up_e x); with B, plus the low-rank term of the position's
// adapter, sum_j t[p][j] B[ids[p]][m][j].
struct RaggedProduct {
    const uint8_t *codes, *up_codes;    // E packed matrices each; up_codes null: plain
    const uint16_t *scales, *up_scales;
    int64_t E, M, K;
    const uint16_t *X;                  // bf16 [T][K]
    int64_t T;
    const int32_t *offsets;             // [E + 1], or null: one group of R rows (E == 1)
    const int32_t *rows;                // [R], or null: row p
    int64_t R;
    bool bf16;                          // output type
    void *Y;
    const uint16_t *B;                  // bf16 [L][M][r], or null
    const float *t;                     // fp32 [R][r], the adapter's scaling in it
    const uint16_t *A;                  // where ragged_shrinks holds: what t is made of
    const float *scaling;
    const int32_t *ids;                 // [R]
    int64_t r, L;
};

// Whether the launches of this shape stay within what a grid can hold.
bool ragged_fits(int64_t E, int64_t M, int64_t K, int64_t T, int64_t R, bool up);
size_t ragged_ws_bytes(int64_t E, int64_t M, int64_t K, int64_t T, int64_t R, bool up, int64_t r);
hipError_t launch_ragged(const RaggedProduct &p, void *workspace, hipStream_t stream);

inline size_t round16(size_t n) { return (n + 15) & ~(size_t)15; }

// The activations of R positions as the few-rows kernel reads them: fp16
// times 2^exps[slice of 256 k][position], in pieces of 8 k, [K / 8][R][8].
// They lie at the start of the product's workspace; where
// ragged_takes_pieces holds beside an adapter (lora), the adapters' first
// launch writes them.
struct Pieces {
    uint16_t *x16;
    int32_t *exps;
};
inline size_t pieces_bytes(int64_t K, int64_t R) {
    return round16((size_t)K * R * 2) + round16((size_t)((K + 255) / 256) * R * 4);
}
inline Pieces pieces_at(int64_t K, int64_t R, void *workspace) {
    char *w = static_cast<char *>(workspace);
    return {reinterpret_cast<uint16_t *>(w), reinterpret_cast<int32_t *>(w + round16((size_t)K * R * 2))};
}
// Workgroups that write them: a wave takes a slice of two positions.
inline int64_t pieces_blocks(int64_t K, int64_t R) { return ((K + 255) / 256 * ((R + 1) / 2) + 3) / 4; }
// Whether the product itself makes t (written to p.t) beside its first launch.
bool ragged_shrinks(int64_t E, int64_t M, int64_t K, int64_t R, int64_t r);
bool ragged_takes_pieces(int64_t E, int64_t M, int64_t K, int64_t R, int64_t r);

// The current device's number of compute units (256 where it cannot be read).
int compute_units();

// Slots sorted by bin, in order within a bin: bins[i] outside [0, E) goes
// behind the last bin.  offsets [E + 1]; at position p: the slot's number
// divided by `per`, in rows; pos (or null): the position of each slot.
size_t sort_ws_bytes(int64_t slots, int64_t E);
hipError_t launch_sort(const int32_t *bins, int64_t slots, int64_t E, int64_t per, int32_t *offsets, int32_t *rows,
                       int32_t *pos, void *workspace, hipStream_t stream);

// Router and weighted sum.
size_t route_ws_bytes(int64_t T, int64_t E, int64_t k);
hipError_t launch_route(const void *logits, bool bf16, int64_t T, int64_t E, int64_t k, bool all, int32_t *experts,
                        float *weights, int32_t *offsets, int32_t *rows, int32_t *pos, void *workspace,
                        hipStream_t stream);
bool combine_fits(int64_t M, int64_t T);  // (within what a grid can hold)
hipError_t launch_combine(const void *Y, bool y_bf16, int64_t R, int64_t M, const float *weights, const int32_t *pos,
                          int64_t T, int64_t k, bool out_bf16, void *out, hipStream_t stream);

// Adapters.
struct LoraCall {
    const uint8_t *codes;
    const uint16_t *scales;
    int64_t M, K;
    const uint16_t *X;   // bf16 [N][K]
    int64_t N;
    const uint16_t *A, *B;
    const float *scaling;
    const int32_t *ids;
    int64_t r, L;
};
size_t lora_ws_bytes(int64_t M, int64_t K, int64_t N, int64_t r, int64_t L);
hipError_t launch_lora(const LoraCall &c, bool bf16, void *Y, void *workspace, hipStream_t stream);
bool lora_backward_fits(int64_t M, int64_t K, int64_t N, int64_t L);
size_t lora_backward_ws_bytes(int64_t M, int64_t K, int64_t N, int64_t r, int64_t L);
hipError_t launch_lora_backward(const LoraCall &c, const uint16_t *dY, uint16_t *dX, float *dA, float *dB,
                                void *workspace, hipStream_t stream);

}  // namespace q4
