/*
 * q4_lora.h -- part of the C ABI of libq4: low-rank adapters beside a packed
 * projection (the NF4-style format of q4.h), for many requests at once, and
 * their backward pass with the packed matrix frozen.
 *
 *   Y[n]  = What X[n] + s_a B_a (A_a X[n]),   a = ids[n]
 *
 *   A: bf16 bits [L][r][K], B: bf16 bits [L][M][r] (16-byte aligned; adapters
 *     of lower rank are padded with zeros), scaling: fp32 [L].
 *   ids: int32 [N]; a token whose id lies outside [0, L) has no adapter.
 *   r: a multiple of 8, 8 <= r <= Q4_MAX_RANK.
 *
 * Conventions (device pointers, host checks before any launch, streams,
 * return codes) are those of q4.h.  Workspaces are 16-byte aligned; calls
 * that may run at the same time need different ones.
 */
#ifndef Q4_LORA_H
#define Q4_LORA_H

#include "q4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define Q4_MAX_RANK 128
#define Q4_MAX_ADAPTERS 1024
#define Q4_MAX_TOKENS ((int64_t)1 << 22) /* N                                    */

/*
 * q4_gemm_lora -- the formula above for any number N of tokens.
 *   X: bf16 bits [N][K], 16-byte aligned; Y: [N][M] of out_type (Q4_OUT_F32
 *   or Q4_OUT_BF16), 16-byte aligned, overlapping no input.
 *   With L == 0 the adapter arrays may be NULL and Y = What X.
 * Accuracy: the packed product as q4_gemm_grouped; A_a X[n] in fp32, carried
 * to the second product to 2^-16 of each value; one rounding to out_type.
 * Values of one adapter that are not finite reach only its own tokens.
 * N == 0 or M == 0 is a no-op.
 */
size_t q4_gemm_lora_ws_bytes(int64_t M, int64_t K, int64_t N, int64_t r,
                             int64_t L);
int q4_gemm_lora(const uint8_t *codes, const uint16_t *scales, int64_t M,
                 int64_t K, const uint16_t *X, int64_t N, const uint16_t *A,
                 const uint16_t *B, const float *scaling, const int32_t *ids,
                 int64_t r, int64_t L, int out_type, void *Y, void *workspace,
                 size_t workspace_bytes, void *stream);

/*
 * q4_gemm_lora_backward -- for dY bf16 bits [N][M] (16-byte aligned), with
 * u[n] = s_a B_a^T dY[n]:
 *   dX[n][k]    = sum_m What[m,k] dY[n][m] + sum_j A_a[j,k] u[n][j]
 *                 (bf16 bits [N][K], 16-byte aligned)
 *   dA[a][j][k] = sum over n with ids[n] == a of u[n][j] X[n][k]
 *   dB[a][m][j] = s_a * sum over n with ids[n] == a of dY[n][m] (A_a X[n])[j]
 *                 (fp32, 16-byte aligned; adapters without a token get 0)
 * dX may be NULL (the first layer), as may dA and dB together (frozen
 * adapters).  Sums are added in a fixed order: every call gives the same bits.
 * Accuracy: the packed product of dX is within (2^-10 + (M + 64) 2^-24) *
 * sum_m |What dY| + 2^-25 * sum_m s_m |dY_m| + 2^-26 * M * max_m s_m |dY_m| of
 * its exact value, s_m the largest |scale| of packed row m; u is carried to
 * 2^-16 of each value, one rounding to bf16; dA and dB in fp32.
 * M >= 1 (a matrix of no rows has no gradients and is refused as a shape);
 * N == 0 clears dA and dB.
 */
size_t q4_gemm_lora_backward_ws_bytes(int64_t M, int64_t K, int64_t N,
                                      int64_t r, int64_t L);
int q4_gemm_lora_backward(const uint16_t *dY, const uint8_t *codes,
                          const uint16_t *scales, int64_t M, int64_t K,
                          const uint16_t *X, int64_t N, const uint16_t *A,
                          const uint16_t *B, const float *scaling,
                          const int32_t *ids, int64_t r, int64_t L,
                          uint16_t *dX, float *dA, float *dB, void *workspace,
                          size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* Q4_LORA_H */
