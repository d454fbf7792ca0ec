/*
 * q4_experts.h -- part of the C ABI of libq4: feed-forward layers of many
 * experts whose matrices are in the NF4-style packed format of q4.h.
 *
 *   q4_route_topk    router logits -> the experts of each token, their
 *                    weights, and the plan that groups tokens by expert;
 *   q4_gemm_grouped  the packed product of every group of rows with its
 *                    expert's matrix (ragged groups, any of them empty), plain
 *                    or as silu(gate) * up;
 *   q4_moe_combine   the weighted sum of each token's expert outputs.
 *
 * A layer is four calls:
 *   q4_route_topk  (logits)                          -> weights, offsets, rows, pos
 *   q4_gemm_grouped(gate, up, X,  offsets, rows)     -> H   [T k][F]
 *   q4_gemm_grouped(down,     H,  offsets, NULL)     -> Y   [T k][M]
 *   q4_moe_combine (Y, weights, pos)                 -> out [T][M]
 *
 * Conventions (device pointers, host checks before any launch, streams,
 * return codes) are those of q4.h.  Nothing is allocated, and no call waits
 * for the device: group sizes stay in device memory.
 */
#ifndef Q4_EXPERTS_H
#define Q4_EXPERTS_H

#include "q4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define Q4_MAX_EXPERTS 1024
#define Q4_MAX_TOPK 16
#define Q4_MAX_SLOTS ((int64_t)1 << 22) /* T k, R and T: rows of one call      */
#define Q4_MAX_ROWS ((int64_t)1 << 24)  /* M: rows of one matrix              */

#define Q4_ROUTE_TOPK 0 /* softmax over the k chosen logits                   */
#define Q4_ROUTE_ALL 1  /* softmax over all E logits, the k chosen kept       */

/*
 * q4_route_topk -- logits [T][E] (type Q4_OUT_F32 or Q4_OUT_BF16, aligned to
 * its element) to, for 1 <= k <= min(E, Q4_MAX_TOPK):
 *   experts int32 [T][k]: the k largest logits of a token in descending
 *     order, equal logits by ascending index; NaN counts as -infinity.
 *   weights fp32 [T][k]: p_j / sum p with p_j = 1 where l_j equals the token's
 *     largest logit and exp(l_j - largest) elsewhere, the sum over the chosen
 *     (Q4_ROUTE_TOPK) or over all (Q4_ROUTE_ALL).  A token whose logits are
 *     all -infinity (or NaN) gets weights of 0.
 *   offsets int32 [E + 1]: the slots (token, choice) of expert e are positions
 *     offsets[e] .. offsets[e + 1] - 1 of the grouped order.
 *   rows int32 [T k]: the token at each position.
 *   pos int32 [T][k]: the position of each slot.
 * Slots of one expert keep their order, so every call gives the same plan.
 * All outputs 4-byte aligned; no output may overlap the logits or another.
 *   workspace: q4_route_topk_ws_bytes(T, E, k) bytes, 16-byte aligned (may be
 *     NULL where that is 0).
 * T == 0 clears offsets.  E <= Q4_MAX_EXPERTS, T k <= Q4_MAX_SLOTS.
 */
size_t q4_route_topk_ws_bytes(int64_t T, int64_t E, int64_t k);
int q4_route_topk(const void *logits, int logits_type, int64_t T, int64_t E,
                  int64_t k, int mode, int32_t *experts, float *weights,
                  int32_t *offsets, int32_t *rows, int32_t *pos,
                  void *workspace, size_t workspace_bytes, void *stream);

/*
 * q4_gemm_grouped -- for every position p of group e (offsets[e] <= p <
 * offsets[e + 1]), with x = X[rows[p]] (X[p] where rows is NULL):
 *   up_codes NULL:  Y[p][m] = sum_k What_e[m,k] x[k]
 *   otherwise:      Y[p][m] = silu(sum_k What_e[m,k] x[k])
 *                             * sum_k Up_e[m,k] x[k]
 *   codes, scales (and up_codes, up_scales): E packed M x K matrices, one
 *     after the other (codes 16-byte, scales 2-byte aligned).
 *   X: bf16 bits [T][K], 16-byte aligned.
 *   offsets: int32 [E + 1], non-decreasing within 0 .. R.  Positions outside
 *     every group keep what Y held.  (Values outside that contract are held
 *     to 0 .. R: no access leaves the buffers, the results are unspecified.)
 *   rows: int32 [R] or NULL; a row outside [0, T) reads as zeros (with rows
 *     NULL, where R > T: every position from T on).
 *   Y: [R][M] of out_type (Q4_OUT_F32 or Q4_OUT_BF16), 16-byte aligned.
 * Accuracy: each sum is within (2^-10 + (K + 64) 2^-24) * sum_k |What x| +
 * 2^-27 * (max_k |x| * sum_k |What| + max_b |scale_b| * sum_k |x|) of its
 * exact value: fp16 table entries, times the block's scale rounded to fp16
 * (under a power of two per row; calls of single rows take the scale in
 * fp32), activations in fp16 under a power of two per row, exact where they
 * are above 2^-28 of the row's largest, fp32 sums.  Unlike the products of
 * q4.h, smaller activations lose bits, and the scaled weight is rounded: with
 * bf16 outputs their own rounding covers both, with fp32 outputs the error
 * (2.2e-4 of the outputs' magnitude, 1.6e-4 from the table entries alone) is
 * this one.  silu is within 2^-16 of its value and -0 for sums below -88; it
 * and the product are in fp32, with one rounding to out_type.  A non-finite
 * activation reaches only the outputs of its own row, as in the formula
 * (a weight of 0 times an infinity is NaN).
 *   workspace: q4_gemm_grouped_ws_bytes(...) bytes, 16-byte aligned; calls
 *     that may run at the same time need different ones.
 * R == 0 or M == 0 is a no-op; T == 0 makes every row zeros.
 */
size_t q4_gemm_grouped_ws_bytes(int64_t E, int64_t M, int64_t K, int64_t T,
                                int64_t R, int has_up);
int q4_gemm_grouped(const uint8_t *codes, const uint16_t *scales,
                    const uint8_t *up_codes, const uint16_t *up_scales,
                    int64_t E, int64_t M, int64_t K, const uint16_t *X,
                    int64_t T, const int32_t *offsets, const int32_t *rows,
                    int64_t R, int out_type, void *Y, void *workspace,
                    size_t workspace_bytes, void *stream);

/*
 * q4_moe_combine -- out[t][m] = sum_s weights[t][s] * Y[pos[t][s]][m], the
 * products added in fp32 in the order of s, one rounding to out_type.
 *   Y: [R][M] of y_type (Q4_OUT_F32 or Q4_OUT_BF16), 16-byte aligned.
 *   weights fp32 [T][k], pos int32 [T][k] (4-byte aligned): a position outside
 *     [0, R) adds nothing, whatever its weight.
 *   out: [T][M] of out_type, 16-byte aligned, overlapping no input.
 * T == 0 or M == 0 is a no-op; 1 <= k <= Q4_MAX_TOPK.
 */
int q4_moe_combine(const void *Y, int y_type, int64_t R, int64_t M,
                   const float *weights, const int32_t *pos, int64_t T,
                   int64_t k, int out_type, void *out, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* Q4_EXPERTS_H */
