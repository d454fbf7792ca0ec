/*
 * q4_cache.h -- part of the C ABI of libq4: a paged cache of keys and values
 * kept in the affine 4-bit format of q4.h, and attention over it.
 *
 *   q4_cache_append  rotates new keys (and queries), packs keys and values,
 *                    and writes them to their slots;
 *   q4_cache_read    rows of the cache, dequantised;
 *   q4_cache_attend  softmax attention of new tokens over their sequences'
 *                    pages: single tokens, drafts, prompts and chunks of them.
 *
 * A layer of a serving step, between its projections:
 *   q4_cache_append(cache, k, v, slots, positions, inv_freq, q) -> q rotated
 *   q4_cache_attend(q, cache, table, lens, q_offsets)           -> out
 *
 * Conventions (device pointers, host checks before any launch, streams,
 * return codes) are those of q4.h.  Nothing is allocated, and no call waits
 * for the device: lengths, slots and page tables stay in device memory, so a
 * step can be captured once and replayed as its sequences grow.
 */
#ifndef Q4_CACHE_H
#define Q4_CACHE_H

#include "q4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define Q4_CACHE_MAX_HEADS 1024     /* heads of the cache, heads of q           */
#define Q4_CACHE_MAX_TOKENS 4194304 /* T, n, B * heads of one call              */
#define Q4_CACHE_MAX_KEYS 1073741824 /* table_pages * page of q4_cache_attend   */
#define Q4_CACHE_MAX_ROWS 536870912 /* T * q_heads of q4_cache_attend           */
#define Q4_CACHE_MAX_D 256          /* D: a multiple of 64 up to this           */
#define Q4_CACHE_MIN_PAGE 16        /* page: a power of two between these       */
#define Q4_CACHE_MAX_PAGE 4096

/*
 * A cache: for keys and for values one packed matrix in the affine format,
 * with pages * heads * page rows of D values.  Row (p, h, i) holds position i
 * of page p for head h; slot p * page + i names that position in all heads.
 *   codes: uint8 [pages][heads][page][D/2], 16-byte aligned;
 *   scales, zeros: fp16 bits [pages][heads][page][D/64], 16-byte aligned.
 * A value is (code - zero) * scale.  For q4_cache_attend zeros are integers
 * from 0 to 15 and scales positive or 0, not -0 (what q4_cache_append and
 * q4_pack_affine write), or NaN for a block that is; a token that sees a key
 * of other ones has unspecified results.  pages * page < 2^31.
 */
typedef struct {
    uint8_t *k_codes;
    uint16_t *k_scales, *k_zeros;
    uint8_t *v_codes;
    uint16_t *v_scales, *v_zeros;
    int64_t pages, heads, page, D;
} q4_cache;

/*
 * q4_cache_append -- for every token t < T with 0 <= slots[t] < pages * page:
 * the keys k[t] (rotated) and values v[t] of all heads, packed by the rule of
 * q4_pack_affine, written to the rows of that slot.  Another slot (-1 for
 * padding) is skipped.  The slots of one call are distinct: what the rows of
 * a slot given twice hold is unspecified (other rows are not affected).
 *   k, v: [T][heads][D] of in_type (Q4_OUT_F32 or Q4_OUT_BF16), 16-byte
 *     aligned; a token's heads are contiguous, tokens k_stride and v_stride
 *     elements apart (>= heads * D, a multiple of 16 bytes).
 *   Rotation: with a = positions[t] * inv_freq[i] for i < rot / 2, the pair
 *     (x1, x2) at dimensions (i, i + rot/2), or (2i, 2i + 1) if interleaved,
 *     becomes (f (x1 cos a - x2 sin a), f (x2 cos a + x1 sin a)) with
 *     f = amplitude; dimensions from rot on stay as they are.
 *     positions int32 [T], inv_freq fp32 [rot/2], 4-byte aligned; rot is a
 *     multiple of 16 up to D.  rot = 0: no rotation, both may be NULL.
 *   q: NULL, or the queries [T][q_heads][D] of in_type with q_stride as k;
 *     rotated like the keys into q_out, bf16 bits [T][q_heads][D], 16-byte
 *     aligned (every token's, whatever its slot).
 * Angles, the keys' rotation and the decisions of the packing are in 64 bits:
 * the packed row is that of the exact formula (but for decisions that 2^-50 of
 * the values would turn).  Queries are turned in fp32: q_out is within half a
 * bf16 step of a value that is within 2^-22 f (|x1| + |x2|) of the exact one.
 * A block of 64 values that holds a NaN or an infinity, or whose scale
 * rounds to an infinity, is written as NaN (scale NaN, codes and zero 0).
 * No output may overlap an input or another output.  T == 0 is a no-op.
 */
int q4_cache_append(const q4_cache *cache, const void *k, const void *v,
                    int in_type, int64_t T, int64_t k_stride, int64_t v_stride,
                    const int32_t *slots, const int32_t *positions,
                    const float *inv_freq, int64_t rot, int interleaved,
                    float amplitude, const void *q, int64_t q_heads,
                    int64_t q_stride, uint16_t *q_out, void *stream);

/*
 * q4_cache_read -- k_out[i][h], v_out[i][h] = the rows of slots[i], rounded
 * once to out_type (Q4_OUT_F32 or Q4_OUT_BF16); a slot outside the cache
 * reads as zeros.  slots int32 [n]; k_out, v_out [n][heads][D], 16-byte
 * aligned, one of them may be NULL.  n == 0 is a no-op.
 */
int q4_cache_read(const q4_cache *cache, const int32_t *slots, int64_t n,
                  int out_type, void *k_out, void *v_out, void *stream);

/*
 * q4_cache_attend -- for sequence b < B with lens[b] keys and the new tokens
 * q_offsets[b] .. q_offsets[b + 1] - 1 (n of them; q_offsets NULL: token b
 * alone): token j stands at position p = lens[b] - n + j and sees the keys
 * 0 .. p (causal), of these only p - window + 1 .. p where window > 0, or all
 * keys 0 .. lens[b] - 1 (causal == 0).  With the seen keys and values of head
 * h / (q_heads / heads) of the cache:
 *   s_i = scale * q . k_i;  out = sum_i exp(s_i) v_i / sum_i exp(s_i);
 *   lse = ln sum_i exp(s_i).
 * A token that sees no key, or only scores of -infinity, gets zeros and an
 * lse of -infinity.  Keys that a token does not see never reach its output,
 * whatever they hold; a NaN that it sees does, as in the formula: of a value
 * in the outputs of its block, of a key in all.  (The bits of its sums may
 * differ with what other tokens of the call see.)  A row of q that holds a NaN
 * or an infinity and sees a key gets NaN, or what the formula gives.  Weights,
 * and in prompts decoded values, are rounded to fp16 (2^-11 each, of themselves:
 * whatever other blocks and keys hold), in fp32 outputs too; keys are exact
 * where there are few tokens or lse is asked for, and rounded to fp16 otherwise,
 * so that the bits of out may differ between calls with lse and without.  lse
 * has the precision of fp32.  Scores are below 2^24 in magnitude (fp32 does not
 * hold the differences of larger ones, whose rows are unspecified).
 *   q: bf16 bits [T][q_heads][D], 16-byte aligned, tokens q_stride elements
 *     apart (>= q_heads * D, a multiple of 8).  q_heads is a multiple of
 *     heads.
 *   table: int32 [B][table_pages], the pages of each sequence in order; an
 *     entry that is needed and outside [0, pages) hides its keys.
 *   lens: int32 [B], held to 0 .. table_pages * page.
 *   q_offsets: int32 [B + 1], non-decreasing, held to 0 .. T.  Tokens outside
 *     every sequence keep what out and lse held.
 *   max_q: at most this many new tokens belong to one sequence (with
 *     q_offsets NULL: 1); tokens of a sequence past it keep what out and lse
 *     held.  It chooses the kernels and their grids: single tokens beside
 *     longer rows are faster in a call of their own.
 *   scale: finite and positive, whatever the size.  window >= 0, 0 where causal == 0.
 *   out: [T][q_heads][D] of out_type (Q4_OUT_F32 or Q4_OUT_BF16), 16-byte
 *     aligned.  lse: fp32 [T][q_heads], 4-byte aligned, or NULL.
 *   workspace: q4_cache_attend_ws_bytes(...) bytes, 16-byte aligned; calls
 *     that may run at the same time need different ones.
 * T == 0 or B == 0 is a no-op.
 */
size_t q4_cache_attend_ws_bytes(int64_t T, int64_t q_heads, int64_t heads,
                                int64_t D, int64_t B, int64_t max_q);
int q4_cache_attend(const uint16_t *q, int64_t T, int64_t q_heads,
                    int64_t q_stride, const q4_cache *cache,
                    const int32_t *table, int64_t B, int64_t table_pages,
                    const int32_t *lens, const int32_t *q_offsets,
                    int64_t max_q, int causal, int64_t window, float scale,
                    int out_type, void *out, float *lse, void *workspace,
                    size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif
#endif /* Q4_CACHE_H */
