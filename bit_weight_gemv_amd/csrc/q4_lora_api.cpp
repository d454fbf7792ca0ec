// q4_lora_api.cpp -- the exported entry points of q4_lora.h: argument checks
// on the host, then the launches on the caller's stream.
#include "q4_lora.h"

#include "q4_checks.h"
#include "q4_ragged.h"

using namespace q4::checks;

namespace {

bool lora_shape_ok(int64_t M, int64_t K, int64_t N, int64_t r, int64_t L) {
    if (M < 0 || M > (INT64_C(1) << 24) || !k_ok(K) || N < 0 || N > Q4_MAX_TOKENS || L < 0 || L > Q4_MAX_ADAPTERS)
        return false;
    if (L > 0 && (r < 8 || r > Q4_MAX_RANK || r % 8 != 0)) return false;
    return q4::ragged_fits(1, M, K, N, N, false);
}

bool backward_shape_ok(int64_t M, int64_t K, int64_t N, int64_t r, int64_t L) {
    return lora_shape_ok(M, K, N, r, L) && q4::lora_backward_fits(M, K, N, L);
}

int workspace_check(size_t need, void *workspace, size_t bytes, Range *out, int nout, const Range *in, int nin) {
    if (need == 0) return Q4_OK;
    if (!workspace || bytes < need) return Q4_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return Q4_ERR_ALIGN;
    out[nout] = range_of(workspace, need);
    return clash(out, nout + 1, in, nin) ? Q4_ERR_OVERLAP : Q4_OK;
}

}  // namespace

extern "C" {

size_t q4_gemm_lora_ws_bytes(int64_t M, int64_t K, int64_t N, int64_t r, int64_t L) {
    if (!lora_shape_ok(M, K, N, r, L) || M == 0 || N == 0) return 0;
    return q4::lora_ws_bytes(M, K, N, r, L);
}

int q4_gemm_lora(const uint8_t *codes, const uint16_t *scales, int64_t M, int64_t K, const uint16_t *X, int64_t N,
                 const uint16_t *A, const uint16_t *B, const float *scaling, const int32_t *ids, int64_t r, int64_t L,
                 int out_type, void *Y, void *workspace, size_t workspace_bytes, void *stream) {
    if (!type_ok(out_type) || !lora_shape_ok(M, K, N, r, L)) return Q4_ERR_SHAPE;
    if (M == 0 || N == 0) return Q4_OK;
    if (!codes || !scales || !X || !Y || (L > 0 && (!A || !B || !scaling || !ids))) return Q4_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 2) || !aligned(X, 16) || !aligned(Y, 16)) return Q4_ERR_ALIGN;
    if (L > 0 && (!aligned(A, 16) || !aligned(B, 16) || !aligned(scaling, 4) || !aligned(ids, 4))) return Q4_ERR_ALIGN;
    if (L == 0) r = 0;
    const Range in[7] = {range_of(codes, (uint64_t)M * (K / 2)),
                         range_of(scales, (uint64_t)M * (K / 64) * 2),
                         range_of(X, (uint64_t)N * K * 2),
                         range_of(A, (uint64_t)L * r * K * 2),
                         range_of(B, (uint64_t)L * r * M * 2),
                         range_of(scaling, (uint64_t)L * 4),
                         range_of(ids, L > 0 ? (uint64_t)N * 4 : 0)};
    Range out[2] = {range_of(Y, (uint64_t)N * M * elt(out_type)), {0, 0}};
    if (clash(out, 1, in, 7)) return Q4_ERR_OVERLAP;
    const int st = workspace_check(q4::lora_ws_bytes(M, K, N, r, L), workspace, workspace_bytes, out, 1, in, 7);
    if (st != Q4_OK) return st;
    const q4::LoraCall c = {codes, scales, M, K, X, N, A, B, scaling, ids, r, L};
    return launch_status(q4::launch_lora(c, out_type == Q4_OUT_BF16, Y, workspace, (hipStream_t)stream));
}

size_t q4_gemm_lora_backward_ws_bytes(int64_t M, int64_t K, int64_t N, int64_t r, int64_t L) {
    if (!backward_shape_ok(M, K, N, r, L) || M == 0) return 0;
    return q4::lora_backward_ws_bytes(M, K, N, L > 0 ? r : 0, L);
}

int q4_gemm_lora_backward(const uint16_t *dY, const uint8_t *codes, const uint16_t *scales, int64_t M, int64_t K,
                          const uint16_t *X, int64_t N, const uint16_t *A, const uint16_t *B, const float *scaling,
                          const int32_t *ids, int64_t r, int64_t L, uint16_t *dX, float *dA, float *dB,
                          void *workspace, size_t workspace_bytes, void *stream) {
    if (M == 0 || !backward_shape_ok(M, K, N, r, L)) return Q4_ERR_SHAPE;
    if ((dA == nullptr) != (dB == nullptr) || (!dX && !dA)) return Q4_ERR_NULL;
    if (N > 0 && (!dY || (dX && (!codes || !scales)) || (dA && !X))) return Q4_ERR_NULL;
    if (N > 0 && L > 0 && (!A || !B || !scaling || !ids)) return Q4_ERR_NULL;
    if (!aligned(dY, 16) || !aligned(codes, 16) || !aligned(scales, 2) || !aligned(X, 16) || !aligned(dX, 16) ||
        !aligned(dA, 16) || !aligned(dB, 16))
        return Q4_ERR_ALIGN;
    if (L > 0 && (!aligned(A, 16) || !aligned(B, 16) || !aligned(scaling, 4) || !aligned(ids, 4))) return Q4_ERR_ALIGN;
    if (L == 0) {
        r = 0;
        if (!dX) return Q4_OK;  // (gradients of no adapter)
    }
    const Range in[8] = {range_of(dY, (uint64_t)N * M * 2),
                         range_of(codes, (uint64_t)M * (K / 2)),
                         range_of(scales, (uint64_t)M * (K / 64) * 2),
                         range_of(X, (uint64_t)N * K * 2),
                         range_of(A, (uint64_t)L * r * K * 2),
                         range_of(B, (uint64_t)L * r * M * 2),
                         range_of(scaling, (uint64_t)L * 4),
                         range_of(ids, L > 0 ? (uint64_t)N * 4 : 0)};
    Range out[4] = {range_of(dX, (uint64_t)N * K * 2), range_of(dA, (uint64_t)L * r * K * 4),
                    range_of(dB, (uint64_t)L * r * M * 4), {0, 0}};
    if (clash(out, 3, in, 8)) return Q4_ERR_OVERLAP;
    const int st =
        workspace_check(q4::lora_backward_ws_bytes(M, K, N, r, L), workspace, workspace_bytes, out, 3, in, 8);
    if (st != Q4_OK) return st;
    const q4::LoraCall c = {codes, scales, M, K, X, N, A, B, scaling, ids, r, L};
    return launch_status(q4::launch_lora_backward(c, dY, dX, dA, dB, workspace, (hipStream_t)stream));
}

}  // extern "C"
