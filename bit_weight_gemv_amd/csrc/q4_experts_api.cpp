// q4_experts_api.cpp -- the exported entry points of q4_experts.h: argument
// checks on the host, then the launches on the caller's stream.
#include "q4_experts.h"

#include "q4_checks.h"
#include "q4_ragged.h"

using namespace q4::checks;

namespace {

bool route_shape_ok(int64_t T, int64_t E, int64_t k) {
    return T >= 0 && E >= 1 && E <= Q4_MAX_EXPERTS && k >= 1 && k <= Q4_MAX_TOPK && k <= E && T <= Q4_MAX_SLOTS / k;
}

bool grouped_shape_ok(int64_t E, int64_t M, int64_t K, int64_t T, int64_t R, bool up) {
    return E >= 1 && E <= Q4_MAX_EXPERTS && M >= 0 && M <= Q4_MAX_ROWS && k_ok(K) && T >= 0 && T <= Q4_MAX_SLOTS &&
           R >= 0 && R <= Q4_MAX_SLOTS && q4::ragged_fits(E, M, K, T, R, up);
}

}  // namespace

extern "C" {

size_t q4_route_topk_ws_bytes(int64_t T, int64_t E, int64_t k) {
    return route_shape_ok(T, E, k) ? q4::route_ws_bytes(T, E, k) : 0;
}

int q4_route_topk(const void *logits, int logits_type, int64_t T, int64_t E, int64_t k, int mode, int32_t *experts,
                  float *weights, int32_t *offsets, int32_t *rows, int32_t *pos, void *workspace,
                  size_t workspace_bytes, void *stream) {
    if (!type_ok(logits_type) || (mode != Q4_ROUTE_TOPK && mode != Q4_ROUTE_ALL) || !route_shape_ok(T, E, k))
        return Q4_ERR_SHAPE;
    if (!offsets || (T > 0 && (!logits || !experts || !weights || !rows || !pos))) return Q4_ERR_NULL;
    if (!aligned(logits, elt(logits_type)) || !aligned(experts, 4) || !aligned(weights, 4) || !aligned(offsets, 4) ||
        !aligned(rows, 4) || !aligned(pos, 4))
        return Q4_ERR_ALIGN;
    const uint64_t slots = (uint64_t)T * k * 4;
    Range out[6] = {range_of(experts, slots), range_of(weights, slots), range_of(offsets, (uint64_t)(E + 1) * 4),
                    range_of(rows, slots), range_of(pos, slots), {0, 0}};
    const Range in[1] = {range_of(logits, (uint64_t)T * E * elt(logits_type))};
    if (clash(out, 5, in, 1)) return Q4_ERR_OVERLAP;
    const size_t need = q4::route_ws_bytes(T, E, k);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return Q4_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return Q4_ERR_ALIGN;
        out[5] = range_of(workspace, need);
        if (clash(out, 6, in, 1)) return Q4_ERR_OVERLAP;
    }
    return launch_status(q4::launch_route(logits, logits_type == Q4_OUT_BF16, T, E, k, mode == Q4_ROUTE_ALL, experts,
                                          weights, offsets, rows, pos, workspace, (hipStream_t)stream));
}

size_t q4_gemm_grouped_ws_bytes(int64_t E, int64_t M, int64_t K, int64_t T, int64_t R, int has_up) {
    if (!grouped_shape_ok(E, M, K, T, R, has_up != 0) || M == 0 || R == 0) return 0;
    return q4::ragged_ws_bytes(E, M, K, T, R, has_up != 0, 0);
}

int q4_gemm_grouped(const uint8_t *codes, const uint16_t *scales, const uint8_t *up_codes, const uint16_t *up_scales,
                    int64_t E, int64_t M, int64_t K, const uint16_t *X, int64_t T, const int32_t *offsets,
                    const int32_t *rows, int64_t R, int out_type, void *Y, void *workspace, size_t workspace_bytes,
                    void *stream) {
    const bool up = up_codes != nullptr;
    if (!type_ok(out_type) || !grouped_shape_ok(E, M, K, T, R, up)) return Q4_ERR_SHAPE;
    if (M == 0 || R == 0) return Q4_OK;
    if (!codes || !scales || (up && !up_scales) || (T > 0 && !X) || !offsets || !Y) return Q4_ERR_NULL;
    if (!aligned(codes, 16) || !aligned(scales, 2) || !aligned(up_codes, 16) || !aligned(up_scales, 2) ||
        !aligned(X, 16) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(Y, 16))
        return Q4_ERR_ALIGN;
    const uint64_t cb = (uint64_t)E * M * (K / 2), sb = (uint64_t)E * M * (K / 64) * 2;
    const Range in[7] = {range_of(codes, cb),
                         range_of(scales, sb),
                         range_of(up_codes, cb),
                         range_of(up ? up_scales : nullptr, sb),
                         range_of(X, (uint64_t)T * K * 2),
                         range_of(offsets, (uint64_t)(E + 1) * 4),
                         range_of(rows, (uint64_t)R * 4)};
    Range out[2] = {range_of(Y, (uint64_t)R * M * elt(out_type)), {0, 0}};
    if (clash(out, 1, in, 7)) return Q4_ERR_OVERLAP;
    const size_t need = q4::ragged_ws_bytes(E, M, K, T, R, up, 0);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return Q4_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return Q4_ERR_ALIGN;
        out[1] = range_of(workspace, need);
        if (clash(out, 2, in, 7)) return Q4_ERR_OVERLAP;
    }
    q4::RaggedProduct p = {};
    p.codes = codes;
    p.up_codes = up_codes;
    p.scales = scales;
    p.up_scales = up ? up_scales : nullptr;
    p.E = E;
    p.M = M;
    p.K = K;
    p.X = X;
    p.T = T;
    p.offsets = offsets;
    p.rows = rows;
    p.R = R;
    p.bf16 = out_type == Q4_OUT_BF16;
    p.Y = Y;
    return launch_status(q4::launch_ragged(p, workspace, (hipStream_t)stream));
}

int q4_moe_combine(const void *Y, int y_type, int64_t R, int64_t M, const float *weights, const int32_t *pos,
                   int64_t T, int64_t k, int out_type, void *out, void *stream) {
    if (!type_ok(y_type) || !type_ok(out_type) || R < 0 || R > Q4_MAX_SLOTS || M < 0 || M > Q4_MAX_ROWS || T < 0 ||
        T > Q4_MAX_SLOTS || k < 1 || k > Q4_MAX_TOPK || !q4::combine_fits(M, T))
        return Q4_ERR_SHAPE;
    if (T == 0 || M == 0) return Q4_OK;
    if ((R > 0 && !Y) || !weights || !pos || !out) return Q4_ERR_NULL;
    if (!aligned(Y, 16) || !aligned(weights, 4) || !aligned(pos, 4) || !aligned(out, 16)) return Q4_ERR_ALIGN;
    const Range o = range_of(out, (uint64_t)T * M * elt(out_type));
    const Range in[3] = {range_of(Y, (uint64_t)R * M * elt(y_type)), range_of(weights, (uint64_t)T * k * 4),
                         range_of(pos, (uint64_t)T * k * 4)};
    if (clash(&o, 1, in, 3)) return Q4_ERR_OVERLAP;
    return launch_status(q4::launch_combine(Y, y_type == Q4_OUT_BF16, R, M, weights, pos, T, k,
                                            out_type == Q4_OUT_BF16, out, (hipStream_t)stream));
}

}  // extern "C"
