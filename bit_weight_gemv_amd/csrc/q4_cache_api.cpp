// q4_cache_api.cpp -- the exported entry points of q4_cache.h: argument
// checks on the host, then the launches on the caller's stream.
#include "q4_cache.h"

#include <math.h>

#include "q4_cache_internal.h"
#include "q4_checks.h"

using namespace q4::checks;

namespace {

constexpr int64_t kMost = Q4_CACHE_MAX_TOKENS;
constexpr int64_t kMostKeys = Q4_CACHE_MAX_KEYS;
constexpr int64_t kMostRows = Q4_CACHE_MAX_ROWS;

bool d_ok(int64_t D) { return D > 0 && D % 64 == 0 && D <= Q4_CACHE_MAX_D; }

bool cache_shape_ok(const q4_cache &c) {
    return d_ok(c.D) && c.heads >= 1 && c.heads <= Q4_CACHE_MAX_HEADS && c.page >= Q4_CACHE_MIN_PAGE &&
           c.page <= Q4_CACHE_MAX_PAGE && (c.page & (c.page - 1)) == 0 && c.pages >= 0 &&
           c.pages <= INT32_MAX / c.page;
}

struct Planes {
    Range r[6];
    bool null, misaligned;
};

// The cache's six planes: codes, scales and zeros of keys and of values.
Planes planes_of(const q4_cache &c) {
    const uint64_t rows = (uint64_t)c.pages * c.heads * c.page;
    const void *p[6] = {c.k_codes, c.k_scales, c.k_zeros, c.v_codes, c.v_scales, c.v_zeros};
    Planes out = {};
    for (int i = 0; i < 6; ++i) {
        const bool codes = i % 3 == 0;
        out.null = out.null || (rows > 0 && !p[i]);
        out.misaligned = out.misaligned || !aligned(p[i], 16);
        out.r[i] = range_of(p[i], rows * (codes ? c.D / 2 : c.D / 64 * 2));
    }
    return out;
}

// Rows of `width` elements, `stride` apart.
bool stride_ok(int64_t stride, int64_t width, uint64_t size) {
    return stride >= width && stride <= (int64_t)1 << 32 && (uint64_t)stride * size % 16 == 0;
}
Range strided(const void *p, int64_t T, int64_t stride, int64_t width, uint64_t size) {
    return range_of(p, ((uint64_t)(T - 1) * stride + width) * size);
}

bool attend_shape_ok(int64_t T, int64_t q_heads, int64_t heads, int64_t D, int64_t B, int64_t max_q) {
    return T >= 0 && T <= kMost && heads >= 1 && heads <= Q4_CACHE_MAX_HEADS && q_heads >= 1 &&
           q_heads <= Q4_CACHE_MAX_HEADS && q_heads % heads == 0 && T * q_heads <= kMostRows && d_ok(D) && B >= 0 &&
           B <= kMost && B * heads <= kMost && max_q >= 1 && max_q <= kMost;
}

}  // namespace

extern "C" {

int q4_cache_append(const q4_cache *cache, const void *k, const void *v, int in_type, int64_t T, int64_t k_stride,
                    int64_t v_stride, const int32_t *slots, const int32_t *positions, const float *inv_freq,
                    int64_t rot, int interleaved, float amplitude, const void *q, int64_t q_heads, int64_t q_stride,
                    uint16_t *q_out, void *stream) {
    if (!cache) return Q4_ERR_NULL;
    const q4_cache &c = *cache;
    if (!cache_shape_ok(c) || !type_ok(in_type) || T < 0 || T > kMost || rot < 0 || rot > c.D || rot % 16 != 0)
        return Q4_ERR_SHAPE;
    const uint64_t e = elt(in_type);
    const int64_t width = c.heads * c.D;
    if (T > 0 && (!stride_ok(k_stride, width, e) || !stride_ok(v_stride, width, e))) return Q4_ERR_SHAPE;
    if (q && (q_heads < 1 || q_heads > Q4_CACHE_MAX_HEADS || (T > 0 && !stride_ok(q_stride, q_heads * c.D, e))))
        return Q4_ERR_SHAPE;
    if (T == 0) return Q4_OK;
    const Planes planes = planes_of(c);
    if (planes.null || !k || !v || !slots || (rot > 0 && (!positions || !inv_freq)) || (q && !q_out))
        return Q4_ERR_NULL;
    if (planes.misaligned || !aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 4) || !aligned(positions, 4) ||
        !aligned(inv_freq, 4) || !aligned(q, 16) || (q && !aligned(q_out, 16)))
        return Q4_ERR_ALIGN;
    Range out[7];
    for (int i = 0; i < 6; ++i) out[i] = planes.r[i];
    out[6] = q ? range_of(q_out, (uint64_t)T * q_heads * c.D * 2) : Range{0, 0};
    const Range in[6] = {strided(k, T, k_stride, width, e),
                         strided(v, T, v_stride, width, e),
                         q ? strided(q, T, q_stride, q_heads * c.D, e) : Range{0, 0},
                         range_of(slots, (uint64_t)T * 4),
                         rot > 0 ? range_of(positions, (uint64_t)T * 4) : Range{0, 0},
                         rot > 0 ? range_of(inv_freq, (uint64_t)rot * 2) : Range{0, 0}};
    if (clash(out, 7, in, 6)) return Q4_ERR_OVERLAP;
    q4::CacheAppend a = {};
    a.cache = c;
    a.k = k;
    a.v = v;
    a.q = q;
    a.bf16 = in_type == Q4_OUT_BF16;
    a.T = T;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.q_stride = q ? q_stride : 0;
    a.q_heads = q ? q_heads : 0;
    a.slots = slots;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.rot = rot;
    a.interleaved = interleaved != 0;
    a.amplitude = amplitude;
    a.q_out = q_out;
    return launch_status(q4::launch_cache_append(a, (hipStream_t)stream));
}

int q4_cache_read(const q4_cache *cache, const int32_t *slots, int64_t n, int out_type, void *k_out, void *v_out,
                  void *stream) {
    if (!cache) return Q4_ERR_NULL;
    const q4_cache &c = *cache;
    if (!cache_shape_ok(c) || !type_ok(out_type) || n < 0 || n > kMost) return Q4_ERR_SHAPE;
    if (n == 0) return Q4_OK;
    const Planes planes = planes_of(c);
    if (planes.null || !slots || (!k_out && !v_out)) return Q4_ERR_NULL;
    if (planes.misaligned || !aligned(slots, 4) || !aligned(k_out, 16) || !aligned(v_out, 16)) return Q4_ERR_ALIGN;
    const uint64_t bytes = (uint64_t)n * c.heads * c.D * elt(out_type);
    const Range out[2] = {range_of(k_out, bytes), range_of(v_out, bytes)};
    Range in[7];
    for (int i = 0; i < 6; ++i) in[i] = planes.r[i];
    in[6] = range_of(slots, (uint64_t)n * 4);
    if (clash(out, 2, in, 7)) return Q4_ERR_OVERLAP;
    return launch_status(
        q4::launch_cache_read(c, slots, n, out_type == Q4_OUT_BF16, k_out, v_out, (hipStream_t)stream));
}

size_t q4_cache_attend_ws_bytes(int64_t T, int64_t q_heads, int64_t heads, int64_t D, int64_t B, int64_t max_q) {
    if (!attend_shape_ok(T, q_heads, heads, D, B, max_q) || T == 0 || B == 0) return 0;
    return q4::attend_ws_bytes(T, q_heads, heads, D, B, max_q);
}

int q4_cache_attend(const uint16_t *q, int64_t T, int64_t q_heads, int64_t q_stride, const q4_cache *cache,
                    const int32_t *table, int64_t B, int64_t table_pages, const int32_t *lens,
                    const int32_t *q_offsets, int64_t max_q, int causal, int64_t window, float scale, int out_type,
                    void *out, float *lse, void *workspace, size_t workspace_bytes, void *stream) {
    if (!cache) return Q4_ERR_NULL;
    const q4_cache &c = *cache;
    if (!cache_shape_ok(c) || !attend_shape_ok(T, q_heads, c.heads, c.D, B, max_q) || !type_ok(out_type) ||
        table_pages < 0 || table_pages > kMostKeys / c.page || window < 0 || window > INT32_MAX ||
        (!causal && window != 0) || !isfinite(scale) || !(scale > 0))
        return Q4_ERR_SHAPE;
    if (!q_offsets && (T != B || max_q != 1)) return Q4_ERR_SHAPE;
    if (T > 0 && !stride_ok(q_stride, q_heads * c.D, 2)) return Q4_ERR_SHAPE;
    if (T == 0 || B == 0) return Q4_OK;
    const Planes planes = planes_of(c);
    if (planes.null || !q || (table_pages > 0 && !table) || !lens || !out) return Q4_ERR_NULL;
    if (planes.misaligned || !aligned(q, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(q_offsets, 4) ||
        !aligned(out, 16) || !aligned(lse, 4))
        return Q4_ERR_ALIGN;
    Range in[10];
    for (int i = 0; i < 6; ++i) in[i] = planes.r[i];
    in[6] = strided(q, T, q_stride, q_heads * c.D, 2);
    in[7] = range_of(table, (uint64_t)B * table_pages * 4);
    in[8] = range_of(lens, (uint64_t)B * 4);
    in[9] = range_of(q_offsets, (uint64_t)(B + 1) * 4);
    Range o[3] = {range_of(out, (uint64_t)T * q_heads * c.D * elt(out_type)), range_of(lse, (uint64_t)T * q_heads * 4),
                  {0, 0}};
    if (clash(o, 2, in, 10)) return Q4_ERR_OVERLAP;
    const size_t need = q4::attend_ws_bytes(T, q_heads, c.heads, c.D, B, max_q);
    if (need > 0) {
        if (!workspace || workspace_bytes < need) return Q4_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return Q4_ERR_ALIGN;
        o[2] = range_of(workspace, need);
        if (clash(o, 3, in, 10)) return Q4_ERR_OVERLAP;
    }
    q4::CacheAttend a = {};
    a.q = q;
    a.T = T;
    a.q_heads = q_heads;
    a.q_stride = q_stride;
    a.cache = c;
    a.table = table;
    a.B = B;
    a.table_pages = table_pages;
    a.lens = lens;
    a.q_offsets = q_offsets;
    a.max_q = max_q < T ? max_q : T;
    a.causal = causal != 0;
    a.window = window;
    a.scale = scale;
    a.bf16 = out_type == Q4_OUT_BF16;
    a.out = out;
    a.lse = lse;
    return launch_status(q4::launch_cache_attend(a, workspace, (hipStream_t)stream));
}

}  // extern "C"
