// q4_checks.h -- the host checks that the experts' and the adapters' entry
// points share.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "q4.h"

namespace q4 {
namespace checks {

// (A null pointer counts as aligned.)
inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Range {
    uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void *p, uint64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return {a, p ? a + (uintptr_t)bytes : a};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

// Whether any of the outputs overlaps an input or another output.
inline bool clash(const Range *out, int nout, const Range *in, int nin) {
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j)
            if (overlap(out[i], in[j])) return true;
        for (int j = i + 1; j < nout; ++j)
            if (overlap(out[i], out[j])) return true;
    }
    return false;
}

inline bool k_ok(int64_t K) { return K > 0 && K % 64 == 0 && K <= Q4_MAX_K; }
inline bool type_ok(int t) { return t == Q4_OUT_F32 || t == Q4_OUT_BF16; }
inline uint64_t elt(int t) { return t == Q4_OUT_BF16 ? 2 : 4; }

inline int launch_status(hipError_t e) { return e == hipSuccess ? Q4_OK : Q4_ERR_DEVICE; }

}  // namespace checks
}  // namespace q4
