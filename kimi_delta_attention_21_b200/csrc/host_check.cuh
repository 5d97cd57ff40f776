// Host-side argument checks shared by the entry-point files.
#pragma once

#include <math.h>

#include "kda_internal.cuh"

namespace kda {

inline bool aligned_to(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline size_t esize(kda_dtype_t dt) { return dt == KDA_F32 ? 4 : 2; }

inline bool overlap(const void *a, size_t na, const void *b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}

struct Buf {
    const void *p;
    size_t n;
    const char *name;
};

// Checks that `out` overlaps none of `ins` (except an input listed as `allowed_equal`
// that starts at the same address with the same size).
inline kda_status_t check_no_overlap(const Buf &out, const Buf *ins, int nin,
                                     const void *allowed_equal = nullptr) {
    for (int i = 0; i < nin; ++i) {
        if (!ins[i].p) continue;
        if (allowed_equal && ins[i].p == allowed_equal && out.p == allowed_equal && ins[i].n == out.n)
            continue;
        if (overlap(out.p, out.n, ins[i].p, ins[i].n))
            return fail(KDA_ERR_INVALID_ARG, "output %s overlaps input %s", out.name, ins[i].name);
    }
    return KDA_OK;
}

inline kda_status_t check_dtype(kda_dtype_t dt) {
    if (dt != KDA_F32 && dt != KDA_BF16) return fail(KDA_ERR_UNSUPPORTED, "dtype %d not supported", (int)dt);
    return KDA_OK;
}

inline kda_status_t check_gmin(float g_min) {
    if (!(isfinite(g_min) && g_min < 0.0f))
        return fail(KDA_ERR_INVALID_ARG, "g_min must be a finite negative number (got %g)", (double)g_min);
    return KDA_OK;
}

#define KDA_TRY(expr)                      \
    do {                                   \
        kda_status_t s_ = (expr);          \
        if (s_ != KDA_OK) return s_;       \
    } while (0)

// Pointers must be non-NULL (REQ) and aligned to their element size `al`.
#define KDA_REQ_PTR(p, name, al)                                                               \
    do {                                                                                       \
        if (!(p)) return fail(KDA_ERR_INVALID_ARG, "%s is NULL", name);                        \
        if (!aligned_to(p, al)) return fail(KDA_ERR_INVALID_ARG, "%s is not %d-byte aligned", name, (int)(al)); \
    } while (0)

#define KDA_OPT_PTR(p, name, al)                                                               \
    do {                                                                                       \
        if ((p) && !aligned_to(p, al))                                                         \
            return fail(KDA_ERR_INVALID_ARG, "%s is not %d-byte aligned", name, (int)(al));     \
    } while (0)

}  // namespace kda
