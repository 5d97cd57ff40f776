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

// The pointer, workspace and overlap checks the backward entry points share (need: the workspace bytes;
// scalar_decay: z, log_decay and dz hold one value per token and head).
inline kda_status_t bwd_check_buffers(const kda_recurrent_bwd_args *a, size_t need, bool scalar_decay = false) {
    const size_t es = esize(a->dtype);
    const size_t nk = (size_t)a->B * a->S * a->H * a->D_k, nv = (size_t)a->B * a->S * a->H * a->D_v;
    const size_t nb = (size_t)a->B * a->S * a->H, ns = (size_t)a->B * a->H * a->D_k * a->D_v * 4;
    const size_t nz = scalar_decay ? nb : nk;
    if (a->S > 0) {
        KDA_REQ_PTR(a->q, "q", es);
        KDA_REQ_PTR(a->k, "k", es);
        KDA_REQ_PTR(a->v, "v", es);
        KDA_REQ_PTR(a->beta, "beta", es);
        KDA_REQ_PTR(a->d_o, "d_o", es);
        if (!a->log_decay) KDA_REQ_PTR(a->z, "z (or log_decay)", es);
        KDA_OPT_PTR(a->log_decay, "log_decay", 4);
        KDA_REQ_PTR(a->dq, "dq", 4);
        KDA_REQ_PTR(a->dk, "dk", 4);
        KDA_REQ_PTR(a->dv, "dv", 4);
        KDA_REQ_PTR(a->dbeta, "dbeta", 4);
        KDA_REQ_PTR(a->dz, "dz", 4);
    }
    KDA_OPT_PTR(a->initial_state, "initial_state", 4);
    KDA_OPT_PTR(a->d_final_state, "d_final_state", 4);
    KDA_OPT_PTR(a->d_initial_state, "d_initial_state", 4);
    KDA_OPT_PTR(a->workspace, "workspace", 256);
    if (a->S > 0 && need > 0 && (!a->workspace || a->workspace_bytes < need))
        return fail(KDA_ERR_WORKSPACE, "workspace needs %zu bytes (got %zu)", need,
                    a->workspace ? a->workspace_bytes : (size_t)0);
    const Buf ins[] = {
        {a->S ? a->q : nullptr, nk * es, "q"}, {a->S ? a->k : nullptr, nk * es, "k"},
        {a->S ? a->v : nullptr, nv * es, "v"}, {a->S && !a->log_decay ? a->z : nullptr, nz * es, "z"},
        {a->S ? a->log_decay : nullptr, nz * 4, "log_decay"}, {a->S ? a->beta : nullptr, nb * es, "beta"},
        {a->S ? a->d_o : nullptr, nv * es, "d_o"}, {a->initial_state, ns, "initial_state"},
        {a->d_final_state, ns, "d_final_state"}, {a->S && need ? a->workspace : nullptr, need, "workspace"},
    };
    const int nin = (int)(sizeof(ins) / sizeof(ins[0]));
    const Buf outs[] = {{a->S ? a->dq : nullptr, nk * 4, "dq"}, {a->S ? a->dk : nullptr, nk * 4, "dk"},
                        {a->S ? a->dv : nullptr, nv * 4, "dv"}, {a->S ? a->dbeta : nullptr, nb * 4, "dbeta"},
                        {a->S ? a->dz : nullptr, nz * 4, "dz"}, {a->d_initial_state, ns, "d_initial_state"}};
    for (const Buf &o : outs) {
        if (!o.p) continue;
        KDA_TRY(check_no_overlap(o, ins, nin));
        for (const Buf &o2 : outs)
            if (&o2 != &o && o2.p && overlap(o.p, o.n, o2.p, o2.n))
                return fail(KDA_ERR_INVALID_ARG, "outputs %s and %s overlap", o.name, o2.name);
    }
    return KDA_OK;
}

}  // namespace kda
