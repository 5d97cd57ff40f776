// The gated delta rule token by token (one scalar decay per token and head), from a pool of states
// advanced in place:
//   S' = alpha S,  p = S'^T k,  r = beta (v - p),  S = S' + k r^T,  o~ = S^T q = S'^T q + (q . k) r
// for T new tokens of each sequence (T = 1: a decode step; T > 1: drafted tokens, or a short prompt).
//
// The state is the whole cost: 2 * D_k * D_v * 4 bytes per (sequence, head) and call, whatever T is.  It
// is read once into registers, stays there over the T tokens, and is written once.  A CTA of 8 warps per
// (sequence, head): lane l of warp w owns the key rows w, w + 8, ... and four value columns, so that a
// warp reads whole rows; the sums over key rows are partial sums of 8 warps joined in shared memory, one
// barrier each (the buffers alternate, so the next token's sums need no second one).
// Sums are fp32 for fp32 inputs too (with fp64 ones, as the per-channel decode step has, four tokens of 33 sequences x 6
// heads of 96 x 72 take 20 us instead of 11, one token of 256 x 32 heads of 128 in fp32 224 us instead of 173).
// Measured (bf16, D = 128, 32 heads): 256 sequences 181 us, 6.0 TB/s (91% of a copy's rate; a plain in-place
// update of as many bytes takes 159 us); with three CTAs on an SM instead of two it spills 312 bytes a thread instead
// of 20 (233 us), with plain stores instead of streaming ones 218 us.  One sequence: 5 us, the call's own time.
// Every instance spills some (16 to 192 bytes).
#include "host_check.cuh"
#include "kda_internal.cuh"
#include "sm100_ptx.cuh"

namespace kda {

namespace {

constexpr int GD_NW = 8, GD_MAXD = 128;

struct GdArgs {
    int64_t slots_n;
    int T, H, Dk, Dv;
    const void *q, *k, *v, *z, *beta, *gate;
    const float *log_decay;
    float g_min, eps;
    float *state;
    const int32_t *slots;
    void *o;
    int32_t *status;
    size_t state_bytes, o_bytes;
    unsigned int *bounds;
};

// VEC: D_v is a multiple of 4 and the state 16-byte aligned; lane l owns columns 4l .. 4l + 3.  Otherwise the columns
// l, l + 32, l + 64, l + 96.  FULL: D_k = D_v = 128 besides, nothing to mask.
// RPW: rows per warp, D_k <= 8 RPW; the fewer, the more CTAs on an SM (4096 sequences x 16 heads of 16: 756 us with 16
// rows, 333 us with 4, 397 us with slots; of 64: 650 us with 8, 781 us with slots).  Lanes past D_v / 4 columns are idle.
template <typename T, bool VEC, bool FULL, int RPW>
__global__ void __launch_bounds__(256, RPW == 16 ? 2 : RPW == 8 ? 3 : 4) gdn_decode_kernel(const __grid_constant__ GdArgs p) {
    sm100::pdl_trigger();
    sm100::pdl_wait();
    __shared__ __align__(16) float s_q[2][GD_MAXD], s_k[2][GD_MAXD];
    __shared__ __align__(16) float s_red[2][2][GD_NW][GD_MAXD];
    const int Dk = FULL ? GD_MAXD : p.Dk, Dv = FULL ? GD_MAXD : p.Dv;
    const int tid = threadIdx.x, w = tid >> 5, l = tid & 31;
    const int64_t b = blockIdx.x / p.H;
    const int h = (int)(blockIdx.x - b * p.H);
    const int64_t slot = p.slots ? p.slots[b] : b;
    if (slot < 0) return;  // a padded row of the batch
    if (slot >= p.slots_n) {
        if (tid == 0 && p.status) *p.status = KDA_ERR_INVALID_ARG;
        return;
    }
    float *S = p.state + (slot * p.H + h) * (int64_t)Dk * Dv;
    auto row = [&](int i) { return w + GD_NW * i; };
    auto col = [&](int j) { return VEC ? 4 * l + j : l + 32 * j; };
    const int64_t tok0 = b * p.T * p.H + h;  // (token, head) index of token 0; p.H further for each token
    auto fetch = [&](int t) {                // this thread's element of token t's q (threads < 128) or k
        const int c = tid & 127;
        const T *src = (const T *)(tid < 128 ? p.q : p.k);
        return c < Dk ? load_elem(src, (tok0 + (int64_t)t * p.H) * Dk + c) : 0.f;
    };
    struct Token {  // what this thread needs of a token besides q and k
        T v[4], gate[4], beta, z;
        float log_decay;
    };
    auto token = [&](int t) {
        const int64_t th = tok0 + (int64_t)t * p.H;
        Token n;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = FULL || col(j) < Dv;
            n.v[j] = in ? ((const T *)p.v)[th * Dv + col(j)] : T(0.f);
            n.gate[j] = (in && p.gate) ? ((const T *)p.gate)[th * Dv + col(j)] : T(0.f);
        }
        n.beta = ((const T *)p.beta)[th];
        if (p.log_decay) n.log_decay = p.log_decay[th];
        else n.z = ((const T *)p.z)[th];
        return n;
    };
    float pre = fetch(0);  // ahead of the state: behind it they would wait for all of it (203 -> 183 us at 256 x 32)
    Token now = token(0);
    float s[RPW][4];
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
        const int c = row(i);
        if (VEC) {
            const float4 t = FULL || (c < Dk && 4 * l < Dv) ? __ldcs(reinterpret_cast<const float4 *>(S + c * Dv + 4 * l))
                                                            : make_float4(0.f, 0.f, 0.f, 0.f);
            s[i][0] = t.x; s[i][1] = t.y; s[i][2] = t.z; s[i][3] = t.w;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = (c < Dk && col(j) < Dv) ? S[c * Dv + col(j)] : 0.f;
        }
    }
    // A slot that an earlier sequence of the batch has: two CTAs would race on its state.  Every CTA looks through the slots
    // before its own, B^2 H / 2 reads of 4 bytes from the caches in all: 1024 sequences x 32 heads of 128 take 719 us instead
    // of 674, 16384 x 4 of 16 472 instead of 333, 65536 x 1 of 16 838 instead of 333.
    if (p.slots) {
        bool twice = false;
        for (int64_t e = tid; e < b; e += 256) twice |= p.slots[e] == (int32_t)slot;
        if (__syncthreads_or(twice)) {
            if (tid == 0 && p.status) *p.status = KDA_ERR_INVALID_ARG;
            return;
        }
    }
    for (int t = 0; t < p.T; ++t) {
        const int64_t th = tok0 + (int64_t)t * p.H;
        const int buf = t & 1;
        if (RPW == 16 || (tid & 127) < GD_NW * RPW)  // a warp's rows side by side
            (tid < 128 ? s_q : s_k)[buf][RPW * (tid & 7) + ((tid & 127) >> 3)] = pre;
        float v[4], gt[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = (float)now.v[j];
            gt[j] = (float)now.gate[j];
        }
        const float bt = (float)now.beta;
        const float a = expf(p.log_decay ? clamp_log_decay(now.log_decay, p.g_min) : log_alpha_of((float)now.z, p.g_min));
        if (t + 1 < p.T) pre = fetch(t + 1);
        __syncthreads();  // q and k of token t
        // q . k first, in every warp, although one needs it: behind the products it costs T = 1 11% (203 us, so 181)
        float qk = 0.f, pp[4] = {0.f, 0.f, 0.f, 0.f}, qs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < RPW / 4; ++j) qk = fmaf(s_q[buf][l + 32 * j], s_k[buf][l + 32 * j], qk);
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) qk += __shfl_xor_sync(0xffffffffu, qk, m);
#pragma unroll
        for (int ii = 0; ii < RPW; ii += 4) {
            const float4 k4 = *reinterpret_cast<const float4 *>(&s_k[buf][RPW * w + ii]);
            const float4 q4 = *reinterpret_cast<const float4 *>(&s_q[buf][RPW * w + ii]);
            const float kc[4] = {k4.x, k4.y, k4.z, k4.w}, qc[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    s[ii + i][j] *= a;
                    pp[j] = fmaf(kc[i], s[ii + i][j], pp[j]);
                    qs[j] = fmaf(qc[i], s[ii + i][j], qs[j]);
                }
        }
        *reinterpret_cast<float4 *>(&s_red[buf][0][w][4 * l]) = make_float4(pp[0], pp[1], pp[2], pp[3]);
        *reinterpret_cast<float4 *>(&s_red[buf][1][w][4 * l]) = make_float4(qs[0], qs[1], qs[2], qs[3]);
        __syncthreads();  // the partial sums
        float r[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int u = 0; u < GD_NW; ++u) {
            const float4 x = *reinterpret_cast<const float4 *>(&s_red[buf][0][u][4 * l]);
            r[0] += x.x; r[1] += x.y; r[2] += x.z; r[3] += x.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = bt * (v[j] - r[j]);
#pragma unroll
        for (int ii = 0; ii < RPW; ii += 4) {
            const float4 k4 = *reinterpret_cast<const float4 *>(&s_k[buf][RPW * w + ii]);
            const float kc[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) s[ii + i][j] = fmaf(kc[i], r[j], s[ii + i][j]);
        }
        if (w == (t & 7)) {  // one warp has the outputs of this token, another those of the next
            float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int u = 0; u < GD_NW; ++u) {
                const float4 y = *reinterpret_cast<const float4 *>(&s_red[buf][1][u][4 * l]);
                o[0] += y.x; o[1] += y.y; o[2] += y.z; o[3] += y.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = fmaf(qk, r[j], o[j]);
            if (p.gate) {
                float ss = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) ss = (FULL || col(j) < Dv) ? fmaf(o[j], o[j], ss) : ss;
#pragma unroll
                for (int m = 16; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
                const float inv = 1.0f / sqrtf(ss / (float)Dv + p.eps);
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] *= inv * sigmoid_precise(gt[j]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if ((FULL || col(j) < Dv) &&
                    in_bounds((const T *)p.o + th * Dv + col(j), sizeof(T), p.o, p.o_bytes, p.bounds))
                    store_elem((T *)p.o, th * Dv + col(j), o[j]);
        }
        if (t + 1 < p.T) now = token(t + 1);  // here, not above: its registers beside the sums cost 8% of eight tokens
    }
    if (!in_bounds(S, (size_t)Dk * Dv * 4, p.state, p.state_bytes, p.bounds)) return;
#pragma unroll
    for (int i = 0; i < RPW; ++i) {
        const int c = row(i);
        if (VEC) {
            if (FULL || (c < Dk && 4 * l < Dv))
                __stcs(reinterpret_cast<float4 *>(S + c * Dv + 4 * l), make_float4(s[i][0], s[i][1], s[i][2], s[i][3]));
        } else if (c < Dk) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (col(j) < Dv) S[c * Dv + col(j)] = s[i][j];
        }
    }
}

template <typename T>
cudaError_t gd_launch(const kda_gdn_decode_args &a, const GdArgs &p, cudaStream_t st) {
    const dim3 grid((unsigned)(a.B * a.H));
    const bool vec = a.D_v % 4 == 0 && aligned_to(a.state, 16);
    auto go = [&](auto kernel) { return launch_pdl(kernel, grid, dim3(256), 0, st, p); };
    if (vec && a.D_k == GD_MAXD && a.D_v == GD_MAXD) return go(gdn_decode_kernel<T, true, true, 16>);
    if (a.D_k <= 4 * GD_NW) return go(vec ? gdn_decode_kernel<T, true, false, 4> : gdn_decode_kernel<T, false, false, 4>);
    if (a.D_k <= 8 * GD_NW) return go(vec ? gdn_decode_kernel<T, true, false, 8> : gdn_decode_kernel<T, false, false, 8>);
    return go(vec ? gdn_decode_kernel<T, true, false, 16> : gdn_decode_kernel<T, false, false, 16>);
}

}  // namespace

}  // namespace kda

using namespace kda;

extern "C" kda_status_t kda_gdn_decode_step(const kda_gdn_decode_args *a) {
    clear_error();
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    KDA_TRY(check_dtype(a->dtype));
    KDA_TRY(check_gmin(a->g_min));
    if (a->B < 0 || a->T < 0 || a->H < 1 || a->D_k < 1 || a->D_v < 1 || a->num_slots < 0)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes B=%lld T=%d H=%d D_k=%d D_v=%d num_slots=%lld", (long long)a->B, a->T,
                    a->H, a->D_k, a->D_v, (long long)a->num_slots);
    if (a->D_k > GD_MAXD || a->D_v > GD_MAXD) return fail(KDA_ERR_UNSUPPORTED, "D_k and D_v must be <= 128");
    if (a->B > 0x7fffffffLL / a->H) return fail(KDA_ERR_UNSUPPORTED, "B*H exceeds 2^31 - 1");
    if (a->num_slots > ((int64_t)1 << 40) / a->H) return fail(KDA_ERR_UNSUPPORTED, "num_slots too large");
    if (a->B == 0 || a->T == 0) return KDA_OK;
    if (!a->slots && a->num_slots < a->B)
        return fail(KDA_ERR_INVALID_ARG, "without slots the pool needs a state for each of the %lld sequences (has %lld)",
                    (long long)a->B, (long long)a->num_slots);
    if (a->gate_logits && !(isfinite(a->eps) && a->eps >= 0.0f))
        return fail(KDA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    const size_t es = esize(a->dtype), n = (size_t)a->B * a->T * a->H;
    KDA_REQ_PTR(a->q, "q", es);
    KDA_REQ_PTR(a->k, "k", es);
    KDA_REQ_PTR(a->v, "v", es);
    KDA_REQ_PTR(a->beta, "beta", es);
    KDA_REQ_PTR(a->o, "o", es);
    if (!a->log_decay) KDA_REQ_PTR(a->z, "z (or log_decay)", es);
    KDA_OPT_PTR(a->log_decay, "log_decay", 4);
    KDA_OPT_PTR(a->gate_logits, "gate_logits", es);
    KDA_OPT_PTR(a->slots, "slots", 4);
    KDA_OPT_PTR(a->dev_status, "dev_status", 4);
    if (a->num_slots > 0) KDA_REQ_PTR(a->state, "state", 4);
    const size_t ns = (size_t)a->num_slots * a->H * a->D_k * a->D_v * 4, nv = n * a->D_v * es;
    const Buf ins[] = {{a->q, n * a->D_k * es, "q"}, {a->k, n * a->D_k * es, "k"}, {a->v, nv, "v"},
                       {a->log_decay ? nullptr : a->z, n * es, "z"}, {a->log_decay, n * 4, "log_decay"},
                       {a->beta, n * es, "beta"}, {a->gate_logits, nv, "gate_logits"},
                       {a->slots, (size_t)a->B * 4, "slots"}, {a->dev_status, 4, "dev_status"}};
    const int nin = (int)(sizeof(ins) / sizeof(ins[0]));
    KDA_TRY(check_no_overlap(Buf{a->state, ns, "state"}, ins, nin));
    KDA_TRY(check_no_overlap(Buf{a->o, nv, "o"}, ins, nin));
    if (overlap(a->o, nv, a->state, ns)) return fail(KDA_ERR_INVALID_ARG, "o overlaps state");
    const GdArgs p = {a->num_slots, a->T,  a->H,    a->D_k,         a->D_v,       a->q,     a->k,
                      a->v,         a->z,  a->beta, a->gate_logits, a->log_decay, a->g_min, a->eps,
                      a->state,     a->slots, a->o, a->dev_status,  checked_size(ns), checked_size(nv),
                      device_bounds_counter()};
    cudaStream_t st = (cudaStream_t)a->stream;
    const cudaError_t e = a->dtype == KDA_F32 ? gd_launch<float>(*a, p, st) : gd_launch<__nv_bfloat16>(*a, p, st);
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "gdn_decode_kernel: %s", cudaGetErrorString(e));
    return check_launch("gdn_decode_kernel");
}
