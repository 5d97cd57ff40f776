// Norms of queries and keys for each head with the rotation by position in the same pass, and their
// gradients.
//
// Forward, per row x of D channels:  r = (sum x^2 * s + eps)^{-1/2}  (s = 1: L2, s = 1/D: RMS),
// y = r x w, and the first R channels turned in pairs by the angle pos * f_j:
//   (a, b) -> (a cos - b sin, a sin + b cos).
// Backward:  g = the turn back of dy,  dw = sum over rows of g x r,  h = g w,
//   dx = r (h - x r^2 s sum(h x)).
// r is recomputed from x, so the backward needs nothing kept from the forward.
//
// Both are bound by HBM: a row is read once and written once, every intermediate stays in registers.  Measured (bf16,
// heads of 128): forward, 4096 tokens x 32 heads, 12 us (10 at the copy rate); backward, 16384 tokens x 64 heads with
// fp32 gradients, 198 us (164).  What bounds the backward is not one thing: issue and DRAM are half busy, 128 registers leave
// 16 warps an SM, whose waits for loads lead the stalls; but more rows in flight were no faster (a shared-memory ring of any
// depth: 241 us), and the angles of a token cost as much as three rows (without rotation 187 us).  Heads of no whole vectors,
// or rotated halves of none, take the kernel of a warp per row: 4096 tokens x 32 heads of 80 with R = 40, 52 us (6.4), backward
// of 16384 x 64 such heads 712 us (102).
// A group of G lanes holds one row, 16 bytes of input per lane and register vector, so that a warp's
// loads are whole rows; the pairs of a half-split rotation are 16-byte vectors apart and meet by a
// shuffle.  A group takes `hc` heads of one token in turn: the token's cosines and sines are computed
// once for all of them.  pos * f is an fp64 product, reduced to a fraction of a turn in fp64 before the fp32
// sine: the roundings of pos * f, of 1 / 2 pi and of their product are 3 * 2^-53 of the angle (7e-7 radians at
// 2^31), the fraction's in fp32 2^-26 of a turn.
#include "host_check.cuh"
#include "kda_internal.cuh"
#include "sm100_ptx.cuh"

namespace kda {

namespace {

constexpr int QN_NT = 256;     // threads per CTA
constexpr int QN_MAXD = 256;   // channels per head

enum { ROT_NONE = 0, ROT_HALF = 1, ROT_INTERLEAVED = 2 };

struct QnSide {       // queries, or keys
    const void *x;    // rows of H heads; (b, s) at b * sb + s * ss elements
    int64_t sb, ss;
    int H, hc, chunks;  // hc heads per item, chunks items per token
    const float *w;
    void *y;          // forward: out; backward: dx
    const void *dy;
    float *dw;
    size_t y_bytes;
};

struct QnArgs {
    QnSide side[2];
    int64_t tokens, S;
    int D, R;
    float share, eps;
    const int64_t *pos;
    const float *inv;
    float *partial;   // [gridDim.x][2][D] weight gradients of each CTA
    size_t partial_bytes, dw_bytes;
    unsigned int *bounds;
};

// A store that the checked build tests (n bytes at `at`, into y or the partial sums).
template <typename V>
__device__ __forceinline__ void qn_put(const QnArgs &p, void *base, size_t bytes, V *at, const V &v) {
    if (in_bounds(at, sizeof(V), base, bytes, p.bounds)) *at = v;
}

// cos and sin of pos * f
__device__ __forceinline__ void qn_angle(int64_t pos, float f, float &c, float &s) {
    double t = (double)pos * (double)f * 0.15915494309189533577;  // turns
    t -= rint(t);
    sincospif(2.0f * (float)t, &s, &c);
}

// VEC consecutive gradient values of type GT
template <typename GT, int VEC>
__device__ __forceinline__ void qn_load_grad(const GT *p, float (&f)[VEC]) {
    constexpr int N = Vec16<GT>::N;
    static_assert(VEC % N == 0, "whole 16-byte vectors");
#pragma unroll
    for (int i = 0; i < VEC / N; ++i) {
        float t[N];
        Vec16<GT>::unpack(*reinterpret_cast<const uint4 *>(p + N * i), t);
#pragma unroll
        for (int e = 0; e < N; ++e) f[N * i + e] = t[e];
    }
}

template <int G>
__device__ __forceinline__ float qn_sum(float v) {
#pragma unroll
    for (int m = G / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// This lane's cosines and signed sines: out = own * cs + partner * sn.
template <int VEC, int G, int NV, int ROT>
__device__ __forceinline__ void qn_phases(const QnArgs &p, int64_t pos, int lane, float (&cs)[NV][VEC],
                                          float (&sn)[NV][VEC]) {
    const int half = p.R >> 1;
    if (ROT == ROT_HALF && NV == 1 && p.R == G * VEC) {  // lanes j and j + G / 2 have the same angles: each makes half
        const bool second = lane >= G / 2;               // of them (backward of 16384 tokens: 198 -> 195 us)
        const int j0 = (lane & (G / 2 - 1)) * VEC + (second ? VEC / 2 : 0);
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
            float c, s;
            qn_angle(pos, p.inv[j0 + e], c, s);
            const float oc = __shfl_xor_sync(0xffffffffu, c, G / 2), os = __shfl_xor_sync(0xffffffffu, s, G / 2);
            cs[0][e] = second ? oc : c;
            sn[0][e] = second ? os : -s;
            cs[0][e + VEC / 2] = second ? c : oc;
            sn[0][e + VEC / 2] = second ? s : -os;
        }
        return;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const int c = (lane + G * v) * VEC + e;
            if (ROT == ROT_INTERLEAVED && (e & 1)) {  // the pair's second channel has the first one's angle
                cs[v][e] = cs[v][e - 1];
                sn[v][e] = -sn[v][e - 1];
                continue;
            }
            cs[v][e] = 1.f;
            sn[v][e] = 0.f;
            if (c < p.R) {
                const bool second = ROT == ROT_HALF && c >= half;
                const int j = ROT == ROT_HALF ? (second ? c - half : c) : c >> 1;
                float s;
                qn_angle(pos, p.inv[j], cs[v][e], s);
                sn[v][e] = second ? s : -s;
            }
        }
}

// The partners of this lane's channels (half-split: the vector R/2 channels away); zero past R, where an infinite or NaN
// neighbour times a sine of zero would be NaN.
template <int VEC, int G, int NV, int ROT>
__device__ __forceinline__ void qn_partner(const QnArgs &p, int lane, const float (&y)[NV][VEC], float (&o)[NV][VEC]) {
    if (ROT == ROT_INTERLEAVED) {
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int e = 0; e < VEC; ++e) o[v][e] = (lane + G * v) * VEC + e < p.R ? y[v][e ^ 1] : 0.f;
        return;
    }
    const int d = (p.R >> 1) / VEC;
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int j = lane + G * v, other = j < d ? j + d : (j < 2 * d ? j - d : j);
        const int src = other & (G - 1);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            float t = __shfl_sync(0xffffffffu, y[0][e], src, G);
            if (NV == 2) {
                const float t1 = __shfl_sync(0xffffffffu, y[NV - 1][e], src, G);
                t = other >= G ? t1 : t;
            }
            o[v][e] = j < 2 * d ? t : 0.f;
        }
    }
}

// ---------------------------------------------------------------- forward
template <typename T, int G, int NV, int ROT>
__global__ void __launch_bounds__(QN_NT) qk_norm_kernel(const __grid_constant__ QnArgs p) {
    sm100::pdl_trigger();
    sm100::pdl_wait();
    constexpr int VEC = Vec16<T>::N, U = NV == 1 ? 4 : 2, PER = QN_NT / G;
    const QnSide &s = p.side[blockIdx.y];
    const int lane = threadIdx.x & (G - 1);
    const int64_t items = p.tokens * s.chunks;
    // every lane of a warp makes the same passes (the shuffles below are warp-wide)
    for (int64_t base = (int64_t)blockIdx.x * PER; base < items; base += (int64_t)gridDim.x * PER) {
        const int64_t it = base + threadIdx.x / G;
        const bool live = it < items;
        const int64_t tok = live ? it / s.chunks : 0;
        const int h0 = live ? (int)(it - tok * s.chunks) * s.hc : 0, h1 = live ? min(h0 + s.hc, s.H) : 0;
        const int64_t b = tok / p.S;
        const T *x = (const T *)s.x + b * s.sb + (tok - b * p.S) * s.ss;
        T *y = (T *)s.y + tok * s.H * p.D;
        float w[NV][VEC], cs[NV][VEC], sn[NV][VEC];
        bool in[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const int c = (lane + G * v) * VEC;
            in[v] = c < p.D;
#pragma unroll
            for (int e = 0; e < VEC; ++e) w[v][e] = (s.w && in[v]) ? s.w[c + e] : 1.f;
        }
        if (ROT != ROT_NONE) qn_phases<VEC, G, NV, ROT>(p, p.pos[tok], lane, cs, sn);
        for (int i = 0; i < s.hc; i += U) {
            uint4 raw[U][NV];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int v = 0; v < NV; ++v)
                    raw[u][v] = (in[v] && h0 + i + u < h1)
                                    ? __ldcs(reinterpret_cast<const uint4 *>(x + (int64_t)(h0 + i + u) * p.D +
                                                                             (lane + G * v) * VEC))
                                    : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[NV][VEC], o[NV][VEC];
                float ss = 0.f;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    Vec16<T>::unpack(raw[u][v], f[v]);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) ss = fmaf(f[v][e], f[v][e], ss);
                }
                const float r = rsqrtf(fmaf(qn_sum<G>(ss), p.share, p.eps));
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) f[v][e] *= r * w[v][e];
                if (ROT != ROT_NONE) {
                    qn_partner<VEC, G, NV, ROT>(p, lane, f, o);
#pragma unroll
                    for (int v = 0; v < NV; ++v)
#pragma unroll
                        for (int e = 0; e < VEC; ++e) f[v][e] = fmaf(o[v][e], sn[v][e], f[v][e] * cs[v][e]);
                }
                if (h0 + i + u < h1)
#pragma unroll
                    for (int v = 0; v < NV; ++v)
                        if (in[v])
                            qn_put(p, s.y, s.y_bytes,
                                   reinterpret_cast<uint4 *>(y + (int64_t)(h0 + i + u) * p.D + (lane + G * v) * VEC),
                                   Vec16<T>::pack(f[v]));
            }
        }
    }
}

// ---------------------------------------------------------------- backward
template <typename T, typename GT, int G, int NV, int ROT>
__global__ void __launch_bounds__(QN_NT) qk_norm_bwd_kernel(const __grid_constant__ QnArgs p) {
    sm100::pdl_trigger();
    sm100::pdl_wait();
    constexpr int VEC = Vec16<T>::N, U = NV == 1 ? 2 : 1, PER = QN_NT / G;
    __shared__ float s_dw[PER][G * NV * VEC];
    const QnSide &s = p.side[blockIdx.y];
    const int lane = threadIdx.x & (G - 1);
    const int64_t items = p.tokens * s.chunks;
    float w[NV][VEC], dw[NV][VEC];
    bool in[NV];
#pragma unroll
    for (int v = 0; v < NV; ++v) {
        const int c = (lane + G * v) * VEC;
        in[v] = c < p.D;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            w[v][e] = (s.w && in[v]) ? s.w[c + e] : 1.f;
            dw[v][e] = 0.f;
        }
    }
    for (int64_t base = (int64_t)blockIdx.x * PER; base < items; base += (int64_t)gridDim.x * PER) {
        const int64_t it = base + threadIdx.x / G;
        const bool live = it < items;
        const int64_t tok = live ? it / s.chunks : 0;
        const int h0 = live ? (int)(it - tok * s.chunks) * s.hc : 0, h1 = live ? min(h0 + s.hc, s.H) : 0;
        const int64_t b = tok / p.S;
        const T *x = (const T *)s.x + b * s.sb + (tok - b * p.S) * s.ss;
        const int64_t row = tok * s.H * p.D;
        float cs[NV][VEC], sn[NV][VEC];
        if (ROT != ROT_NONE) qn_phases<VEC, G, NV, ROT>(p, p.pos[tok], lane, cs, sn);
        for (int i = 0; i < s.hc; i += U) {
            uint4 raw[U][NV];
            float g[U][NV][VEC];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    const bool ok = in[v] && h0 + i + u < h1;
                    const int64_t at = (int64_t)(h0 + i + u) * p.D + (lane + G * v) * VEC;
                    raw[u][v] = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) g[u][v][e] = 0.f;
                    if (ok) {
                        raw[u][v] = __ldcs(reinterpret_cast<const uint4 *>(x + at));
                        qn_load_grad<GT, VEC>((const GT *)s.dy + row + at, g[u][v]);
                    }
                }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float f[NV][VEC], o[NV][VEC];
                if (ROT != ROT_NONE) {
                    qn_partner<VEC, G, NV, ROT>(p, lane, g[u], o);
#pragma unroll
                    for (int v = 0; v < NV; ++v)
#pragma unroll
                        for (int e = 0; e < VEC; ++e)
                            g[u][v][e] = fmaf(-o[v][e], sn[v][e], g[u][v][e] * cs[v][e]);
                }
                float ss = 0.f, hx = 0.f;
#pragma unroll
                for (int v = 0; v < NV; ++v) {
                    Vec16<T>::unpack(raw[u][v], f[v]);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        ss = fmaf(f[v][e], f[v][e], ss);
                        hx = fmaf(g[u][v][e] * w[v][e], f[v][e], hx);
                    }
                }
                const float r = rsqrtf(fmaf(qn_sum<G>(ss), p.share, p.eps));
                const float k = qn_sum<G>(hx) * r * r * p.share;
#pragma unroll
                for (int v = 0; v < NV; ++v)
#pragma unroll
                    for (int e = 0; e < VEC; ++e) {
                        // rows outside the tensor have x = 0: with eps = 0 their r is infinite, so they add nothing
                        if (h0 + i + u < h1) dw[v][e] = fmaf(g[u][v][e] * f[v][e], r, dw[v][e]);
                        f[v][e] = r * (g[u][v][e] * w[v][e] - f[v][e] * k);
                    }
                if (h0 + i + u < h1)
#pragma unroll
                    for (int v = 0; v < NV; ++v)
                        if (in[v])
                            qn_put(p, s.y, s.y_bytes,
                                   reinterpret_cast<uint4 *>((T *)s.y + row + (int64_t)(h0 + i + u) * p.D +
                                                             (lane + G * v) * VEC),
                                   Vec16<T>::pack(f[v]));
            }
        }
    }
    if (!s.dw) return;  // (the same for the whole CTA)
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int e = 0; e < VEC; ++e) s_dw[threadIdx.x / G][(lane + G * v) * VEC + e] = dw[v][e];
    __syncthreads();
    for (int c = threadIdx.x; c < p.D; c += QN_NT) {
        float t = 0.f;
        for (int i = 0; i < PER; ++i) t += s_dw[i][c];
        qn_put(p, p.partial, p.partial_bytes, p.partial + ((int64_t)blockIdx.x * 2 + blockIdx.y) * p.D + c, t);
    }
}

// The CTAs' weight gradients added in a fixed order (the same result on every run): 32 channels per CTA,
// 32 threads share a channel.
__global__ void __launch_bounds__(1024) qk_norm_dw_kernel(const __grid_constant__ QnArgs p, int parts) {
    sm100::pdl_trigger();
    sm100::pdl_wait();
    __shared__ float red[32][33];
    float *dw = p.side[blockIdx.y].dw;
    if (!dw) return;
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5, c = blockIdx.x * 32 + cx;
    float t = 0.f;
    if (c < p.D)
        for (int i = ry; i < parts; i += 32) t += p.partial[((int64_t)i * 2 + blockIdx.y) * p.D + c];
    red[ry][cx] = t;
    __syncthreads();
    if (ry == 0 && c < p.D) {
        t = 0.f;
        for (int i = 0; i < 32; ++i) t += red[i][cx];
        qn_put(p, dw, p.dw_bytes, dw + c, t);
    }
}

// ---------------------------------------------------------------- any D <= 256, any alignment
// A warp per item, channels c = lane + 32 j; rotation partners meet in shared memory.
constexpr int QN_J = QN_MAXD / 32;

__device__ __forceinline__ void qn_turn_generic(const QnArgs &p, bool inter, float *buf, int lane, float (&f)[QN_J],
                                                const float (&cs)[QN_J], const float (&sn)[QN_J], float sign) {
    __syncwarp();
#pragma unroll
    for (int j = 0; j < QN_J; ++j) buf[lane + 32 * j] = f[j];
    __syncwarp();
    const int half = p.R >> 1;
#pragma unroll
    for (int j = 0; j < QN_J; ++j) {
        const int c = lane + 32 * j;
        if (c < p.R) {
            const int o = inter ? (c ^ 1) : (c < half ? c + half : c - half);
            f[j] = fmaf(buf[o] * sign, sn[j], f[j] * cs[j]);
        }
    }
}

template <typename T, typename GT, bool BWD>
__global__ void __launch_bounds__(QN_NT) qk_norm_generic_kernel(const __grid_constant__ QnArgs p, int inter) {
    sm100::pdl_trigger();
    sm100::pdl_wait();
    constexpr int NW = QN_NT / 32;
    __shared__ float buf[NW][QN_MAXD];
    const QnSide &s = p.side[blockIdx.y];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    const int64_t items = p.tokens * s.chunks;
    float w[QN_J], dw[QN_J];
#pragma unroll
    for (int j = 0; j < QN_J; ++j) {
        const int c = lane + 32 * j;
        w[j] = (s.w && c < p.D) ? s.w[c] : 1.f;
        dw[j] = 0.f;
    }
    for (int64_t it = (int64_t)blockIdx.x * NW + wid; it < items; it += (int64_t)gridDim.x * NW) {
        const int64_t tok = it / s.chunks, b = tok / p.S;
        const int h0 = (int)(it - tok * s.chunks) * s.hc, h1 = min(h0 + s.hc, s.H);
        const T *x = (const T *)s.x + b * s.sb + (tok - b * p.S) * s.ss;
        float cs[QN_J], sn[QN_J];
        const int half = p.R >> 1;
        if (p.R) {
            const int64_t pos = p.pos[tok];
#pragma unroll
            for (int j = 0; j < QN_J; ++j) {
                const int c = lane + 32 * j;
                cs[j] = 1.f;
                sn[j] = 0.f;
                if (c < p.R) {
                    const bool second = inter ? (c & 1) : c >= half;
                    float t;
                    qn_angle(pos, p.inv[inter ? c >> 1 : (second ? c - half : c)], cs[j], t);
                    sn[j] = second ? t : -t;
                }
            }
        }
        for (int h = h0; h < h1; ++h) {
            const int64_t row = (tok * s.H + h) * p.D;
            float f[QN_J], g[QN_J];
            float ss = 0.f, hx = 0.f;
#pragma unroll
            for (int j = 0; j < QN_J; ++j) {
                const int c = lane + 32 * j;
                f[j] = c < p.D ? load_elem(x, (int64_t)h * p.D + c) : 0.f;
                ss = fmaf(f[j], f[j], ss);
                if (BWD) g[j] = c < p.D ? load_elem((const GT *)s.dy, row + c) : 0.f;
            }
            const float r = rsqrtf(fmaf(qn_sum<32>(ss), p.share, p.eps));
            if (BWD) {
                if (p.R) qn_turn_generic(p, inter, buf[wid], lane, g, cs, sn, -1.f);
#pragma unroll
                for (int j = 0; j < QN_J; ++j) hx = fmaf(g[j] * w[j], f[j], hx);
                const float k = qn_sum<32>(hx) * r * r * p.share;
#pragma unroll
                for (int j = 0; j < QN_J; ++j) {
                    if (lane + 32 * j < p.D) dw[j] = fmaf(g[j] * f[j], r, dw[j]);
                    f[j] = r * (g[j] * w[j] - f[j] * k);
                }
            } else {
#pragma unroll
                for (int j = 0; j < QN_J; ++j) f[j] *= r * w[j];
                if (p.R) qn_turn_generic(p, inter, buf[wid], lane, f, cs, sn, 1.f);
            }
#pragma unroll
            for (int j = 0; j < QN_J; ++j) {
                const int c = lane + 32 * j;
                if (c < p.D && in_bounds((const T *)s.y + row + c, sizeof(T), s.y, s.y_bytes, p.bounds))
                    store_elem((T *)s.y, row + c, f[j]);
            }
        }
    }
    if (!BWD || !s.dw) return;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < QN_J; ++j) buf[wid][lane + 32 * j] = dw[j];
    __syncthreads();
    for (int c = threadIdx.x; c < p.D; c += QN_NT) {
        float t = 0.f;
        for (int i = 0; i < NW; ++i) t += buf[i][c];
        qn_put(p, p.partial, p.partial_bytes, p.partial + ((int64_t)blockIdx.x * 2 + blockIdx.y) * p.D + c, t);
    }
}

// ---------------------------------------------------------------- host side
int sm_count() {
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

// Whether the 16-byte kernels take the call: whole vectors per row, aligned rows, and rotation halves
// (half-split) that start on a vector.
bool qn_vector(const kda_qk_norm_args &a, const void *const *ptrs, int n) {
    const int vec = a.dtype == KDA_F32 ? 4 : 8;
    if (a.D % vec || a.q_stride_b % vec || a.q_stride_s % vec || a.k_stride_b % vec || a.k_stride_s % vec) return false;
    if (a.rot_dim && !a.interleaved && (a.rot_dim / 2) % vec) return false;
    for (int i = 0; i < n; ++i)
        if (!aligned_to(ptrs[i], 16)) return false;
    return true;
}

// Heads per item: one token's phases serve all its heads when there are enough tokens to fill the GPU
// (64 groups of 16 lanes per SM); fewer tokens split their heads, down to the kernel's unroll of 4.
void qn_items(QnSide &s, int64_t tokens, int lanes, int sms) {
    const int64_t want = (int64_t)sms * 1024 / lanes;
    int64_t hc = (tokens * s.H + want - 1) / want;
    hc = (hc + 3) / 4 * 4;
    s.hc = (int)(hc < s.H ? hc : s.H);
    s.chunks = (s.H + s.hc - 1) / s.hc;
}

QnArgs qn_args(const kda_qk_norm_args &a) {
    QnArgs p = {};
    p.side[0] = {a.q, a.q_stride_b, a.q_stride_s, a.H_q, 0, 0, a.q_weight, a.q_out, nullptr, nullptr, 0};
    p.side[1] = {a.k, a.k_stride_b, a.k_stride_s, a.H_k, 0, 0, a.k_weight, a.k_out, nullptr, nullptr, 0};
    p.tokens = a.B * a.S;
    p.S = a.S;
    p.D = a.D;
    p.R = a.rot_dim;
    p.share = a.norm == KDA_NORM_L2 ? 1.f : 1.f / (float)a.D;
    p.eps = a.eps;
    p.pos = a.positions;
    p.inv = a.inv_freq;
    const size_t rows = (size_t)p.tokens * a.D * esize(a.dtype);
    p.side[0].y_bytes = checked_size(rows * a.H_q);
    p.side[1].y_bytes = checked_size(rows * a.H_k);
    p.bounds = checked_counter();
    return p;
}

int qn_lanes(int vectors) { return vectors <= 4 ? 4 : vectors <= 8 ? 8 : vectors <= 16 ? 16 : 32; }

// CTAs along x: enough for every item, and at most `cap`
unsigned qn_grid(const QnArgs &p, int per_cta, int64_t cap) {
    int64_t items = 0;
    for (const QnSide &s : p.side) items = s.chunks * p.tokens > items ? s.chunks * p.tokens : items;
    const int64_t n = (items + per_cta - 1) / per_cta;
    return (unsigned)(n < cap ? n : cap);
}

constexpr int QN_BWD_CTAS_PER_SM = 2;  // per side: both sides resident at once (4 per side: 209 us against 205 us)

template <typename T, typename GT, int G, int NV>
cudaError_t qn_launch_rot(const QnArgs &p, int rot, bool bwd, dim3 grid, cudaStream_t st) {
#define KDA_QN_GO(ROT)                                                                                    \
    return bwd ? launch_pdl(qk_norm_bwd_kernel<T, GT, G, NV, ROT>, grid, dim3(QN_NT), 0, st, p)            \
               : launch_pdl(qk_norm_kernel<T, G, NV, ROT>, grid, dim3(QN_NT), 0, st, p)
    if (rot == ROT_HALF) KDA_QN_GO(ROT_HALF);
    if (rot == ROT_INTERLEAVED) KDA_QN_GO(ROT_INTERLEAVED);
    KDA_QN_GO(ROT_NONE);
#undef KDA_QN_GO
}

template <typename T, typename GT>
kda_status_t qn_launch(const kda_qk_norm_args &a, QnArgs p, bool vector, bool bwd, unsigned max_ctas, unsigned *ctas,
                       cudaStream_t st) {
    constexpr int VEC = Vec16<T>::N;
    const int rot = !a.rot_dim ? ROT_NONE : a.interleaved ? ROT_INTERLEAVED : ROT_HALF;
    const int sms = sm_count();
    cudaError_t e;
    if (vector) {
        const int vectors = (a.D + VEC - 1) / VEC, G = qn_lanes(vectors < 32 ? vectors : 32);
        for (QnSide &s : p.side) qn_items(s, p.tokens, G, sms);
        const dim3 grid(*ctas = qn_grid(p, QN_NT / G, max_ctas), 2);
        if (vectors > 32) e = qn_launch_rot<T, GT, 32, 2>(p, rot, bwd, grid, st);
        else if (G == 32) e = qn_launch_rot<T, GT, 32, 1>(p, rot, bwd, grid, st);
        else if (G == 16) e = qn_launch_rot<T, GT, 16, 1>(p, rot, bwd, grid, st);
        else if (G == 8) e = qn_launch_rot<T, GT, 8, 1>(p, rot, bwd, grid, st);
        else e = qn_launch_rot<T, GT, 4, 1>(p, rot, bwd, grid, st);
    } else {
        for (QnSide &s : p.side) qn_items(s, p.tokens, 32, sms);
        const dim3 grid(*ctas = qn_grid(p, QN_NT / 32, max_ctas), 2);
        e = bwd ? launch_pdl(qk_norm_generic_kernel<T, GT, true>, grid, dim3(QN_NT), 0, st, p, (int)a.interleaved)
                : launch_pdl(qk_norm_generic_kernel<T, GT, false>, grid, dim3(QN_NT), 0, st, p, (int)a.interleaved);
    }
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "qk_norm: %s", cudaGetErrorString(e));
    return check_launch("qk_norm");
}

kda_status_t qn_validate(const kda_qk_norm_args &a) {
    KDA_TRY(check_dtype(a.dtype));
    if (a.B < 0 || a.S < 0 || a.H_q < 1 || a.H_k < 1 || a.D < 1)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes B=%lld S=%lld H_q=%d H_k=%d D=%d", (long long)a.B, (long long)a.S,
                    a.H_q, a.H_k, a.D);
    if (a.D > QN_MAXD) return fail(KDA_ERR_UNSUPPORTED, "D must be <= %d (got %d)", QN_MAXD, a.D);
    if (a.H_q > 65536 || a.H_k > 65536) return fail(KDA_ERR_UNSUPPORTED, "more than 65536 heads");
    if (a.S > 0 && a.B > 0x7fffffffLL / a.S) return fail(KDA_ERR_UNSUPPORTED, "more than 2^31 - 1 tokens");
    if (a.norm != KDA_NORM_L2 && a.norm != KDA_NORM_RMS) return fail(KDA_ERR_INVALID_ARG, "unknown norm %d", (int)a.norm);
    if (!(isfinite(a.eps) && a.eps >= 0.0f)) return fail(KDA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (a.rot_dim < 0 || a.rot_dim > a.D || a.rot_dim % 2)
        return fail(KDA_ERR_INVALID_ARG, "rot_dim must be even and within 0 .. D (got %d)", a.rot_dim);
    const int64_t lim = (int64_t)1 << 40;
    for (int64_t st : {a.q_stride_b, a.q_stride_s, a.k_stride_b, a.k_stride_s})
        if (st < 0 || st > lim) return fail(KDA_ERR_INVALID_ARG, "strides must be within 0 .. 2^40 elements");
    return KDA_OK;
}

// Bytes from the first to the last element of a strided (B, S, H, D) input.
size_t qn_extent(const kda_qk_norm_args &a, int64_t sb, int64_t ss, int H) {
    return ((size_t)(a.B - 1) * sb + (size_t)(a.S - 1) * ss + (size_t)H * a.D) * esize(a.dtype);
}

kda_status_t qn_check_common(const kda_qk_norm_args &a) {
    const size_t es = esize(a.dtype);
    KDA_REQ_PTR(a.q, "q", es);
    KDA_REQ_PTR(a.k, "k", es);
    KDA_OPT_PTR(a.q_weight, "q_weight", 4);
    KDA_OPT_PTR(a.k_weight, "k_weight", 4);
    if (a.rot_dim) {
        KDA_REQ_PTR(a.positions, "positions", 8);
        KDA_REQ_PTR(a.inv_freq, "inv_freq", 4);
    }
    return KDA_OK;
}

unsigned qn_bwd_ctas() { return (unsigned)(sm_count() * QN_BWD_CTAS_PER_SM); }

}  // namespace

}  // namespace kda

using namespace kda;

extern "C" {

kda_status_t kda_qk_norm_fwd(const kda_qk_norm_args *a) {
    clear_error();
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    KDA_TRY(qn_validate(*a));
    if (a->B == 0 || a->S == 0) return KDA_OK;
    const size_t es = esize(a->dtype), n = (size_t)a->B * a->S;
    KDA_TRY(qn_check_common(*a));
    KDA_REQ_PTR(a->q_out, "q_out", es);
    KDA_REQ_PTR(a->k_out, "k_out", es);
    const Buf ins[] = {{a->q, qn_extent(*a, a->q_stride_b, a->q_stride_s, a->H_q), "q"},
                       {a->k, qn_extent(*a, a->k_stride_b, a->k_stride_s, a->H_k), "k"},
                       {a->q_weight, (size_t)a->D * 4, "q_weight"},
                       {a->k_weight, (size_t)a->D * 4, "k_weight"},
                       {a->rot_dim ? a->positions : nullptr, n * 8, "positions"},
                       {a->rot_dim ? a->inv_freq : nullptr, (size_t)a->rot_dim * 2, "inv_freq"}};
    const size_t nq = n * a->H_q * a->D * es, nk = n * a->H_k * a->D * es;
    KDA_TRY(check_no_overlap(Buf{a->q_out, nq, "q_out"}, ins, 6));
    KDA_TRY(check_no_overlap(Buf{a->k_out, nk, "k_out"}, ins, 6));
    if (overlap(a->q_out, nq, a->k_out, nk)) return fail(KDA_ERR_INVALID_ARG, "outputs q_out and k_out overlap");
    const void *ptrs[] = {a->q, a->k, a->q_out, a->k_out};
    const bool vec = qn_vector(*a, ptrs, 4);
    const QnArgs p = qn_args(*a);
    unsigned ctas = 0;
    cudaStream_t st = (cudaStream_t)a->stream;
    return a->dtype == KDA_F32 ? qn_launch<float, float>(*a, p, vec, false, 0x7fffffffu, &ctas, st)
                               : qn_launch<__nv_bfloat16, __nv_bfloat16>(*a, p, vec, false, 0x7fffffffu, &ctas, st);
}

kda_status_t kda_qk_norm_bwd_workspace_size(const kda_qk_norm_bwd_args *a, size_t *bytes) {
    clear_error();
    if (!bytes) return fail(KDA_ERR_INVALID_ARG, "bytes is NULL");
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    KDA_TRY(qn_validate(a->fwd));
    *bytes = (a->dq_weight || a->dk_weight) ? (size_t)qn_bwd_ctas() * 2 * a->fwd.D * 4 : 0;
    return KDA_OK;
}

kda_status_t kda_qk_norm_bwd(const kda_qk_norm_bwd_args *a) {
    clear_error();
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    const kda_qk_norm_args &f = a->fwd;
    KDA_TRY(qn_validate(f));
    KDA_TRY(check_dtype(a->grad_dtype));
    if (a->grad_dtype != f.dtype && a->grad_dtype != KDA_F32)
        return fail(KDA_ERR_UNSUPPORTED, "grad_dtype must be fp32 or the dtype of q and k");
    KDA_OPT_PTR(a->dq_weight, "dq_weight", 4);
    KDA_OPT_PTR(a->dk_weight, "dk_weight", 4);
    cudaStream_t st = (cudaStream_t)f.stream;
    if (f.B == 0 || f.S == 0) {  // no token: the weights' gradients are zero
        for (float *dw : {a->dq_weight, a->dk_weight})
            if (dw && cudaMemsetAsync(dw, 0, (size_t)f.D * 4, st) != cudaSuccess)
                return fail(KDA_ERR_CUDA, "qk_norm_bwd: %s", cudaGetErrorString(cudaGetLastError()));
        return KDA_OK;
    }
    const size_t es = esize(f.dtype), gs = esize(a->grad_dtype), n = (size_t)f.B * f.S;
    KDA_TRY(qn_check_common(f));
    KDA_REQ_PTR(a->dq_out, "dq_out", gs);
    KDA_REQ_PTR(a->dk_out, "dk_out", gs);
    KDA_REQ_PTR(a->dq, "dq", es);
    KDA_REQ_PTR(a->dk, "dk", es);
    KDA_OPT_PTR(a->workspace, "workspace", 256);
    const size_t need = (a->dq_weight || a->dk_weight) ? (size_t)qn_bwd_ctas() * 2 * f.D * 4 : 0;
    if (need && (!a->workspace || a->workspace_bytes < need))
        return fail(KDA_ERR_WORKSPACE, "workspace needs %zu bytes (got %zu)", need,
                    a->workspace ? a->workspace_bytes : (size_t)0);
    const size_t eq = n * f.H_q * f.D, ek = n * f.H_k * f.D;
    const Buf ins[] = {{f.q, qn_extent(f, f.q_stride_b, f.q_stride_s, f.H_q), "q"},
                       {f.k, qn_extent(f, f.k_stride_b, f.k_stride_s, f.H_k), "k"},
                       {f.q_weight, (size_t)f.D * 4, "q_weight"},
                       {f.k_weight, (size_t)f.D * 4, "k_weight"},
                       {f.rot_dim ? f.positions : nullptr, n * 8, "positions"},
                       {f.rot_dim ? f.inv_freq : nullptr, (size_t)f.rot_dim * 2, "inv_freq"},
                       {a->dq_out, eq * gs, "dq_out"},
                       {a->dk_out, ek * gs, "dk_out"}};
    const Buf outs[] = {{a->dq, eq * es, "dq"}, {a->dk, ek * es, "dk"}, {a->dq_weight, (size_t)f.D * 4, "dq_weight"},
                        {a->dk_weight, (size_t)f.D * 4, "dk_weight"}, {need ? a->workspace : nullptr, need, "workspace"}};
    for (const Buf &o : outs) {
        if (!o.p) continue;
        KDA_TRY(check_no_overlap(o, ins, 8));
        for (const Buf &o2 : outs)
            if (&o2 != &o && overlap(o.p, o.n, o2.p, o2.n))
                return fail(KDA_ERR_INVALID_ARG, "outputs %s and %s overlap", o.name, o2.name);
    }
    QnArgs p = qn_args(f);
    p.side[0].y = a->dq;
    p.side[1].y = a->dk;
    p.side[0].dy = a->dq_out;
    p.side[1].dy = a->dk_out;
    p.side[0].dw = a->dq_weight;
    p.side[1].dw = a->dk_weight;
    p.partial = (float *)a->workspace;
    p.partial_bytes = checked_size(need);
    p.dw_bytes = checked_size((size_t)f.D * 4);
    const void *ptrs[] = {f.q, f.k, a->dq, a->dk, a->dq_out, a->dk_out};
    const bool vec = qn_vector(f, ptrs, 6);
    unsigned ctas = 0;
    const unsigned cap = qn_bwd_ctas();
    kda_status_t s;
    if (f.dtype == KDA_F32) s = qn_launch<float, float>(f, p, vec, true, cap, &ctas, st);
    else if (a->grad_dtype == KDA_F32) s = qn_launch<__nv_bfloat16, float>(f, p, vec, true, cap, &ctas, st);
    else s = qn_launch<__nv_bfloat16, __nv_bfloat16>(f, p, vec, true, cap, &ctas, st);
    if (s != KDA_OK || !need) return s;
    cudaError_t e = launch_pdl(qk_norm_dw_kernel, dim3((f.D + 31) / 32, 2), dim3(1024), 0, st, p, (int)ctas);
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "qk_norm_dw_kernel: %s", cudaGetErrorString(e));
    return check_launch("qk_norm_dw_kernel");
}

}  // extern "C"
