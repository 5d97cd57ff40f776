// Quantisation to e4m3 with one fp32 scale per block of 128 channels: of activations (1 x 128), of
// weights (128 x 128), and of the layer's normalised and gated output as it is produced:
//   scale = max(amax / 448, 2^-126) over the block (1 for a block of zeros),  value = rn_e4m3(x / scale).
// The scale maps the block's largest magnitude to e4m3's largest, so nothing saturates.
//
// Each input is read once, the values leave as 1 byte each.  The quantisers are bound by HBM: 65536 x 4096 bf16 values
// 146 us (123 at the copy rate), a 4096 x 4096 weight 13 us (8; its blocks are held in registers, two CTAs an SM).  Norm
// and gate are bound by what a channel issues (85% of the issue slots): 8192 rows x 32 heads of 128 in bf16 40 us (26),
// in fp32 66 us (46).
#include <cuda_fp8.h>

#include "host_check.cuh"
#include "kda_internal.cuh"
#include "sm100_ptx.cuh"

namespace kda {

namespace {

// What the checked build holds the stores against: bytes of the values and of the scales, and the counter.
struct Q8Size {
    size_t v, s;
    unsigned int *bounds;
};
__device__ __forceinline__ void put_scale(float *scales, int64_t i, float s, const Q8Size &z) {
    if (in_bounds(scales + i, 4, scales, z.s, z.bounds)) scales[i] = s;
}

constexpr float E4M3_MAX = 448.f, SCALE_MIN = 1.17549435e-38f;  // the smallest normal fp32 value

// An infinite or NaN element makes the scale infinite or leaves it (fmaxf ignores NaN): the block then holds
// zeros and NaN, as the division says.
__device__ __forceinline__ float q8_scale(float amax) { return amax > 0.f ? fmaxf(amax / E4M3_MAX, SCALE_MIN) : 1.f; }

__device__ __forceinline__ uint32_t q8_pack4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
__device__ __forceinline__ uint8_t q8_one(float a) { return __nv_cvt_float_to_fp8(a, __NV_SATFINITE, __NV_E4M3); }

template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int m = G / 2; m > 0; m >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, m));
    return v;
}
template <int G, typename AT>
__device__ __forceinline__ AT group_sum(AT v) {
#pragma unroll
    for (int m = G / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// ---------------------------------------------------------------- 1 x 128 blocks of a matrix
// f / s, rounded to nearest, r = 1 / s: the product with r and one correction by the remainder f - q s, which an fma
// gives exactly (Markstein, "Computation of elementary functions on the IBM RISC System/6000 processor", 1990), for
// scales with which nothing over- or underflows on the way; quotients that do are zero in e4m3.  (With the division
// alone 65536 x 4096 bf16 values take 181 us, so 146.)
template <int VEC>
__device__ __forceinline__ void divide(float (&f)[VEC], float s, float r) {
    if (s > 0x1p-60f && s < 0x1p100f) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            const float q = f[e] * r;
            f[e] = fmaf(fmaf(-q, s, f[e]), r, q);
        }
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] /= s;
    }
}

// VEC (4 or 8) values as e4m3, from the at-th of the output on
template <int VEC>
__device__ __forceinline__ void put8(uint8_t *base, int64_t at, const float (&f)[VEC], const Q8Size &z) {
    uint8_t *out = base + at;
    if (!in_bounds(out, VEC, base, z.v, z.bounds)) return;
    uint32_t w[VEC / 4];
#pragma unroll
    for (int e = 0; e < VEC; e += 4) w[e / 4] = q8_pack4(f[e], f[e + 1], f[e + 2], f[e + 3]);
    if (VEC == 8) *reinterpret_cast<uint2 *>(out) = make_uint2(w[0], w[VEC / 4 - 1]);
    else *reinterpret_cast<uint32_t *>(out) = w[0];
}

__device__ __forceinline__ void put1(uint8_t *out, int64_t at, float f, const Q8Size &z) {
    if (in_bounds(out + at, 1, out, z.v, z.bounds)) out[at] = q8_one(f);
}

// Rows of whole 16-byte vectors: 128 / VEC lanes per block, four blocks of each lane group in flight together.
// FLAT: whole blocks, that follow one another without gaps (no division per block).
template <typename T, bool FLAT>
__global__ void __launch_bounds__(256) quant_rows_vec_kernel(const T *__restrict__ x, int64_t rows, int64_t cols,
                                                             uint8_t *__restrict__ out, float *__restrict__ scales,
                                                             const Q8Size z) {
    sm100::pdl_trigger();
    sm100::pdl_wait();
    constexpr int VEC = Vec16<T>::N, G = 128 / VEC, PER = 256 / G, U = 4;
    const int lane = threadIdx.x & (G - 1);
    const unsigned nb = (unsigned)((cols + 127) / 128), blocks = (unsigned)rows * nb;
    const unsigned b0 = blockIdx.x * (PER * U) + threadIdx.x / G;
    uint4 v[U];
    int64_t at[U];
    bool in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const unsigned b = b0 + u * PER;
        if (FLAT) {
            in[u] = b < blocks;
            at[u] = (int64_t)b * 128 + lane * VEC;
        } else {
            const unsigned r = b / nb;
            const int64_t c = (int64_t)(b - r * nb) * 128 + lane * VEC;
            in[u] = b < blocks && c < cols;
            at[u] = r * cols + c;
        }
        v[u] = in[u] ? __ldcs(reinterpret_cast<const uint4 *>(x + at[u])) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float f[VEC], amax = 0.f;
        Vec16<T>::unpack(v[u], f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) amax = fmaxf(amax, fabsf(f[e]));
        const float s = q8_scale(group_max<G>(amax)), r = 1.0f / s;
        divide<VEC>(f, s, r);
        if (in[u]) {
            put8<VEC>(out, at[u], f, z);
            if (lane == 0) put_scale(scales, b0 + u * PER, s, z);
        }
    }
}

// Any others: a warp per block, lane l holds channels l + 32 j.
template <typename T>
__global__ void __launch_bounds__(256) quant_rows_kernel(const T *__restrict__ x, int64_t rows, int64_t cols,
                                                         uint8_t *__restrict__ out, float *__restrict__ scales,
                                                         const Q8Size z) {
    sm100::pdl_trigger();
    sm100::pdl_wait();
    const int l = threadIdx.x & 31;
    const int64_t nb = (cols + 127) / 128, blocks = rows * nb;
    for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < blocks; u += (int64_t)gridDim.x * 8) {
        const int64_t r = u / nb, c0 = (u - r * nb) * 128;
        const T *src = x + r * cols + c0;
        float f[4], amax = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            f[j] = c0 + l + 32 * j < cols ? load_elem(src, l + 32 * j) : 0.f;
            amax = fmaxf(amax, fabsf(f[j]));
        }
        const float s = q8_scale(group_max<32>(amax));
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (c0 + l + 32 * j < cols) put1(out, r * cols + c0 + l + 32 * j, f[j] / s, z);
        if (l == 0) put_scale(scales, u, s, z);
    }
}

// ---------------------------------------------------------------- 128 x 128 blocks of a matrix
// Rows of whole 16-byte vectors: a CTA holds its block in registers from its largest magnitude to its values.
template <typename T>
__global__ void __launch_bounds__(256) quant_tiles_vec_kernel(const T *__restrict__ x, int64_t rows, int64_t cols,
                                                              uint8_t *__restrict__ out, float *__restrict__ scales,
                                                              const Q8Size z) {
    sm100::pdl_trigger();
    sm100::pdl_wait();
    constexpr int VEC = Vec16<T>::N, G = 128 / VEC, PER = 256 / G, U = 128 / PER;
    __shared__ float s_max[8];
    const int tid = threadIdx.x;
    const int64_t nb = (cols + 127) / 128, r0 = blockIdx.x / nb * 128 + tid / G;
    const int64_t c = blockIdx.x % nb * 128 + (tid & (G - 1)) * VEC;
    uint4 v[U];
    float f[VEC], amax = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u)
        v[u] = r0 + u * PER < rows && c < cols ? __ldcs(reinterpret_cast<const uint4 *>(x + (r0 + u * PER) * cols + c))
                                               : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        Vec16<T>::unpack(v[u], f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) amax = fmaxf(amax, fabsf(f[e]));
    }
    amax = group_max<32>(amax);
    if ((tid & 31) == 0) s_max[tid >> 5] = amax;
    __syncthreads();
    amax = s_max[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) amax = fmaxf(amax, s_max[i]);
    const float s = q8_scale(amax), r = 1.0f / s;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        Vec16<T>::unpack(v[u], f);
        divide<VEC>(f, s, r);
        if (r0 + u * PER < rows && c < cols) put8<VEC>(out, (r0 + u * PER) * cols + c, f, z);
    }
    if (tid == 0) put_scale(scales, blockIdx.x, s, z);
}

// Any others: the largest magnitude of the block, then its values (the second read comes from L1/L2).
template <typename T>
__global__ void __launch_bounds__(256) quant_tiles_kernel(const T *__restrict__ x, int64_t rows, int64_t cols,
                                                          uint8_t *__restrict__ out, float *__restrict__ scales,
                                                          const Q8Size z) {
    sm100::pdl_trigger();
    sm100::pdl_wait();
    __shared__ float s_max[8];
    const int tid = threadIdx.x;
    const int64_t nb = (cols + 127) / 128, r0 = blockIdx.x / nb * 128, c0 = blockIdx.x % nb * 128;
    const int h = (int)min((int64_t)128, rows - r0), c = tid & 127;
    const bool in = c0 + c < cols;
    const T *src = x + r0 * cols + c0 + c;
    float amax = 0.f;
#pragma unroll 8
    for (int r = tid >> 7; r < h; r += 2)
        if (in) amax = fmaxf(amax, fabsf(load_elem(src, (int64_t)r * cols)));
    amax = group_max<32>(amax);
    if ((tid & 31) == 0) s_max[tid >> 5] = amax;
    __syncthreads();
    amax = s_max[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) amax = fmaxf(amax, s_max[i]);
    const float s = q8_scale(amax);
#pragma unroll 8
    for (int r = tid >> 7; r < h; r += 2)
        if (in) put1(out, (r0 + r) * cols + c0 + c, load_elem(src, (int64_t)r * cols) / s, z);
    if (tid == 0) put_scale(scales, blockIdx.x, s, z);
}

// ---------------------------------------------------------------- norm, gate and quantisation
// sigmoid to 8 half-steps of fp32 for every x, without a division: with e = exp(-|x|) (4) and d = 1 + e (1), in [1, 2], it
// is 1 / d (2), or e / d for a negative x (1).  (8192 x 32 heads of 128: 40 us; with 1 / (1 + exp(-x)) by division 61 us.)
__device__ __forceinline__ float ng8_sigmoid(float x) {
    const float e = expf(-fabsf(x));
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return x < 0.f ? e * r : r;
}

// 1 / rms of a head from its sum of squares, inv_dv = 1 / D_v.  fp32 inputs: an fp64 sum, which holds the squares of any of
// them; the root in fp64 too where the mean is not one of fp32's.
__device__ __forceinline__ float ng8_inv(float ss, float inv_dv, float eps) { return rsqrtf(fmaf(ss, inv_dv, eps)); }
__device__ __forceinline__ float ng8_inv(double ss, double inv_dv, float eps) {
    const double m = fma(ss, inv_dv, (double)eps);
    const float f = (float)m;
    return f > 1e-37f && f < 1e38f ? rsqrtf(f) : (float)(1.0 / sqrt(m));
}

// D_v = 8 (fp32: 4) .. 128, a power of two: a block of 128 channels holds whole heads.  A group of 128 / VEC
// lanes per block, 16 bytes of o and of the gate per lane; `hl` lanes share a head's norm.  Four blocks per group
// are in flight together.
// FLAT: K is a multiple of 128, so that the blocks follow one another without gaps (no division per block).
template <typename T, bool FLAT>
__global__ void __launch_bounds__(256) norm_gate_fp8_vec_kernel(const T *__restrict__ o, const T *__restrict__ gate,
                                                                int64_t N, int K, int nb, int hl,
                                                                typename AccT<T>::type inv_dv, float eps,
                                                                uint8_t *__restrict__ out, float *__restrict__ scales,
                                                                const Q8Size z) {
    sm100::pdl_trigger();
    sm100::pdl_wait();
    using AT = typename AccT<T>::type;
    constexpr int VEC = Vec16<T>::N, G = 128 / VEC, PER = 256 / G, U = 4;
    const int lane = threadIdx.x & (G - 1);
    const int64_t units = N * nb, u0 = (int64_t)blockIdx.x * (PER * U) + threadIdx.x / G;
    uint4 ov[U], gv[U];
    int64_t at[U];
    bool in[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t unit = u0 + u * PER;
        if (FLAT) {
            in[u] = unit < units;
            at[u] = unit * 128 + lane * VEC;
        } else {
            const int64_t tok = unit / nb;
            const int c = (int)(unit - tok * nb) * 128 + lane * VEC;
            in[u] = unit < units && c < K;
            at[u] = tok * K + c;
        }
        ov[u] = in[u] ? __ldcs(reinterpret_cast<const uint4 *>(o + at[u])) : make_uint4(0, 0, 0, 0);
        gv[u] = in[u] ? __ldcs(reinterpret_cast<const uint4 *>(gate + at[u])) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float f[VEC], t[VEC];
        Vec16<T>::unpack(ov[u], f);
        Vec16<T>::unpack(gv[u], t);
        AT ss = 0;
        float amax = 0.f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss += (AT)f[e] * (AT)f[e];
        for (int m = hl >> 1; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float inv = in[u] ? ng8_inv(ss, inv_dv, eps) : 0.f;  // (infinite for an absent row with eps = 0)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            f[e] = f[e] * inv * ng8_sigmoid(t[e]);
            amax = fmaxf(amax, fabsf(f[e]));
        }
        const float s = q8_scale(group_max<G>(amax)), r = 1.0f / s;
        divide<VEC>(f, s, r);
        if (in[u]) {
            put8<VEC>(out, at[u], f, z);
            if (lane == 0) put_scale(scales, u0 + u * PER, s, z);
        }
    }
}

// D_v a multiple of the vector that is no power of two: heads straddle the blocks.  A CTA of NT threads per token keeps
// the token's vectors in registers (K <= NT NG8_V vectors): their sums of squares meet in shared memory, a thread per
// head adds them up, then the blocks (128 / VEC neighbouring lanes) are quantised.
constexpr int NG8_V = 4;
template <typename T, int NT>
__global__ void __launch_bounds__(NT) norm_gate_fp8_row_kernel(const T *__restrict__ o, const T *__restrict__ gate, int H,
                                                                int Dv, float eps, uint8_t *__restrict__ out,
                                                                float *__restrict__ scales, const Q8Size z) {
    sm100::pdl_trigger();
    sm100::pdl_wait();
    using AT = typename AccT<T>::type;
    constexpr int VEC = Vec16<T>::N, G = 128 / VEC;
    __shared__ AT s_ss[NT * NG8_V];
    __shared__ float s_inv[NT * NG8_V];  // per vector; per head (a head has one vector at least)
    const int K = H * Dv, nv = K / VEC, per = Dv / VEC, nb = (K + 127) / 128;
    const int64_t base = (int64_t)blockIdx.x * K;
    uint4 ov[NG8_V], gv[NG8_V];
#pragma unroll
    for (int u = 0; u < NG8_V; ++u) {
        const int i = threadIdx.x + NT * u;
        ov[u] = gv[u] = make_uint4(0, 0, 0, 0);
        if (i < nv) {
            ov[u] = __ldcs(reinterpret_cast<const uint4 *>(o + base + i * VEC));
            gv[u] = __ldcs(reinterpret_cast<const uint4 *>(gate + base + i * VEC));
        }
    }
#pragma unroll
    for (int u = 0; u < NG8_V; ++u) {
        float f[VEC];
        AT ss = 0;
        Vec16<T>::unpack(ov[u], f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) ss += (AT)f[e] * (AT)f[e];
        s_ss[threadIdx.x + NT * u] = ss;
    }
    __syncthreads();
    for (int h = threadIdx.x; h < H; h += NT) {
        AT ss = 0;
        for (int i = 0; i < per; ++i) ss += s_ss[h * per + i];
        s_inv[h] = ng8_inv(ss, AT(1) / (AT)Dv, eps);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < NG8_V; ++u) {
        const int i = threadIdx.x + NT * u;
        if (i - (int)(threadIdx.x & 31) >= nv) break;  // (the whole warp)
        const bool in = i < nv;
        const float inv = in ? s_inv[i / per] : 0.f;
        float f[VEC], t[VEC], amax = 0.f;
        Vec16<T>::unpack(ov[u], f);
        Vec16<T>::unpack(gv[u], t);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
            f[e] = f[e] * inv * ng8_sigmoid(t[e]);
            amax = fmaxf(amax, fabsf(f[e]));
        }
        const float s = q8_scale(group_max<G>(amax)), r = 1.0f / s;
        divide<VEC>(f, s, r);
        if (in) {
            put8<VEC>(out, base + i * VEC, f, z);
            if (i % G == 0) put_scale(scales, (int64_t)blockIdx.x * nb + i / G, s, z);
        }
    }
}

// Any H and D_v: a CTA per token, first the heads' 1 / rms, then a warp per block of 128 channels.
template <typename T>
__global__ void __launch_bounds__(256) norm_gate_fp8_kernel(const T *__restrict__ o, const T *__restrict__ gate, int H,
                                                            int Dv, float eps, uint8_t *__restrict__ out,
                                                            float *__restrict__ scales, const Q8Size z) {
    sm100::pdl_trigger();
    sm100::pdl_wait();
    using AT = typename AccT<T>::type;
    extern __shared__ float s_inv[];
    const int l = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int K = H * Dv, nb = (K + 127) / 128;
    const int64_t base = (int64_t)blockIdx.x * K;
    for (int h = w; h < H; h += 8) {
        AT ss = 0;
        for (int j = l; j < Dv; j += 32) {
            const AT v = load_elem(o, base + (int64_t)h * Dv + j);
            ss += v * v;
        }
        ss = group_sum<32>(ss);
        if (l == 0) s_inv[h] = ng8_inv(ss, AT(1) / (AT)Dv, eps);
    }
    __syncthreads();
    for (int u = w; u < nb; u += 8) {
        float f[4], amax = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = 128 * u + l + 32 * j;
            f[j] = c < K ? load_elem(o, base + c) * s_inv[c / Dv] * ng8_sigmoid(load_elem(gate, base + c)) : 0.f;
            amax = fmaxf(amax, fabsf(f[j]));
        }
        const float s = q8_scale(group_max<32>(amax));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = 128 * u + l + 32 * j;
            if (c < K) put1(out, base + c, f[j] / s, z);
        }
        if (l == 0) put_scale(scales, (int64_t)blockIdx.x * nb + u, s, z);
    }
}

template <typename T>
cudaError_t ng8_launch(const void *o, const void *gl, int64_t N, int H, int Dv, float eps, void *x8, float *scales,
                       cudaStream_t st) {
    constexpr int VEC = Vec16<T>::N;
    const int K = H * Dv, nb = (K + 127) / 128;
    const Q8Size z = {checked_size((size_t)N * K), checked_size((size_t)N * nb * 4), checked_counter()};
    // whole 16-byte vectors of one head per lane, whole heads per block, aligned rows
    if (Dv >= VEC && Dv <= 128 && (Dv & (Dv - 1)) == 0 && aligned_to(o, 16) && aligned_to(gl, 16) && aligned_to(x8, VEC)) {
        const int64_t ctas = (N * nb + 8 * VEC - 1) / (8 * VEC);  // 256 threads: 2 VEC groups of four blocks
        if (ctas <= 0x7fffffffLL)
            return launch_pdl(K % 128 ? norm_gate_fp8_vec_kernel<T, false> : norm_gate_fp8_vec_kernel<T, true>,
                              dim3((unsigned)ctas), dim3(256), 0, st, (const T *)o, (const T *)gl, N, K, nb, Dv / VEC,
                              typename AccT<T>::type(1) / Dv, eps, (uint8_t *)x8, scales, z);
    }
    if (Dv % VEC == 0 && K / VEC <= 256 * NG8_V && aligned_to(o, 16) && aligned_to(gl, 16) && aligned_to(x8, VEC)) {
        // the fewest threads that hold the token: 9109 tokens x 4 heads of 80 take 37 us with 256, 12 us with 64
        const int nv = K / VEC, nt = nv <= 64 * NG8_V ? 64 : nv <= 128 * NG8_V ? 128 : 256;
        const auto kernel = nt == 64    ? norm_gate_fp8_row_kernel<T, 64>
                            : nt == 128 ? norm_gate_fp8_row_kernel<T, 128>
                                        : norm_gate_fp8_row_kernel<T, 256>;
        return launch_pdl(kernel, dim3((unsigned)N), dim3(nt), 0, st, (const T *)o, (const T *)gl, H, Dv, eps,
                          (uint8_t *)x8, scales, z);
    }
    return launch_pdl(norm_gate_fp8_kernel<T>, dim3((unsigned)N), dim3(256), (size_t)H * 4, st, (const T *)o,
                      (const T *)gl, H, Dv, eps, (uint8_t *)x8, scales, z);
}

template <typename T>
cudaError_t launch_quant(const void *x, int64_t rows, int64_t cols, int block_rows, int64_t units, uint8_t *y,
                         float *scales, cudaStream_t st) {
    constexpr int VEC = Vec16<T>::N, PER = 256 / (128 / VEC) * 4;
    const Q8Size z = {checked_size((size_t)rows * cols), checked_size((size_t)units * 4), checked_counter()};
    auto go = [&](auto kernel, int64_t ctas) {
        return launch_pdl(kernel, dim3((unsigned)(ctas < 0x7fffffffLL ? ctas : 0x7fffffffLL)), dim3(256), 0, st,
                          (const T *)x, rows, cols, y, scales, z);
    };
    const bool vec = cols % VEC == 0 && aligned_to(x, 16) && aligned_to(y, VEC);
    if (block_rows != 1) return go(vec ? quant_tiles_vec_kernel<T> : quant_tiles_kernel<T>, units);
    if (vec && units < 0x7fffffffLL)
        return go(cols % 128 == 0 ? quant_rows_vec_kernel<T, true> : quant_rows_vec_kernel<T, false>, (units + PER - 1) / PER);
    return go(quant_rows_kernel<T>, (units + 7) / 8);
}

}  // namespace

}  // namespace kda

using namespace kda;

extern "C" {

kda_status_t kda_quant_fp8(const void *x, kda_dtype_t dtype, int64_t rows, int64_t cols, int32_t block_rows, void *x8,
                           float *scales, void *stream) {
    clear_error();
    KDA_TRY(check_dtype(dtype));
    if (rows < 0 || cols < 1) return fail(KDA_ERR_INVALID_ARG, "bad sizes");
    if (block_rows != 1 && block_rows != 128) return fail(KDA_ERR_INVALID_ARG, "block_rows must be 1 or 128");
    if (cols > 0x7fffffffLL || rows > ((int64_t)1 << 46) / cols) return fail(KDA_ERR_UNSUPPORTED, "matrix too large");
    const int64_t nb = (cols + 127) / 128, units = block_rows == 1 ? rows * nb : (rows + 127) / 128 * nb;
    if (block_rows == 128 && units > 0x7fffffffLL) return fail(KDA_ERR_UNSUPPORTED, "matrix too large");
    if (rows == 0) return KDA_OK;
    const size_t es = esize(dtype), n = (size_t)rows * cols;
    KDA_REQ_PTR(x, "x", es);
    KDA_REQ_PTR(x8, "x8", 1);
    KDA_REQ_PTR(scales, "scales", 4);
    const Buf in[] = {{x, n * es, "x"}};
    KDA_TRY(check_no_overlap(Buf{x8, n, "x8"}, in, 1));
    KDA_TRY(check_no_overlap(Buf{scales, (size_t)units * 4, "scales"}, in, 1));
    if (overlap(x8, n, scales, (size_t)units * 4)) return fail(KDA_ERR_INVALID_ARG, "outputs x8 and scales overlap");
    cudaStream_t st = (cudaStream_t)stream;
    uint8_t *y = (uint8_t *)x8;
    cudaError_t e = dtype == KDA_F32 ? launch_quant<float>(x, rows, cols, block_rows, units, y, scales, st)
                                     : launch_quant<__nv_bfloat16>(x, rows, cols, block_rows, units, y, scales, st);
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "quant_fp8: %s", cudaGetErrorString(e));
    return check_launch("quant_fp8");
}

kda_status_t kda_norm_gate_fp8(const void *o, const void *gl, int64_t N, int32_t H, int32_t Dv, float eps,
                               kda_dtype_t dtype, void *x8, float *scales, void *stream) {
    clear_error();
    KDA_TRY(check_dtype(dtype));
    if (N < 0 || H < 1 || Dv < 1) return fail(KDA_ERR_INVALID_ARG, "bad sizes");
    if (!(isfinite(eps) && eps >= 0.0f)) return fail(KDA_ERR_INVALID_ARG, "eps must be finite and >= 0");
    if (H > 8192 || Dv > 8192) return fail(KDA_ERR_UNSUPPORTED, "H and D_v must be <= 8192");
    if (N > 0x7fffffffLL) return fail(KDA_ERR_UNSUPPORTED, "more than 2^31 - 1 rows");
    if (N == 0) return KDA_OK;
    const size_t es = esize(dtype), K = (size_t)H * Dv, n = (size_t)N * K, ns = (size_t)N * ((K + 127) / 128) * 4;
    KDA_REQ_PTR(o, "o", es);
    KDA_REQ_PTR(gl, "gate_logits", es);
    KDA_REQ_PTR(x8, "x8", 1);
    KDA_REQ_PTR(scales, "scales", 4);
    const Buf ins[] = {{o, n * es, "o"}, {gl, n * es, "gate_logits"}};
    KDA_TRY(check_no_overlap(Buf{x8, n, "x8"}, ins, 2));
    KDA_TRY(check_no_overlap(Buf{scales, ns, "scales"}, ins, 2));
    if (overlap(x8, n, scales, ns)) return fail(KDA_ERR_INVALID_ARG, "outputs x8 and scales overlap");
    cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = dtype == KDA_F32 ? ng8_launch<float>(o, gl, N, H, Dv, eps, x8, scales, st)
                                           : ng8_launch<__nv_bfloat16>(o, gl, N, H, Dv, eps, x8, scales, st);
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "norm_gate_fp8: %s", cudaGetErrorString(e));
    return check_launch("norm_gate_fp8");
}

}  // extern "C"
