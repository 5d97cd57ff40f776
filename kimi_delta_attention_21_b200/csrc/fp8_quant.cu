// Quantisation to e4m3 with one fp32 scale per block of 128 channels: of activations (1 x 128), of
// weights (128 x 128), and of the layer's normalised and gated output as it is produced:
//   scale = max(amax / 448, 2^-126) over the block (1 for a block of zeros),  value = rn_e4m3(x / scale).
// The scale maps the block's largest magnitude to e4m3's largest, so nothing saturates.
//
// All are bound by HBM: each input is read once, the values leave as 1 byte each.
#include <cuda_fp8.h>

#include "host_check.cuh"
#include "kda_internal.cuh"
#include "sm100_ptx.cuh"

namespace kda {

namespace {

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
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int m = G / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
    return v;
}

// ---------------------------------------------------------------- 1 x 128 blocks of a matrix
// A warp per block; lane l holds channels 4l .. 4l + 3 (VEC: 4-byte aligned quads), or l + 32 j.
template <typename T>
__global__ void __launch_bounds__(256) quant_rows_kernel(const T *__restrict__ x, int64_t rows, int64_t cols,
                                                         uint8_t *__restrict__ out, float *__restrict__ scales) {
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
            if (c0 + l + 32 * j < cols) out[r * cols + c0 + l + 32 * j] = q8_one(f[j] / s);
        if (l == 0) scales[u] = s;
    }
}

// ---------------------------------------------------------------- 128 x 128 blocks of a matrix
// A CTA per block: its largest magnitude, then its values (the second read comes from L1/L2).
template <typename T>
__global__ void __launch_bounds__(256) quant_tiles_kernel(const T *__restrict__ x, int64_t rows, int64_t cols,
                                                          uint8_t *__restrict__ out, float *__restrict__ scales) {
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
        if (in) out[(r0 + r) * cols + c0 + c] = q8_one(load_elem(src, (int64_t)r * cols) / s);
    if (tid == 0) scales[blockIdx.x] = s;
}

// ---------------------------------------------------------------- norm, gate and quantisation
// Any H and D_v: a CTA per token, first the heads' 1 / rms, then a warp per block of 128 channels.
template <typename T>
__global__ void __launch_bounds__(256) norm_gate_fp8_kernel(const T *__restrict__ o, const T *__restrict__ gate, int H,
                                                            int Dv, float eps, uint8_t *__restrict__ out,
                                                            float *__restrict__ scales) {
    sm100::pdl_trigger();
    sm100::pdl_wait();
    extern __shared__ float s_inv[];
    const int l = threadIdx.x & 31, w = threadIdx.x >> 5;
    const int K = H * Dv, nb = (K + 127) / 128;
    const int64_t base = (int64_t)blockIdx.x * K;
    for (int h = w; h < H; h += 8) {
        float ss = 0.f;
        for (int j = l; j < Dv; j += 32) {
            const float v = load_elem(o, base + (int64_t)h * Dv + j);
            ss = fmaf(v, v, ss);
        }
        ss = group_sum<32>(ss);
        if (l == 0) s_inv[h] = 1.0f / sqrtf(ss / (float)Dv + eps);
    }
    __syncthreads();
    for (int u = w; u < nb; u += 8) {
        float f[4], amax = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = 128 * u + l + 32 * j;
            f[j] = c < K ? load_elem(o, base + c) * s_inv[c / Dv] * sigmoid_precise(load_elem(gate, base + c)) : 0.f;
            amax = fmaxf(amax, fabsf(f[j]));
        }
        const float s = q8_scale(group_max<32>(amax));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = 128 * u + l + 32 * j;
            if (c < K) out[base + c] = q8_one(f[j] / s);
        }
        if (l == 0) scales[(int64_t)blockIdx.x * nb + u] = s;
    }
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
    const int64_t ctas = block_rows == 1 ? (units + 7) / 8 : units;
    const dim3 grid((unsigned)(ctas < 0x7fffffffLL ? ctas : 0x7fffffffLL));
    cudaError_t e;
    if (dtype == KDA_F32)
        e = launch_pdl(block_rows == 1 ? quant_rows_kernel<float> : quant_tiles_kernel<float>, grid, dim3(256), 0, st,
                       (const float *)x, rows, cols, y, scales);
    else
        e = launch_pdl(block_rows == 1 ? quant_rows_kernel<__nv_bfloat16> : quant_tiles_kernel<__nv_bfloat16>, grid,
                       dim3(256), 0, st, (const __nv_bfloat16 *)x, rows, cols, y, scales);
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
    cudaError_t e;
    if (dtype == KDA_F32)
        e = launch_pdl(norm_gate_fp8_kernel<float>, dim3((unsigned)N), dim3(256), (size_t)H * 4, st, (const float *)o,
                       (const float *)gl, H, Dv, eps, (uint8_t *)x8, scales);
    else
        e = launch_pdl(norm_gate_fp8_kernel<__nv_bfloat16>, dim3((unsigned)N), dim3(256), (size_t)H * 4, st,
                       (const __nv_bfloat16 *)o, (const __nv_bfloat16 *)gl, H, Dv, eps, (uint8_t *)x8, scales);
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "norm_gate_fp8: %s", cudaGetErrorString(e));
    return check_launch("norm_gate_fp8");
}

}  // extern "C"
