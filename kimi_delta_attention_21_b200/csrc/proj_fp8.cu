// Output projection from e4m3 operands with a scale per block of 128:
//   y[n, m] = sum_kb xs[n, kb] ws[m / 128, kb] sum_{i in block kb} x[n, i] W[m, i]
// (x: 1 x 128 blocks, W: 128 x 128 blocks), on the 5th-generation tensor cores (kind::f8f6f4).
//
// The scales change with every 128 of the sum, so the tensor core accumulates one block at a time and the
// blocks are added in fp32 registers: y += (xs ws) * partial.  Persistent, warp-specialised, one CTA per SM
// over 128 x BN output tiles:
//   warp 0       TMA producer: 128 x 128-byte tiles of x and BN x 128-byte tiles of W into a ring of
//                shared-memory stages (128-byte swizzle);
//   warp 1       MMA issuer: 4 tcgen05.mma (M = 128, N = BN, K = 32) per block, into 512 / BN TMEM
//                accumulators in turn;
//   warps 4..11  two warps per TMEM lane quarter, half the columns each: read the block's accumulator,
//                scale and add it to the tile's sums (BN / 2 registers per thread: the register split below)
//                while the tensor core works on the next block; after the last block, through shared memory
//                to y by TMA.
// A block of a 128 x 256 tile takes the tensor core 512 cycles at the nominal rate; the 32768 additions take
// the SM's 128 fp32 lanes 256, so the tensor core stays the bound.
#include <cuda_fp8.h>

#include "host_check.cuh"
#include "kda_internal.cuh"
#include "sm100_ptx.cuh"
#include "tma_host.cuh"

namespace kda {

namespace {

using namespace sm100;

constexpr int PM = 128, PK = 128, PF_NT = 384;

// kind::f8f6f4, e4m3 operands (format 0), fp32 accumulation, both K-major
constexpr uint32_t idesc_e4m3(int M, int N) {
    return (1u << 4) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ void mma_f8_ss(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap *map, const void *smem_src, int x, int y) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(smem_u32(smem_src)), "r"(x), "r"(y)
                 : "memory");
}

template <int BN> struct P8Cfg {
    static constexpr int STAGES = BN >= 256 ? 4 : (BN >= 128 ? 5 : 7);
    static constexpr uint32_t A_BYTES = PM * PK, B_BYTES = BN * PK, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int BUFS = 512 / BN;            // TMEM accumulators
    static constexpr uint32_t OUT_BYTES = 8 * 32 * 128;  // each epilogue warp: 32 rows of 128 bytes
    // bytes of a row that an epilogue warp stores at a time: its BN / 2 columns, at most 128 bytes
    template <typename OT> static constexpr int row_bytes() {
        return BN / 2 * (int)sizeof(OT) < 128 ? BN / 2 * (int)sizeof(OT) : 128;
    }
    static constexpr size_t SMEM = STAGES * STAGE_BYTES + OUT_BYTES + 1024 + 512;
};

// 32 columns of an accumulator, scaled and added: two per instruction, which leaves the other warps twice the issue
// slots (with single fmas 16384 x 4096 x 4096 took 279 us, so 255 us)
template <int HC>
__device__ __forceinline__ void add_scaled(float (&acc)[HC], int c, const uint32_t (&r)[32], float s) {
#pragma unroll
    for (int j = 0; j < 32; j += 2)
        asm("{\n\t.reg .b64 a, b, d;\n\t"
            "mov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %4};\n\tmov.b64 d, {%0, %1};\n\t"
            "fma.rn.f32x2 d, a, b, d;\n\tmov.b64 {%0, %1}, d;\n\t}"
            : "+f"(acc[c + j]), "+f"(acc[c + j + 1])
            : "r"(r[j]), "r"(r[j + 1]), "f"(s));
}

template <int BN, typename OT>
__global__ void __launch_bounds__(PF_NT, 1)
proj_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmY, const float *__restrict__ xs, const float *__restrict__ ws,
                int M, int N, int K, unsigned int *timeouts) {
    pdl_trigger();
    pdl_wait();
    using Cfg = P8Cfg<BN>;
    constexpr int ST = Cfg::STAGES, HC = BN / 2;  // columns per epilogue warp
    constexpr int NB = Cfg::BUFS;
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = smraw + ((1024u - (static_cast<uint32_t>(__cvta_generic_to_shared(smraw)) & 1023u)) & 1023u);
    uint8_t *sA = sm, *sB = sm + ST * Cfg::A_BYTES, *sY = sm + ST * Cfg::STAGE_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(sY + Cfg::OUT_BYTES);
    uint64_t *empty = full + ST;
    uint64_t *acc_full = empty + ST;      // [NB] MMA -> epilogue
    uint64_t *acc_empty = acc_full + NB;  // [NB] epilogue -> MMA
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + NB);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int tiles_m = (M + PM - 1) / PM, tiles_n = (N + BN - 1) / BN, tiles = tiles_m * tiles_n;
    const int KB = (K + PK - 1) / PK;
    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8);  // one arrival per epilogue warp
        }
        fence_barrier_init();
        prefetch_tensormap(&tmA);
        prefetch_tensormap(&tmB);
        prefetch_tensormap(&tmY);
    }
    if (warp == 0) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    bool timed_out = false;

    // groups of 8 row tiles, columns within: CTAs that run at the same time share x and W in L2
    auto tile_mn = [&](int t, int &m0, int &n0) {
        const int group = 8, gm = t / (group * tiles_n), rem = t % (group * tiles_n);
        const int rows = min(group, tiles_m - gm * group);
        m0 = (gm * group + rem % rows) * PM;
        n0 = (rem / rows) * BN;
    };

    if (warp < 4) {
        // registers: 384 threads x 168 at launch = 128 x 72 + 256 x 216
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        if (warp == 0 && lane == 0) {
            int it = 0;
            for (int t = blockIdx.x; t < tiles && !timed_out; t += gridDim.x) {
                int m0, n0;
                tile_mn(t, m0, n0);
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const int s = it % ST;
                    if (it >= ST && !mbar_wait(&empty[s], ((it / ST) - 1) & 1)) {
                        timed_out = true;
                        break;
                    }
                    mbar_arrive_expect_tx(&full[s], Cfg::STAGE_BYTES);
                    tma_load_2d(sA + s * Cfg::A_BYTES, &tmA, &full[s], kb * PK, m0);
                    tma_load_2d(sB + s * Cfg::B_BYTES, &tmB, &full[s], kb * PK, n0);
                }
            }
            if (timed_out)  // let the copies already issued land before the CTA can exit
                for (int j = (it > ST ? it - ST : 0); j < it; ++j) mbar_wait(&full[j % ST], (j / ST) & 1);
        } else if (warp == 1 && lane == 0) {
            constexpr uint32_t idesc = idesc_e4m3(PM, BN);
            int it = 0;
            for (int t = blockIdx.x; t < tiles && !timed_out; t += gridDim.x) {
                for (int kb = 0; kb < KB; ++kb, ++it) {
                    const int s = it % ST, buf = it % NB;
                    // the accumulator was read (NB blocks ago), and the operands are there
                    if ((it >= NB && !mbar_wait(&acc_empty[buf], ((it / NB) - 1) & 1)) ||
                        !mbar_wait(&full[s], (it / ST) & 1)) {
                        timed_out = true;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t ad = smem_desc(smem_u32(sA + s * Cfg::A_BYTES), 16, 1024, LAYOUT_SW128);
                    const uint64_t bd = smem_desc(smem_u32(sB + s * Cfg::B_BYTES), 16, 1024, LAYOUT_SW128);
#pragma unroll
                    for (int k = 0; k < PK / 32; ++k)
                        mma_f8_ss(tmem + buf * BN, ad + (uint64_t)(k * 2), bd + (uint64_t)(k * 2), idesc, k != 0);
                    mma_commit(&acc_full[buf]);
                    mma_commit(&empty[s]);
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        const int e = warp - 4, q = warp & 3, half = e >> 2;  // lane quarter (fixed by the warp), column half
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        uint8_t *out = sY + e * 4096;
        int it = 0;
        for (int t = blockIdx.x; t < tiles && !timed_out; t += gridDim.x) {
            int m0, n0;
            tile_mn(t, m0, n0);
            const int row = m0 + 32 * q + lane, c0 = n0 + half * HC;
            const float *xr = xs + (int64_t)min(row, M - 1) * KB;
            const float *wr = ws + (int64_t)(min(c0, N - 1) / PK) * KB;  // (HC <= 128 columns: one block of W)
            float acc[HC];
#pragma unroll
            for (int i = 0; i < HC; ++i) acc[i] = 0.f;
            // 32 columns at a time: while they are added, the next 32 are on their way, those of the next block too
            constexpr int NC = HC / 32;
            static_assert(NC == 1 || NC % 2 == 0, "two register buffers in turn");
            uint32_t r0[32], r1[32];
            auto ready = [&](int i) {  // waits for block i's accumulator
                if (!__all_sync(0xffffffffu, mbar_wait(&acc_full[i % NB], (i / NB) & 1))) timed_out = true;
                tc_fence_after();
            };
            auto load = [&](int i, int c, uint32_t(&r)[32]) {
                tmem_ld_32x32b_x32(tmem + lane_base + (i % NB) * BN + half * HC + 32 * c, r);
            };
            auto release = [&](int i) {  // everything of block i's accumulator has been read
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&acc_empty[i % NB]);
            };
            float s = xr[0] * wr[0];
            ready(it);
            if (timed_out) break;
            load(it, 0, r0);
            for (int kb = 0; kb < KB; ++kb, ++it) {
                const bool more = kb + 1 < KB;
                const float sx = more ? xr[kb + 1] : 0.f, sw = more ? wr[kb + 1] : 0.f;
                if (NC == 1) {
                    tmem_wait_ld();
                    release(it);
#pragma unroll
                    for (int j = 0; j < 32; ++j) r1[j] = r0[j];
                    if (more) {
                        ready(it + 1);
                        if (timed_out) break;
                        load(it + 1, 0, r0);
                    }
                    add_scaled<HC>(acc, 0, r1, s);
                } else {
#pragma unroll
                    for (int c = 0; c < NC; c += 2) {
                        tmem_wait_ld();
                        load(it, c + 1, r1);
                        add_scaled<HC>(acc, 32 * c, r0, s);
                        tmem_wait_ld();
                        if (c + 2 < NC) {
                            load(it, c + 2, r0);
                        } else {
                            release(it);
                            if (more) {
                                ready(it + 1);
                                if (!timed_out) load(it + 1, 0, r0);
                            }
                        }
                        add_scaled<HC>(acc, 32 * (c + 1), r1, s);
                    }
                    if (timed_out) break;
                }
                s = sx * sw;
            }
            if (timed_out) break;
            // the warp's 32 rows, up to 128 bytes of columns at a time, in the swizzle of the store's map: the
            // 16-byte chunk within a row of RB bytes is xored with the row's place in the swizzle's period
            constexpr int RB = Cfg::template row_bytes<OT>(), PER = RB / (int)sizeof(OT), E = 16 / (int)sizeof(OT);
            const int swz = RB == 128 ? (lane & 7) : ((lane >> 1) & 3);
#pragma unroll
            for (int c = 0; c < HC; c += PER) {
                if (lane == 0) bulk_wait_read_all();  // the store that used the buffer has read it
                __syncwarp();
#pragma unroll
                for (int g = 0; g < RB / 16; ++g) {
                    uint32_t pv[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        if (sizeof(OT) == 2) {
                            const __nv_bfloat162 h2 =
                                __floats2bfloat162_rn(acc[c + E * g + 2 * j], acc[c + E * g + 2 * j + 1]);
                            pv[j] = *reinterpret_cast<const uint32_t *>(&h2);
                        } else {
                            pv[j] = __float_as_uint(acc[c + E * g + j]);
                        }
                    }
                    *reinterpret_cast<uint4 *>(out + lane * RB + ((g ^ swz) << 4)) = make_uint4(pv[0], pv[1], pv[2], pv[3]);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && m0 + 32 * q < M && c0 + c < N) {
                    tma_store_2d(&tmY, out, c0 + c, m0 + 32 * q);
                    bulk_commit();
                }
            }
        }
        if (lane == 0) bulk_wait_all();
    }
    if (timed_out && timeouts) atomicAdd(timeouts, 1u);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- any K, any alignment
// 64 x 64 output tiles, 16 channels at a time, exact fp32.
template <typename OT>
__global__ void __launch_bounds__(256) proj_fp8_simt_kernel(const uint8_t *__restrict__ x, const float *__restrict__ xs,
                                                            const uint8_t *__restrict__ w, const float *__restrict__ ws,
                                                            int64_t M, int N, int K, OT *__restrict__ y) {
    pdl_trigger();
    pdl_wait();
    __shared__ float sX[16][65], sW[16][65];
    const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4, KB = (K + PK - 1) / PK;
    const int64_t tiles_n = (N + 63) / 64, m0 = blockIdx.x / tiles_n * 64;
    const int n0 = (int)(blockIdx.x % tiles_n) * 64;
    auto value = [](uint8_t v) {
        return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)v, __NV_E4M3)));
    };
    float acc[4][4] = {}, part[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += 16) {
        for (int i = tid; i < 1024; i += 256) {
            const int r = i >> 4, c = i & 15;
            const bool k_in = k0 + c < K;
            sX[c][r] = k_in && m0 + r < M ? value(x[(m0 + r) * K + k0 + c]) : 0.f;
            sW[c][r] = k_in && n0 + r < N ? value(w[(int64_t)(n0 + r) * K + k0 + c]) : 0.f;
        }
        __syncthreads();
#pragma unroll
        for (int c = 0; c < 16; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) part[i][j] = fmaf(sX[c][ty + 16 * i], sW[c][tx + 16 * j], part[i][j]);
        __syncthreads();
        if ((k0 + 16) % PK == 0 || k0 + 16 >= K) {  // a block of the sum is complete (blocks of 128: whole steps of 16)
            const int kb = k0 / PK;
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int64_t r = m0 + ty + 16 * i;
                    const int c = n0 + tx + 16 * j;
                    if (r < M && c < N) acc[i][j] = fmaf(xs[r * KB + kb] * ws[(int64_t)(c / PK) * KB + kb], part[i][j], acc[i][j]);
                    part[i][j] = 0.f;
                }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int64_t r = m0 + ty + 16 * i;
            const int c = n0 + tx + 16 * j;
            if (r < M && c < N) store_elem(y, r * N + c, acc[i][j]);
        }
}

// ---------------------------------------------------------------- host side
struct P8Args {
    const void *x, *w;
    const float *xs, *ws;
    int64_t N;
    int K, M;
    void *y;
    kda_dtype_t out;
};

template <int BN, typename OT>
kda_status_t launch_tc(const P8Args &a, int sms, cudaStream_t st) {
    using Cfg = P8Cfg<BN>;
    CUtensorMap ta, tb, ty;
    KDA_TRY(make_tmap_2d(&ta, a.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)a.N, (uint64_t)a.K, (uint64_t)a.K, PM, PK,
                         CU_TENSOR_MAP_SWIZZLE_128B));
    KDA_TRY(make_tmap_2d(&tb, a.w, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)a.M, (uint64_t)a.K, (uint64_t)a.K, BN, PK,
                         CU_TENSOR_MAP_SWIZZLE_128B));
    constexpr int RB = Cfg::template row_bytes<OT>();
    KDA_TRY(make_tmap_2d(&ty, a.y, sizeof(OT) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                         (int)sizeof(OT), (uint64_t)a.N, (uint64_t)a.M, (uint64_t)a.M, 32, RB / sizeof(OT),
                         RB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B));
    cudaFuncSetAttribute(proj_fp8_kernel<BN, OT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Cfg::SMEM);
    const int64_t tiles = ((a.N + PM - 1) / PM) * ((a.M + BN - 1) / BN);
    const cudaError_t e =
        launch_pdl(proj_fp8_kernel<BN, OT>, dim3((unsigned)(tiles < sms ? tiles : sms)), dim3(PF_NT), Cfg::SMEM, st, ta, tb,
                   ty, a.xs, a.ws, (int)a.N, a.M, a.K, device_timeout_counter());
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "proj_fp8_kernel: %s", cudaGetErrorString(e));
    return check_launch("proj_fp8_kernel");
}

template <typename OT>
kda_status_t launch_proj_fp8(const P8Args &a, cudaStream_t st) {
    // whole 16-byte vectors in the rows of x, W and y, and aligned bases: what the TMA maps ask for
    const bool tc = a.K % 16 == 0 && a.M % (16 / (int)sizeof(OT)) == 0 && aligned_to(a.x, 16) && aligned_to(a.w, 16) &&
                    aligned_to(a.y, 16);
    if (!tc) {
        const int64_t ctas = ((a.N + 63) / 64) * ((a.M + 63) / 64);
        const cudaError_t e = launch_pdl(proj_fp8_simt_kernel<OT>, dim3((unsigned)ctas), dim3(256), 0, st,
                                         (const uint8_t *)a.x, a.xs, (const uint8_t *)a.w, a.ws, a.N, a.M, a.K, (OT *)a.y);
        if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "proj_fp8_simt_kernel: %s", cudaGetErrorString(e));
        return check_launch("proj_fp8_simt_kernel");
    }
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    // few rows: narrow tiles, so that more SMs take part
    const int64_t tiles256 = ((a.N + PM - 1) / PM) * ((a.M + 255) / 256);
    if (tiles256 < sms) return launch_tc<64, OT>(a, sms, st);
    return launch_tc<256, OT>(a, sms, st);
}

}  // namespace

}  // namespace kda

using namespace kda;

extern "C" kda_status_t kda_out_proj_fp8(const void *x8, const float *x_scale, const void *W8, const float *W_scale,
                                         int64_t N, int32_t K, int32_t Dm, void *y, kda_dtype_t out_dtype, void *stream) {
    clear_error();
    KDA_TRY(check_dtype(out_dtype));
    if (N < 0 || K < 1 || Dm < 1) return fail(KDA_ERR_INVALID_ARG, "bad sizes");
    // row tiles times column tiles (of 64) within the grid's and the tile counter's 31 bits
    if (N > 0x7fffffffLL - 256 || K > 0x7fffffff - 256 || Dm > 0x7fffffff - 256 ||
        ((N + 63) / 64) * (((int64_t)Dm + 63) / 64) > 0x7fffffffLL)
        return fail(KDA_ERR_UNSUPPORTED, "N=%lld, K=%d, D_model=%d: too large", (long long)N, K, Dm);
    if (N == 0) return KDA_OK;
    const size_t os = esize(out_dtype), kb = ((size_t)K + 127) / 128;
    KDA_REQ_PTR(x8, "x8", 1);
    KDA_REQ_PTR(x_scale, "x_scale", 4);
    KDA_REQ_PTR(W8, "W8", 1);
    KDA_REQ_PTR(W_scale, "W_scale", 4);
    KDA_REQ_PTR(y, "y", os);
    const Buf ins[] = {{x8, (size_t)N * K, "x8"}, {x_scale, (size_t)N * kb * 4, "x_scale"}, {W8, (size_t)Dm * K, "W8"},
                       {W_scale, (((size_t)Dm + 127) / 128) * kb * 4, "W_scale"}};
    KDA_TRY(check_no_overlap(Buf{y, (size_t)N * Dm * os, "y"}, ins, 4));
    const P8Args a = {x8, W8, x_scale, W_scale, N, K, Dm, y, out_dtype};
    return out_dtype == KDA_F32 ? launch_proj_fp8<float>(a, (cudaStream_t)stream)
                                : launch_proj_fp8<__nv_bfloat16>(a, (cudaStream_t)stream);
}
