// Output projection from e4m3 operands with a scale per block of 128:
//   y[n, m] = sum_kb xs[n, kb] ws[m / 128, kb] sum_{i in block kb} x[n, i] W[m, i]
// (x: 1 x 128 blocks, W: 128 x 128 blocks), on the 5th-generation tensor cores (kind::f8f6f4).
//
// The scales change with every 128 of the sum, so the tensor core accumulates one block at a time and the
// blocks are added in fp32 registers: y += (xs ws) * partial.  Warp-specialised:
//   warp 0       TMA producer: 128 x 128-byte tiles of x and of W into a ring of shared-memory stages
//                (128-byte swizzle);
//   warp 1       MMA issuer: 4 tcgen05.mma (K = 32) per block, into TMEM accumulators in turn;
//   warps 4..11  two warps per TMEM lane quarter, half the columns each: read the block's accumulator,
//                scale it and add it to the tile's sums (registers; see the split below) while the tensor
//                core works on the next block.
// Two kernels.  Many rows (proj_fp8_kernel): persistent, one CTA per SM over 128 x 256 tiles.  Per block the
// tensor core needs 512 cycles at the nominal rate, the 32768 additions 256 of the SM's 128 fp32 lanes; what it
// reaches (16384 x 4096 x 4096: 255 us, 2150 TFLOP/s; without the additions 220 us) is held by the loads and, in
// long runs, by the power limit.  CTA pairs (cta_group::2, 256 x 256 tiles) were measured no faster: 262 us,
// 319 us with the accumulators handed over in halves.  Few rows (proj_fp8_split_kernel): a 128 x 128 tile per
// cluster, whose CTAs take a part of the blocks each and add their sums through distributed shared memory, in
// rank order (256 x 4096 x 4096: 12.6 us a call against 15.5 us with 128 x 64 tiles and no split).
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

// What the checked build holds the stores to y against.
struct YSize {
    size_t n;
    unsigned int *bounds;
};

// Address of a shared-memory object of this CTA in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
// Every thread of every CTA of the cluster (all their waits are bounded, so all of them arrive).
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

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

// The epilogue's main loop: adds `n` blocks, from the it-th accumulator on, with the scales xr[0 .. n), wr[0 .. n).
// wait(i) waits for the i-th accumulator (false: it gave up), done(i) hands it back; taddr(i): its address.  32 columns
// at a time: while they are added, the next 32 are on their way, those of the next block too.
template <int HC, typename W, typename D, typename A>
__device__ __forceinline__ bool add_blocks(float (&acc)[HC], const float *xr, const float *wr, int n, int &it, W &&wait,
                                           D &&done, A &&taddr) {
    static_assert(HC % 64 == 0, "two register buffers in turn");
#pragma unroll
    for (int i = 0; i < HC; ++i) acc[i] = 0.f;
    uint32_t r0[32], r1[32];
    auto ready = [&](int i) {
        const bool ok = __all_sync(0xffffffffu, wait(i));
        tc_fence_after();
        return ok;
    };
    auto release = [&](int i) {
        tc_fence_before();
        __syncwarp();
        if ((threadIdx.x & 31) == 0) done(i);
    };
    float s = xr[0] * wr[0];
    if (!ready(it)) return false;
    tmem_ld_32x32b_x32(taddr(it), r0);
    for (int kb = 0; kb < n; ++kb, ++it) {
        const bool more = kb + 1 < n;
        const float sx = more ? xr[kb + 1] : 0.f, sw = more ? wr[kb + 1] : 0.f;
        bool ok = true;
#pragma unroll
        for (int c = 0; c < HC; c += 64) {
            tmem_wait_ld();
            tmem_ld_32x32b_x32(taddr(it) + c + 32, r1);
            add_scaled<HC>(acc, c, r0, s);
            tmem_wait_ld();
            if (c + 64 < HC) {
                tmem_ld_32x32b_x32(taddr(it) + c + 64, r0);
            } else {  // everything of this accumulator has been read
                release(it);
                if (more) {
                    ok = ready(it + 1);
                    if (ok) tmem_ld_32x32b_x32(taddr(it + 1), r0);
                }
            }
            add_scaled<HC>(acc, c + 32, r1, s);
        }
        if (!ok) return false;
        s = sx * sw;
    }
    return true;
}

// ---------------------------------------------------------------- many rows: persistent, 128 x 256 tiles
struct Tile {
    static constexpr int BN = 256, STAGES = 4, BUFS = 2;
    static constexpr uint32_t A_BYTES = PM * PK, B_BYTES = BN * PK, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr uint32_t OUT_BYTES = 8 * 32 * 128;  // each epilogue warp: 32 rows of 128 bytes
    static constexpr size_t SMEM = STAGES * STAGE_BYTES + OUT_BYTES + 1024 + 256;
};

template <typename OT>
__global__ void __launch_bounds__(PF_NT, 1)
proj_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                const __grid_constant__ CUtensorMap tmY, const float *__restrict__ xs, const float *__restrict__ ws,
                int M, int N, int K, OT *__restrict__ y, int tma_y, const YSize yz, unsigned int *timeouts) {
    pdl_trigger();
    pdl_wait();
    constexpr int ST = Tile::STAGES, NB = Tile::BUFS, BN = Tile::BN, HC = BN / 2;  // HC: columns per epilogue warp
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = smraw + ((1024u - (static_cast<uint32_t>(__cvta_generic_to_shared(smraw)) & 1023u)) & 1023u);
    uint8_t *sA = sm, *sB = sm + ST * Tile::A_BYTES, *sY = sm + ST * Tile::STAGE_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(sY + Tile::OUT_BYTES);
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
                    mbar_arrive_expect_tx(&full[s], Tile::STAGE_BYTES);
                    tma_load_2d(sA + s * Tile::A_BYTES, &tmA, &full[s], kb * PK, m0);
                    tma_load_2d(sB + s * Tile::B_BYTES, &tmB, &full[s], kb * PK, n0);
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
                    const uint64_t ad = smem_desc(smem_u32(sA + s * Tile::A_BYTES), 16, 1024, LAYOUT_SW128);
                    const uint64_t bd = smem_desc(smem_u32(sB + s * Tile::B_BYTES), 16, 1024, LAYOUT_SW128);
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
        for (int t = blockIdx.x; t < tiles; t += gridDim.x) {
            int m0, n0;
            tile_mn(t, m0, n0);
            const int row = m0 + 32 * q + lane, c0 = n0 + half * HC;
            float acc[HC];
            if (!add_blocks<HC>(
                    acc, xs + (int64_t)min(row, M - 1) * KB, ws + (int64_t)(min(c0, N - 1) / PK) * KB, KB, it,
                    [&](int i) { return mbar_wait(&acc_full[i % NB], (i / NB) & 1); },
                    [&](int i) { mbar_arrive(&acc_empty[i % NB]); },
                    [&](int i) { return tmem + lane_base + (uint32_t)((i % NB) * BN + half * HC); })) {
                timed_out = true;
                break;
            }
            // the warp's 32 rows, 128 bytes of columns at a time, through shared memory in the swizzle of the store's
            // map: the 16-byte chunk of a row is xored with the row's place in the swizzle's period of 8
            constexpr int PER = 128 / (int)sizeof(OT), E = 16 / (int)sizeof(OT);
#pragma unroll
            for (int c = 0; c < HC; c += PER) {
                if (lane == 0) bulk_wait_read_all();  // the store that used the buffer has read it
                __syncwarp();
#pragma unroll
                for (int g = 0; g < 8; ++g) {
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
                    *reinterpret_cast<uint4 *>(out + lane * 128 + ((g ^ (lane & 7)) << 4)) =
                        make_uint4(pv[0], pv[1], pv[2], pv[3]);
                }
                if (tma_y) {
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0 && m0 + 32 * q < M && c0 + c < N) {
                        tma_store_2d(&tmY, out, c0 + c, m0 + 32 * q);
                        bulk_commit();
                    }
                } else {  // rows of y that do not start on 16 bytes: row by row, neighbouring lanes neighbouring columns
                    __syncwarp();
                    const OT *buf = reinterpret_cast<const OT *>(out);
                    for (int r = 0; r < 32 && m0 + 32 * q + r < M; ++r) {
                        OT *dst = y + (int64_t)(m0 + 32 * q + r) * N + c0 + c;
#pragma unroll
                        for (int i = 0; i < PER; i += 32) {
                            const int j = lane + i;
                            if (c0 + c + j < N && in_bounds(dst + j, sizeof(OT), y, yz.n, yz.bounds))
                                dst[j] = buf[r * PER + (((j / E) ^ (r & 7)) * E + j % E)];
                        }
                    }
                    __syncwarp();
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

// ---------------------------------------------------------------- few rows: the blocks split over a cluster
struct Split {
    static constexpr int BN = 128, STAGES = 6, BUFS = 4;
    static constexpr uint32_t A_BYTES = PM * PK, B_BYTES = BN * PK, STAGE_BYTES = A_BYTES + B_BYTES;
    static constexpr int LY = BN + 4;  // pitch of the CTA's sums, which take the place of the stages
    static constexpr size_t SMEM = STAGES * STAGE_BYTES + 1024 + 256;
    static_assert(sizeof(float) * PM * LY <= STAGES * STAGE_BYTES, "the sums fit");
};

// One 128 x 128 tile per cluster of `parts` CTAs (blockIdx.x = tile * parts + rank); CTA r takes the blocks
// [r KB / parts, (r + 1) KB / parts), and then a share of the tile's rows to add up and store.
template <typename OT>
__global__ void __launch_bounds__(PF_NT, 1)
proj_fp8_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const float *__restrict__ xs, const float *__restrict__ ws, int M, int N, int K, int parts,
                      OT *__restrict__ y, int vec_y, const YSize yz, unsigned int *timeouts) {
    pdl_trigger();
    pdl_wait();
    constexpr int ST = Split::STAGES, NB = Split::BUFS, BN = Split::BN, HC = BN / 2, LY = Split::LY;
    extern __shared__ uint8_t smraw[];
    uint8_t *sm = smraw + ((1024u - (static_cast<uint32_t>(__cvta_generic_to_shared(smraw)) & 1023u)) & 1023u);
    uint8_t *sA = sm, *sB = sm + ST * Split::A_BYTES;
    uint64_t *full = reinterpret_cast<uint64_t *>(sm + ST * Split::STAGE_BYTES);
    uint64_t *empty = full + ST;
    uint64_t *acc_full = empty + ST;      // [NB] MMA -> epilogue
    uint64_t *acc_empty = acc_full + NB;  // [NB] epilogue -> MMA
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + NB);
    float *sY = reinterpret_cast<float *>(sm);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank(), tile = blockIdx.x / parts;
    const int tiles_m = (M + PM - 1) / PM, m0 = tile % tiles_m * PM, n0 = tile / tiles_m * BN;
    const int KB = (K + PK - 1) / PK;
    const int kb0 = (int)((int64_t)KB * rank / parts), kn = (int)((int64_t)KB * (rank + 1) / parts) - kb0;
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

    if (warp == 0 && lane == 0) {
        int it = 0;
        for (; it < kn; ++it) {
            const int s = it % ST;
            if (it >= ST && !mbar_wait(&empty[s], ((it / ST) - 1) & 1)) {
                timed_out = true;
                break;
            }
            mbar_arrive_expect_tx(&full[s], Split::STAGE_BYTES);
            tma_load_2d(sA + s * Split::A_BYTES, &tmA, &full[s], (kb0 + it) * PK, m0);
            tma_load_2d(sB + s * Split::B_BYTES, &tmB, &full[s], (kb0 + it) * PK, n0);
        }
        if (timed_out)  // let the copies already issued land before the CTA can exit
            for (int j = (it > ST ? it - ST : 0); j < it; ++j) mbar_wait(&full[j % ST], (j / ST) & 1);
    } else if (warp == 1 && lane == 0) {
        constexpr uint32_t idesc = idesc_e4m3(PM, BN);
        for (int it = 0; it < kn; ++it) {
            const int s = it % ST, buf = it % NB;
            // the accumulator was read (NB blocks ago), and the operands are there
            if ((it >= NB && !mbar_wait(&acc_empty[buf], ((it / NB) - 1) & 1)) || !mbar_wait(&full[s], (it / ST) & 1)) {
                timed_out = true;
                break;
            }
            tc_fence_after();
            const uint64_t ad = smem_desc(smem_u32(sA + s * Split::A_BYTES), 16, 1024, LAYOUT_SW128);
            const uint64_t bd = smem_desc(smem_u32(sB + s * Split::B_BYTES), 16, 1024, LAYOUT_SW128);
#pragma unroll
            for (int k = 0; k < PK / 32; ++k)
                mma_f8_ss(tmem + buf * BN, ad + (uint64_t)(k * 2), bd + (uint64_t)(k * 2), idesc, k != 0);
            mma_commit(&acc_full[buf]);
            mma_commit(&empty[s]);
        }
    } else if (warp >= 4) {
        const int q = warp & 3, half = (warp - 4) >> 2;  // lane quarter (fixed by the warp), column half
        const uint32_t lane_base = (uint32_t)(32 * q) << 16;
        const int r = 32 * q + lane;
        float acc[HC];
        int it = 0;
        if (!add_blocks<HC>(
                acc, xs + (int64_t)min(m0 + r, M - 1) * KB + kb0, ws + (int64_t)(n0 / PK) * KB + kb0, kn, it,
                [&](int i) { return mbar_wait(&acc_full[i % NB], (i / NB) & 1); },
                [&](int i) { mbar_arrive(&acc_empty[i % NB]); },
                [&](int i) { return tmem + lane_base + (uint32_t)((i % NB) * BN + half * HC); }))
            timed_out = true;
        // every product of the CTA has been taken from the stages by now
#pragma unroll
        for (int c = 0; c < HC; c += 4)
            *reinterpret_cast<float4 *>(sY + r * LY + half * HC + c) = make_float4(acc[c], acc[c + 1], acc[c + 2], acc[c + 3]);
    }
    if (timed_out && timeouts) atomicAdd(timeouts, 1u);
    __syncwarp();
    tc_fence_before();
    cluster_sync();  // every CTA's sums are there
    if (warp == 0) tmem_dealloc(tmem, 512);
    const int col = n0 + 4 * lane;
    for (int r = rank + parts * warp; r < PM && m0 + r < M; r += parts * (PF_NT / 32)) {
        float4 t = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i = 0; i < parts; ++i) {
            float4 v;
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                         : "r"(cluster_addr(sY + r * LY + 4 * lane, (uint32_t)i)));
            t.x += v.x;
            t.y += v.y;
            t.z += v.z;
            t.w += v.w;
        }
        OT *dst = y + (int64_t)(m0 + r) * N + col;
        if (!vec_y || col + 4 > N) {
            const float f[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (col + i < N && in_bounds(dst + i, sizeof(OT), y, yz.n, yz.bounds)) store_elem(dst, i, f[i]);
        } else if (in_bounds(dst, 4 * sizeof(OT), y, yz.n, yz.bounds)) {
            if (sizeof(OT) == 4) {
                *reinterpret_cast<float4 *>(dst) = t;
            } else {
                const __nv_bfloat162 a = __floats2bfloat162_rn(t.x, t.y), b = __floats2bfloat162_rn(t.z, t.w);
                *reinterpret_cast<uint2 *>(dst) =
                    make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
            }
        }
    }
    cluster_sync();  // no CTA leaves while another reads its sums
}

// ---------------------------------------------------------------- any K, any alignment
// 64 x 64 output tiles, 16 channels at a time, exact fp32.
template <typename OT>
__global__ void __launch_bounds__(256) proj_fp8_simt_kernel(const uint8_t *__restrict__ x, const float *__restrict__ xs,
                                                            const uint8_t *__restrict__ w, const float *__restrict__ ws,
                                                            int64_t M, int N, int K, OT *__restrict__ y, const YSize yz) {
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
            if (r < M && c < N && in_bounds(y + r * N + c, sizeof(OT), y, yz.n, yz.bounds))
                store_elem(y, r * N + c, acc[i][j]);
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

// launch_pdl for clusters of CTAs
template <typename... KArgs, typename... Args>
cudaError_t launch_cluster(void (*kernel)(KArgs...), unsigned grid, unsigned cluster, size_t smem, cudaStream_t st,
                           Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(PF_NT);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

kda_status_t map_bytes(CUtensorMap *m, const void *base, int64_t rows, int K, uint32_t box) {  // boxes of box x 128 bytes
    return make_tmap_2d(m, base, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, (uint64_t)rows, (uint64_t)K, (uint64_t)K, box, PK,
                        CU_TENSOR_MAP_SWIZZLE_128B);
}

template <typename OT>
kda_status_t launch_proj_fp8(const P8Args &a, cudaStream_t st) {
    // whole 16-byte vectors in the rows of x and W, and aligned bases: what the TMA maps ask for
    const YSize yz = {checked_size((size_t)a.N * a.M * sizeof(OT)), checked_counter()};
    const bool tc = a.K % 16 == 0 && aligned_to(a.x, 16) && aligned_to(a.w, 16);
    if (!tc) {
        const int64_t ctas = ((a.N + 63) / 64) * ((a.M + 63) / 64);
        const cudaError_t e = launch_pdl(proj_fp8_simt_kernel<OT>, dim3((unsigned)ctas), dim3(256), 0, st,
                                         (const uint8_t *)a.x, a.xs, (const uint8_t *)a.w, a.ws, a.N, a.M, a.K, (OT *)a.y, yz);
        if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "proj_fp8_simt_kernel: %s", cudaGetErrorString(e));
        return check_launch("proj_fp8_simt_kernel");
    }
    int dev = 0, sms = 148;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    CUtensorMap ta, tb, ty;
    KDA_TRY(map_bytes(&ta, a.x, a.N, a.K, PM));
    const int64_t tiles = ((a.N + PM - 1) / PM) * ((a.M + Split::BN - 1) / Split::BN);
    if (tiles <= sms) {
        KDA_TRY(map_bytes(&tb, a.w, a.M, a.K, Split::BN));
        // 128 x 128 tiles do not fill the GPU: as many CTAs per tile as do, with four blocks of the sum each at least
        const int KB = (a.K + PK - 1) / PK;
        int parts = 1;
        while (parts < 8 && tiles * parts * 2 <= sms && KB >= 8 * parts) parts *= 2;
        const cudaError_t e = launch_cluster(proj_fp8_split_kernel<OT>, (unsigned)(tiles * parts), (unsigned)parts, Split::SMEM,
                                             st, ta, tb, a.xs, a.ws, (int)a.N, a.M, a.K, parts, (OT *)a.y,
                                             (int)(a.M % 4 == 0 && aligned_to(a.y, 4 * sizeof(OT))), yz,
                                             device_timeout_counter());
        if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "proj_fp8_split_kernel: %s", cudaGetErrorString(e));
        return check_launch("proj_fp8_split_kernel");
    }
    KDA_TRY(map_bytes(&tb, a.w, a.M, a.K, Tile::BN));
    const int tma_y = a.M % (16 / (int)sizeof(OT)) == 0 && aligned_to(a.y, 16);
    if (tma_y)
        KDA_TRY(make_tmap_2d(&ty, a.y, sizeof(OT) == 2 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32,
                             (int)sizeof(OT), (uint64_t)a.N, (uint64_t)a.M, (uint64_t)a.M, 32, 128 / sizeof(OT),
                             CU_TENSOR_MAP_SWIZZLE_128B));
    else
        ty = ta;  // (not read)
    const int64_t big = ((a.N + PM - 1) / PM) * ((a.M + Tile::BN - 1) / Tile::BN);
    cudaFuncSetAttribute(proj_fp8_kernel<OT>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Tile::SMEM);
    const cudaError_t e = launch_pdl(proj_fp8_kernel<OT>, dim3((unsigned)(big < sms ? big : sms)), dim3(PF_NT), Tile::SMEM, st,
                                     ta, tb, ty, a.xs, a.ws, (int)a.N, a.M, a.K, (OT *)a.y, tma_y, yz,
                                     device_timeout_counter());
    if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "proj_fp8_kernel: %s", cudaGetErrorString(e));
    return check_launch("proj_fp8_kernel");
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
