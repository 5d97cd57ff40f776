// Products of shared-memory tiles to fp32 accuracy on the tensor cores, for the per-chunk algebra of the
// gated delta rule's gradients: warp-level mma.m16n8k8 with tf32 operands.
//
// A tf32 operand has 11 significant bits.  An fp32 value x is split into hi = x rounded to tf32 and
// lo = x - hi (exact), and a product becomes hi hi' + hi lo' + lo hi': what is left out is below 2^-21 of
// the product.  An operand that tf32 holds exactly (bf16 values) has no lo, and its products are one (both
// exact) or two instructions.  Accumulation is fp32.  Measured: 8 clocks an instruction on a sub-partition (288 TFLOP/s
// on 148 SMs at 1.9 GHz), 9 to 12 in the loops below, where splitting and the reads from shared memory take issue slots.
#pragma once

#include "kda_internal.cuh"

namespace kda {
namespace tf32 {

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// x = hi + lo, hi rounded to the nearest tf32 (the carry of the added half step goes into the exponent)
__device__ __forceinline__ void split(float x, uint32_t &hi, uint32_t &lo) {
    hi = (__float_as_uint(x) + 0x1000u) & 0xffffe000u;
    lo = __float_as_uint(x - __uint_as_float(hi));
}

__device__ __forceinline__ void load2(const float *p, float &x, float &y) {
    const float2 t = *reinterpret_cast<const float2 *>(p);
    x = t.x;
    y = t.y;
}
__device__ __forceinline__ void load2(const __nv_bfloat16 *p, float &x, float &y) {
    const uint32_t t = *reinterpret_cast<const uint32_t *>(p);
    x = __uint_as_float(t << 16);
    y = __uint_as_float(t & 0xffff0000u);
}

// Neighbouring bf16 rows k = 2t, 2t + 1 of column g of an 8 x 8 block, packed into one register per block; each lane
// gives the address of a row of 16 bytes (lanes 8b .. 8b + 7: block b).
__device__ __forceinline__ void ldsm_trans(uint32_t (&r)[1], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x1.trans.shared.b16 {%0}, [%1];" : "=r"(r[0]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_trans(uint32_t (&r)[2], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldsm_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// acc += A B^T over k < K (a multiple of 8; UNROLL steps of 8 at a time), for a warp's MT x 16 rows and NT x 8 columns:
// acc[i][j] holds (16i + g, 8j + 2t), (.., + 1), (16i + g + 8, ..), (.., + 1) with g = lane / 4, t = lane % 4.
//   A(m, k) = A[m * lda + k], or A[k * lda + m] with AT;  B(n, k) = B[n * ldb + k], or B[k * ldb + n] with BT.
// Operands are fp32 or bf16 (exact; read by k they come through ldmatrix, from rows on 16-byte boundaries).  AEX / BEX:
// tf32 holds the operand exactly.  The order of k within an instruction is free, as long as A and B share it: unless
// both are fp32 and read by k, a lane takes neighbouring k (one load where the operand is contiguous in k).
// Pitches of 8 mod 32 floats make the reads free of bank conflicts (fp32 read by k in pairs: two-way).
// The lo terms have accumulators of their own, so that the tensor core, which truncates as it adds, does so once per
// step of 8 on the large sums.  KS: B's rows k are multiplied by ks[k] as they are read.
template <int MT, int NT, bool AT, bool BT, bool AEX, bool BEX, int UNROLL = 2, bool KS = false, typename TA, typename TB>
__device__ __forceinline__ void tile(float (&acc)[MT][NT][4], const TA *A, int lda, const TB *B, int ldb,
                                     int K, const float *ks = nullptr) {
    constexpr bool A16 = sizeof(TA) == 2 && AT, B16 = sizeof(TB) == 2 && BT;
    constexpr bool PAIR = !(AT && BT) || A16 || B16;
    static_assert(!KS || (BT && !BEX), "a scaled operand is read by k, and is not exact");
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    float cross[MT][NT][4] = {};
    uint32_t arow = 0, brow = 0;  // this lane's row for ldmatrix: k = lane % 8, of block lane / 8
    if constexpr (A16)
        arow = (uint32_t)__cvta_generic_to_shared(A + (lane & 7) * lda + ((lane >> 3) & (2 * MT - 1)) * 8);
    if constexpr (B16) brow = (uint32_t)__cvta_generic_to_shared(B + (lane & 7) * ldb + ((lane >> 3) & (NT - 1)) * 8);
#pragma unroll UNROLL
    for (int k = 0; k < K; k += 8) {
        const int ka = PAIR ? k + 2 * t : k + t, kb = PAIR ? ka + 1 : ka + 4;
        uint32_t ah[MT][4], al[MT][4], bh[NT][2], bl[NT][2];
        float sc[2] = {1.f, 1.f};
        if constexpr (KS) {
            sc[0] = ks[ka];
            sc[1] = ks[kb];
        }
        if constexpr (A16) {
            uint32_t r[2 * MT];
            ldsm_trans(r, arow);
            arow += 16 * lda;
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                ah[i][0] = r[2 * i] << 16;
                ah[i][2] = r[2 * i] & 0xffff0000u;
                ah[i][1] = r[2 * i + 1] << 16;
                ah[i][3] = r[2 * i + 1] & 0xffff0000u;
            }
        } else {
#pragma unroll
            for (int i = 0; i < MT; ++i) {
                float x[4];
                if (AT) {
                    const TA *p = A + ka * lda + 16 * i + g, *q = A + kb * lda + 16 * i + g;
                    x[0] = load_elem(p, 0);
                    x[1] = load_elem(p, 8);
                    x[2] = load_elem(q, 0);
                    x[3] = load_elem(q, 8);
                } else {
                    load2(A + (16 * i + g) * lda + ka, x[0], x[2]);
                    load2(A + (16 * i + g + 8) * lda + ka, x[1], x[3]);
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (AEX) ah[i][e] = __float_as_uint(x[e]);
                    else split(x[e], ah[i][e], al[i][e]);
                }
            }
        }
        if constexpr (B16) {
            uint32_t r[NT];
            ldsm_trans(r, brow);
            brow += 16 * ldb;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                bh[j][0] = r[j] << 16;
                bh[j][1] = r[j] & 0xffff0000u;
                if constexpr (KS) {
                    split(__uint_as_float(bh[j][0]) * sc[0], bh[j][0], bl[j][0]);
                    split(__uint_as_float(bh[j][1]) * sc[1], bh[j][1], bl[j][1]);
                }
            }
        } else {
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float x[2];
                if (BT) {
                    x[0] = sc[0] * load_elem(B, ka * ldb + 8 * j + g);
                    x[1] = sc[1] * load_elem(B, kb * ldb + 8 * j + g);
                } else {
                    load2(B + (8 * j + g) * ldb + ka, x[0], x[1]);
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    if (BEX) bh[j][e] = __float_as_uint(x[e]);
                    else split(x[e], bh[j][e], bl[j][e]);
                }
            }
        }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                if (!BEX) mma(cross[i][j], ah[i], bl[j]);
                if (!AEX) mma(cross[i][j], al[i], bh[j]);
            }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j) mma(acc[i][j], ah[i], bh[j]);
    }
    if (!(AEX && BEX)) {
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] += cross[i][j][e];
    }
}

// Calls f(i, j, e, row, column) for every element of a warp's tile.
template <int MT, int NT, typename F>
__device__ __forceinline__ void each(F &&f) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) f(i, j, e, 16 * i + g + (e >> 1) * 8, 8 * j + 2 * t + (e & 1));
}

}  // namespace tf32
}  // namespace kda
