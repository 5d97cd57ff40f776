// Gradients of the gated delta rule (one scalar decay per token and head), chunk form, fp32 accuracy.
//
// Inside a chunk of C = 64 tokens, with G_r the cumulative log-decay, E[r,i] = e^{G_r - G_i} (i <= r) and
// e^{D_r} = e^{G_last - G_r}:
//   P[r,i] = (k_r . k_i) E[r,i] (i < r),   A = Diag(beta) P,   T = (I + A)^{-1}
//   Bk = Diag(beta e^G) K,  Bv = Diag(beta) V,  W = T Bk,  U = T Bv,  V' = U - W S
//   M[r,i] = (q_r . k_i) E[r,i] (i <= r),   O = Diag(e^G) Q S + M V',
//   S_next = gamma S + K^T Diag(e^D) V',  gamma = e^{G_last}
// (S: the state entering the chunk), and in reverse, with dS_next the gradient of the state leaving it:
//   dV' = M^T dO + Diag(e^D) K dS_next
//   dS  = gamma dS_next + Q^T Diag(e^G) dO - W^T dV'
//   dQg = dO S^T,  dKd = V' dS_next^T,  dM = dO V'^T (i <= r),  dW = -dV' S^T
//   dT  = dV' Bv^T + dW Bk^T,  dBv = T^T dV',  dBk = T^T dW,  dA = -T^T dT T^T (i < r)
//   dv = beta dBv,   dq = e^G dQg + (dM * E) K
//   dk = beta e^G dBk + e^D dKd + (dP' + dP'^T) K + (dM * E)^T Q,   dP' = Diag(beta) dA * E
//   dbeta = rowsum(dBv * V) + rowsum(dBk * e^G K) + rowsum(dA * P)
// Because the decay is one number per token, its gradient needs no difference of large sums: log alpha_t is a
// factor of every pair (r, i) with i < t <= r, of the rows r >= t of Q e^G and Bk, of the rows i < t of
// K e^D, and of gamma:
//   dlog alpha_t = sum_{r >= t > i} (dA * A + dM * M)[r,i] + sum_{r >= t} (dQg . Qg + dBk . Bk)_r
//                  + sum_{i < t} (dKd . Kd)_i + gamma <dS_next, S>.
// G is cumulated and differenced in fp64: in-chunk sums reach 64 |g_min|, where the fp32 difference of two
// neighbours would be off by 1e-5.  No factor e^{-G} is ever formed, so any g_min works.
//
// Three launches: gb_prep (a CTA per chunk: P, M, T, W, U, and the terms M^T dO and Q^T (e^G dO) that dV' and dS have
// of the chunk itself, into a workspace record), gb_chain (a CTA per (b, h, 16 value columns) and direction: the state
// forward, which leaves S and V' of every chunk, and at the same time its gradient backward, which leaves dS_next and
// dV': the two do not depend on each other), and gb_grad (a CTA per chunk: everything else).  All products run on the
// tensor cores to fp32 accuracy (mma_tf32.cuh); bf16 inputs are exact operands there and cost a third less, which is
// why the scale factors of K and Q rows are applied to the other operand or to the result.
//
// Measured (4096 tokens, 16 heads of 128, bf16): 103 + 228 + 326 = 660 us with the launches.  The bytes that a call
// cannot do without take 26 us; the 28 GFLOP, two or three times over for the split operands, about 250 us at the rate of
// the warp-level tf32 product (8 clocks each on a sub-partition), which is what bounds it: the tensor pipe is busy a
// third to a half of the time, the rest is splitting operands, reading them from shared memory and the row algebra
// around them.  A chain step (64 tokens) takes 3.6 us with two CTAs on the SM, 2.3 us alone.
#include "host_check.cuh"
#include "kda_internal.cuh"
#include "mma_tf32.cuh"

namespace kda {

namespace {

constexpr int C = 64;       // tokens per chunk
constexpr int LD = 136;     // pitch of [64 or 128][D] tiles in shared memory: 8 mod 32
constexpr int LC = 72;      // pitch of [64][64] tiles
constexpr int NT_P = 512;   // threads of the gradient kernel
constexpr int NT_C = 256;   // threads of the chain kernel
constexpr int VS = 16;      // value columns per chain CTA
constexpr int LO = 20;      // chain pitch of [.][16] tiles read in pairs of k, and
constexpr int LV = 24;      // of those read by single k: rows (pairs of rows) 8 banks apart

__host__ __device__ inline int pad16(int x) { return (x + 15) & ~15; }
__host__ __device__ inline int pad32(int x) { return (x + 31) & ~31; }

// One (b, h, chunk) record; offsets in floats, all blocks whole 64-byte rows.  D_k is padded to a
// multiple of 16, D_v to one of 32; the padding holds zeros.
struct Rec {
    int64_t G;          // [64] double
    int64_t eG, eD;     // [64] e^G, e^{G_last - G}
    int64_t T, P, M;    // [64][64]
    int64_t W;          // [64][Dkp]
    int64_t V;          // [64][Dvp]: U, then V'
    int64_t S;          // [Dkp][Dvp]: the state entering the chunk
    int64_t dS;         // [Dkp][Dvp]: Q^T (e^G dO), then the gradient of the state leaving the chunk
    int64_t dV;         // [64][Dvp]: M^T dO, then dV'
    int64_t size;
};

__host__ __device__ inline Rec make_rec(int Dk, int Dv) {
    const int64_t dk = pad16(Dk), dv = pad32(Dv);
    Rec r;
    r.G = 0;
    r.eG = 2 * C;
    r.eD = r.eG + C;
    r.T = r.eD + C;
    r.P = r.T + C * C;
    r.M = r.P + C * C;
    r.W = r.M + C * C;
    r.V = r.W + C * dk;
    r.S = r.V + C * dv;
    r.dS = r.S + dk * dv;
    r.dV = r.dS + dk * dv;
    r.size = r.dV + C * dv;
    return r;
}

struct GbArgs {
    int64_t S;
    int H, Dk, Dv, Nc, nslice;
    bool wide_k, wide_v;  // 16-byte vectors in the token rows of q and k, of v and dO
    bool pair_k, pair_v;  // 8-byte pairs in the rows of dq and dk, of dv
    const void *q, *k, *v, *z, *beta, *dO;
    const float *log_decay;
    float g_min;
    const float *S0, *dST;
    float *dq, *dk, *dv, *dbeta, *dz, *dS0;
    float *ws;
    size_t ws_bytes, ns_bytes, nk_bytes, nv_bytes, nb_bytes;  // ns: dS0; nk: dq, dk; nv: dv; nb: dbeta, dz
    unsigned int *bounds;
};

struct Unit {
    int64_t b, t0, row0;  // row0: index of (token t0, head h) in a (B, S, H) tensor
    int h, len;
};

__device__ __forceinline__ Unit unit_of(const GbArgs &p, int64_t bh, int n) {
    Unit u;
    u.b = bh / p.H;
    u.h = (int)(bh - u.b * p.H);
    u.t0 = (int64_t)n * C;
    u.len = (int)min((int64_t)C, p.S - u.t0);
    u.row0 = (u.b * p.S + u.t0) * p.H + u.h;
    return u;
}

// Staging by NT threads, tid of them.  Token rows (rs elements apart), in their type, into [64][LD]: zero past `len`
// rows and D columns up to Dp.  wide: D is
// a multiple of a 16-byte vector and every row starts on 16 bytes; the copies are asynchronous then.
template <typename T, int NT>
__device__ __forceinline__ void stage_rows(T *dst, const T *src, int64_t rs, int len, int D, int Dp, bool wide,
                                           int tid = threadIdx.x) {
    if (wide) {
        constexpr int E = 16 / (int)sizeof(T), VPR = 128 / E;
#pragma unroll
        for (int i = tid; i < C * VPR; i += NT) {
            const int r = i / VPR, c = i % VPR * E;
            const bool in = r < len && c < D;
            if (c < Dp)
                cp_async16_fill(reinterpret_cast<float *>(dst + r * LD + c),
                                reinterpret_cast<const float *>(src + (in ? r * rs + c : 0)), in);
        }
        return;
    }
    const int c = tid & 127;
    if (c < Dp)
#pragma unroll 4
        for (int r = tid >> 7; r < C; r += NT / 128)
            dst[r * LD + c] = (r < len && c < D) ? src[r * rs + c] : T(0.f);
}

// A record block of `rows` rows of `cols` floats (a multiple of 4, at most 4 VPR; pitch `pitch`) into shared memory.
template <int NT, int VPR>
__device__ __forceinline__ void stage_block(float *dst, int ld, const float *src, int pitch, int rows, int cols,
                                            int tid = threadIdx.x) {
#pragma unroll 4
    for (int i = tid; i < rows * VPR; i += NT) {
        const int r = i / VPR, c = i % VPR * 4;
        if (c < cols) cp_async16_fill(dst + r * ld + c, src + (int64_t)r * pitch + c);
    }
}

// Neighbouring columns c (even) and c + 1 of a token row: zero outside.
template <typename T>
__device__ __forceinline__ float2 row_pair(const T *row, int c, int D, bool in, bool wide) {
    float2 v = make_float2(0.f, 0.f);
    if (in && c < D) {
        if (wide) {
            tf32::load2(row + c, v.x, v.y);
        } else {
            v.x = load_elem(row, c);
            if (c + 1 < D) v.y = load_elem(row, c + 1);
        }
    }
    return v;
}

// Columns c (even) and c + 1 of the row at `at` of an output of `bytes`.
__device__ __forceinline__ void store_pair(float *out, size_t bytes, unsigned int *errors, int64_t at, int c, int D, bool in,
                                           bool pair, float x, float y) {
    if (!in || c >= D) return;
    float *row = out + at;
    if (!in_bounds(row + c, c + 1 < D ? 8 : 4, out, bytes, errors)) return;
    if (pair) {
        *reinterpret_cast<float2 *>(row + c) = make_float2(x, y);
    } else {
        row[c] = x;
        if (c + 1 < D) row[c + 1] = y;
    }
}

// A warp's 32 rows of a 64-row result; its columns are tile warp / 2.  Triangular operands give the two halves of the
// rows sums of different lengths: the four warps of an SM sub-partition (equal warp % 4), which share a tensor core, get
// both (the gradient kernel 335 -> 323 us on prefill_4k).
__device__ __forceinline__ int row_half(int warp) { return 32 * ((warp ^ (warp >> 2)) & 1); }

// ---------------------------------------------------------------- per chunk: P, M, T, W, U, M^T dO, Q^T (e^G dO)
// bf16 inputs: two CTAs of 8 warps on an SM, so that one's products run through the other's loads and inverse.  That
// needs 106 KB a CTA: M gives its place to T once M^T dO is formed, Q to V.  fp32 ones: one CTA of 16 warps.
template <typename T> constexpr int prep_nt() { return sizeof(T) == 2 ? 256 : 512; }
template <typename T> constexpr size_t prep_smem() {
    return sizeof(double) * C + sizeof(float) * (3 * C * LC + 2 * C) + 3 * sizeof(T) * C * LD;
}

template <typename T>
__global__ void __launch_bounds__(prep_nt<T>(), 512 / prep_nt<T>()) gb_prep_kernel(const __grid_constant__ GbArgs p) {
    constexpr bool EX = sizeof(T) == 2;
    constexpr int NT = prep_nt<T>(), NW = NT / 32;
    extern __shared__ __align__(16) uint8_t gb_sm[];
    double *sG = reinterpret_cast<double *>(gb_sm);
    float *sA = reinterpret_cast<float *>(sG + C), *sM = sA + C * LC, *sT = sM, *sY = sM + C * LC;
    float *sb = sY + C * LC, *seG = sb + C;
    T *sK = reinterpret_cast<T *>(seG + C), *sQ = sK + C * LD, *sV = sQ, *sO = sQ + C * LD;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t bh = blockIdx.x / p.Nc;
    const int n = (int)(blockIdx.x - bh * p.Nc);
    const Unit u = unit_of(p, bh, n);
    const int Dkp = pad16(p.Dk), Dvp = pad32(p.Dv);
    const Rec R = make_rec(p.Dk, p.Dv);
    float *rec = p.ws + (int64_t)blockIdx.x * R.size;
    if (!in_bounds(rec, (size_t)R.size * 4, p.ws, p.ws_bytes, p.bounds)) return;

    const int64_t rk = (int64_t)p.H * p.Dk, rv = (int64_t)p.H * p.Dv;
    stage_rows<T, NT>(sK, (const T *)p.k + u.row0 * p.Dk, rk, u.len, p.Dk, Dkp, p.wide_k);
    stage_rows<T, NT>(sQ, (const T *)p.q + u.row0 * p.Dk, rk, u.len, p.Dk, Dkp, p.wide_k);
    cp_async_commit_group();
    stage_rows<T, NT>(sO, (const T *)p.dO + u.row0 * p.Dv, rv, u.len, p.Dv, Dvp, p.wide_v);
    cp_async_commit_group();
    if (warp == 0) {  // the cumulative log-decay: two tokens per lane, a scan over the warp
        double g[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 2 * lane + e;
            float x = 0.f;
            if (r < u.len) {
                const int64_t i = u.row0 + (int64_t)r * p.H;
                x = p.log_decay ? clamp_log_decay(p.log_decay[i], p.g_min)
                                : log_alpha_of(load_elem((const T *)p.z, i), p.g_min);
            }
            g[e] = (double)x;
            sb[r] = r < u.len ? load_elem((const T *)p.beta, u.row0 + (int64_t)r * p.H) : 0.f;
        }
        double s = g[0] + g[1];
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const double o = __shfl_up_sync(0xffffffffu, s, m);
            if (lane >= m) s += o;
        }
        const double last = __shfl_sync(0xffffffffu, s, 31);
        const double G1 = s, G0 = s - g[1];
        sG[2 * lane] = G0;
        sG[2 * lane + 1] = G1;
        double *gG = reinterpret_cast<double *>(rec + R.G);
        gG[2 * lane] = G0;
        gG[2 * lane + 1] = G1;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 2 * lane + e;
            const float a = expf((float)(e ? G1 : G0)), d = expf((float)(last - (e ? G1 : G0)));
            seG[r] = a;
            rec[R.eG + r] = a;
            rec[R.eD + r] = d;
        }
    }
    cp_async_wait<1>();  // k and q
    __syncthreads();
    // P and M: warp (32 rows, 8 or 16 columns); tiles above the diagonal are zeros
    {
        constexpr int NC = 16 / NW;
        const int r0 = row_half(warp), c0 = 8 * NC * (warp >> 1);
        float kk[2][NC][4] = {}, qk[2][NC][4] = {};
        if (c0 < r0 + 32) {
            tf32::tile<2, NC, false, false, EX, EX>(kk, sK + r0 * LD, LD, sK + c0 * LD, LD, Dkp);
            tf32::tile<2, NC, false, false, EX, EX>(qk, sQ + r0 * LD, LD, sK + c0 * LD, LD, Dkp);
        }
        tf32::each<2, NC>([&](int i, int j, int e, int r, int c) {
            r += r0;
            c += c0;
            const float x = c <= r ? expf((float)(sG[r] - sG[c])) : 0.f;
            kk[i][j][e] = c < r ? kk[i][j][e] * x : 0.f;
            qk[i][j][e] = c <= r ? qk[i][j][e] * x : 0.f;
            sA[r * LC + c] = sb[r] * kk[i][j][e];
            sM[r * LC + c] = qk[i][j][e];
            if (e & 1) {
                *reinterpret_cast<float2 *>(rec + R.P + r * C + c - 1) = make_float2(kk[i][j][e - 1], kk[i][j][e]);
                *reinterpret_cast<float2 *>(rec + R.M + r * C + c - 1) = make_float2(qk[i][j][e - 1], qk[i][j][e]);
            }
        });
    }
    cp_async_wait<0>();  // dO
    __syncthreads();
    // 32 rows and 16 or 32 columns of a [64][D] result per warp
    constexpr int NC = 32 / NW;
    const int r0 = row_half(warp), c0 = 8 * NC * (warp >> 1);
    auto put = [&](float *dst, int pitch, const float (&acc)[2][NC][4]) {
        tf32::each<2, NC>([&](int i, int j, int e, int r, int c) {
            if (!(e & 1) && c0 + c < pitch)
                *reinterpret_cast<float2 *>(dst + (r0 + r) * pitch + c0 + c) = make_float2(acc[i][j][e], acc[i][j][e + 1]);
        });
    };
    if (c0 < Dvp) {  // M^T dO: what dV' has of the chunk itself
        float o[2][NC][4] = {};
        tf32::tile<2, NC, true, true, false, EX>(o, sM + r0 + r0 * LC, LC, sO + c0 + r0 * LD, LD, C - r0);
        put(rec + R.dV, Dvp, o);
    }
    // Q^T (e^G dO): what dS has of the chunk itself, 32 x 32 of [Dk][Dv] at a time
    for (int t = warp; t < 16; t += NW) {
        const int m0 = 32 * (t & 3), n0 = 32 * (t >> 2);
        if (m0 >= Dkp || n0 >= Dvp) continue;
        float h[2][4][4] = {};
        tf32::tile<2, 4, true, true, EX, false, 2, true>(h, sQ + m0, LD, sO + n0, LD, C, seG);
        tf32::each<2, 4>([&](int i, int j, int e, int r, int c) {
            if (!(e & 1) && m0 + r < Dkp)
                *reinterpret_cast<float2 *>(rec + R.dS + (m0 + r) * Dvp + n0 + c) = make_float2(h[i][j][e], h[i][j][e + 1]);
        });
    }
    __syncthreads();  // M and Q have been read
    stage_rows<T, NT>(sV, (const T *)p.v + u.row0 * p.Dv, rv, u.len, p.Dv, Dvp, p.wide_v);
    cp_async_commit_group();
    // T = (I + A)^{-1}: the four diagonal blocks of 16 by forward substitution (a thread per column) ...
    if (warp < 4 && lane < 16) {
        const float *a = sA + 16 * warp * (LC + 1);
        float x[16];
#pragma unroll
        for (int r = 0; r < 16; ++r) {
            float s = r == lane ? 1.f : 0.f;
#pragma unroll
            for (int m = 0; m < r; ++m) s = fmaf(-a[r * LC + m], x[m], s);
            x[r] = s;
        }
#pragma unroll
        for (int r = 0; r < 16; ++r) sT[(16 * warp + r) * LC + 16 * warp + lane] = x[r];
    }
    for (int i = tid; i < C * C; i += NT) {  // (the blocks above them are zeros)
        const int r = i >> 6, c = i & 63;
        if ((r >> 4) < (c >> 4)) sT[r * LC + c] = 0.f;
    }
    __syncthreads();
    // ... then T21 = -T22 (A21 T11), blocks of 16 and of 32
#pragma unroll
    for (int i = tid; i < 512; i += NT) {
        const int b0 = 32 * (i >> 8), r = (i & 255) >> 4, c = i & 15;
        float s = 0.f;
#pragma unroll
        for (int m = 0; m < 16; ++m) s = fmaf(sA[(b0 + 16 + r) * LC + b0 + m], sT[(b0 + m) * LC + b0 + c], s);
        sY[(b0 + r) * LC + c] = s;
    }
    __syncthreads();
#pragma unroll
    for (int i = tid; i < 512; i += NT) {
        const int b0 = 32 * (i >> 8), r = (i & 255) >> 4, c = i & 15;
        float s = 0.f;
#pragma unroll
        for (int m = 0; m < 16; ++m) s = fmaf(-sT[(b0 + 16 + r) * LC + b0 + 16 + m], sY[(b0 + m) * LC + c], s);
        sT[(b0 + 16 + r) * LC + b0 + c] = s;
    }
    __syncthreads();
    {
        constexpr int RW = 32 / NW;  // rows per thread
        float s[RW] = {};
        const int c = lane, r = warp;
#pragma unroll 8
        for (int m = 0; m < 32; ++m) {
            const float t = sT[m * LC + c];
#pragma unroll
            for (int e = 0; e < RW; ++e) s[e] = fmaf(sA[(32 + r + NW * e) * LC + m], t, s[e]);
        }
#pragma unroll
        for (int e = 0; e < RW; ++e) sY[(r + NW * e) * LC + c] = s[e];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < RW; ++e) s[e] = 0.f;
#pragma unroll 8
        for (int m = 0; m < 32; ++m) {
            const float y = sY[m * LC + c];
#pragma unroll
            for (int e = 0; e < RW; ++e) s[e] = fmaf(-sT[(32 + r + NW * e) * LC + 32 + m], y, s[e]);
        }
#pragma unroll
        for (int e = 0; e < RW; ++e) sT[(32 + r + NW * e) * LC + c] = s[e];
    }
    cp_async_wait<0>();  // v (made visible by the next barrier but one)
    __syncthreads();
    // T out; T Diag(beta e^G) over A, T Diag(beta) over the scratch: the scales of Bk's and Bv's rows
    for (int i = tid; i < C * C; i += NT) {
        const int r = i >> 6, c = i & 63;
        const float t = sT[r * LC + c], tb = t * sb[c];
        rec[R.T + i] = t;
        sA[r * LC + c] = tb * seG[c];
        sY[r * LC + c] = tb;
    }
    __syncthreads();
    if (c0 < Dkp) {
        float acc[2][NC][4] = {};
        tf32::tile<2, NC, false, true, false, EX>(acc, sA + r0 * LC, LC, sK + c0, LD, r0 + 32);
        put(rec + R.W, Dkp, acc);
    }
    if (c0 < Dvp) {
        float acc[2][NC][4] = {};
        tf32::tile<2, NC, false, true, false, EX>(acc, sY + r0 * LC, LC, sV + c0, LD, r0 + 32);
        put(rec + R.V, Dvp, acc);
    }
}

// ---------------------------------------------------------------- the state and its gradient through the chunks
// What a step reads of its chunk: e^G and e^D, W, K, U or M^T dO, and backwards Q^T (e^G dO).  A step is two products,
// one with W and one with K; each of the two is replaced by the next chunk's while the other is used.
template <typename T> struct Stage {
    float *e, *U, *W, *H;  // e and U: two sets
    T *K;
    float *sY, *sV, *sS;  // the other half of a sum, V' and S (or their gradients)
    __device__ explicit Stage(float *base) {
        e = base;
        U = e + 4 * C;
        W = U + 2 * C * LO;
        H = W + C * LD;
        sY = H + 128 * LO;
        sV = sY + C * LO;
        sS = sV + C * LV;
        K = reinterpret_cast<T *>(sS + 128 * LO);
    }
    static constexpr int FLOATS = 4 * C + 2 * C * LO + C * LD + 128 * LO + C * LO + C * LV + 128 * LO;
};
template <typename T> constexpr size_t chain_smem() { return Stage<T>::FLOATS * sizeof(float) + sizeof(T) * C * LD; }

// 8 warps: [64][16] results as 4 tiles of 16 x 16, the sum over k shared by two groups of warps; [Dk][16] ones as 8
// tiles.  The state, or its gradient, stays in the accumulators of the warps that own it.  Products have accumulators of
// their own: the tensor core truncates as it adds, the state is rounded once a chunk.
struct Chain {
    const float *rec0;  // the records of this (b, h)
    Rec R;
    int Dkp, Dvp, j0;
    int64_t row0, rk;   // token rows of the (b, h)
    int m0, r0, half;   // this warp's rows of a [Dk][16] and of a [64][16] result; its half of the sum over the key
    int kh, kn;         // channels: kn of them from kh
};

__device__ __forceinline__ Chain chain_of(const GbArgs &p, int64_t bh, int j0) {
    const int warp = threadIdx.x >> 5;
    Chain c;
    c.R = make_rec(p.Dk, p.Dv);
    c.rec0 = p.ws + bh * p.Nc * c.R.size;
    c.Dkp = pad16(p.Dk);
    c.Dvp = pad32(p.Dv);
    c.j0 = j0;
    const int64_t b = bh / p.H;
    c.row0 = b * p.S * p.H + (bh - b * p.H);
    c.rk = (int64_t)p.H * p.Dk;
    c.m0 = 16 * warp;
    c.r0 = 16 * (warp & 3);
    c.half = warp >> 2;
    const int mid = (c.Dkp / 2 + 7) & ~7;
    c.kh = c.half ? mid : 0;
    c.kn = c.half ? c.Dkp - mid : mid;
    return c;
}

// NT of the CTA's threads, t of them.
template <int NT, typename T>
__device__ __forceinline__ void stage_keys(const GbArgs &p, const Chain &c, T *sK, int n, int t) {
    const int64_t t0 = (int64_t)n * C;
    stage_rows<T, NT>(sK, (const T *)p.k + (c.row0 + t0 * p.H) * p.Dk, c.rk, (int)min((int64_t)C, p.S - t0), p.Dk, c.Dkp,
                      p.wide_k, t);
}

// V' = U - W S,  S <- gamma S + K^T (e^D V').  FULL: D_k pads to 128.
template <typename T, bool FULL>
__device__ __forceinline__ void chain_forward(const GbArgs &p, int64_t bh, int j0, float *sm) {
    constexpr bool EX = sizeof(T) == 2;
    constexpr int HT = NT_C / 2, lv = EX ? LO : LV;  // V' is read in pairs of k where K comes through ldmatrix
    const Stage<T> g(sm);
    const Chain q = chain_of(p, bh, j0);
    const Rec &R = q.R;
    const int m0 = q.m0, r0 = q.r0, Dkp = FULL ? 128 : q.Dkp, Dvp = q.Dvp;
    const bool own = FULL || m0 < Dkp, first = !q.half;
    const int ht = threadIdx.x & (HT - 1);
    auto stage = [&](const float *rec, int n) {  // W, U, e: by the second group of warps
        stage_block<HT, 32>(g.e + (n & 1) * 2 * C, 2 * C, rec + R.eG, 2 * C, 1, 2 * C, ht);
        stage_block<HT, 32>(g.W, LD, rec + R.W, Dkp, C, Dkp, ht);
        stage_block<HT, 4>(g.U + (n & 1) * C * LO, LO, rec + R.V + j0, Dvp, C, VS, ht);
    };
    float S[1][2][4] = {};
    tf32::each<1, 2>([&](int i, int j, int e, int r, int c) {
        r += m0;
        if (r < p.Dk && j0 + c < p.Dv && p.S0) S[i][j][e] = p.S0[(bh * p.Dk + r) * p.Dv + j0 + c];
        if (own) g.sS[r * LO + c] = S[i][j][e];
    });
    float *rec = const_cast<float *>(q.rec0);
    if (!first) stage(rec, 0);
    cp_async_commit_group();
    for (int n = 0; n < p.Nc; ++n, rec += R.size) {
        const float *e_ = g.e + (n & 1) * 2 * C, *U = g.U + (n & 1) * C * LO;
        cp_async_wait<0>();  // W
        __syncthreads();     // and S; the last chunk's K is read
        stage_keys<NT_C>(p, q, g.K, n, threadIdx.x);
        cp_async_commit_group();
        if (own)  // the state entering the chunk
            tf32::each<1, 2>([&](int i, int j, int e, int r, int c) {
                if (!(e & 1))
                    *reinterpret_cast<float2 *>(rec + R.S + (m0 + r) * Dvp + j0 + c) = make_float2(S[i][j][e], S[i][j][e + 1]);
            });
        float v[1][2][4] = {};
        tf32::tile<1, 2, false, true, false, false, 8>(v, g.W + r0 * LD + q.kh, LD, g.sS + q.kh * LO, LO, FULL ? C : q.kn);
        if (!first) tf32::each<1, 2>([&](int i, int j, int e, int r, int c) { g.sY[(r0 + r) * LO + c] = v[i][j][e]; });
        __syncthreads();  // the other half of the sum; W is read
        if (first)
            tf32::each<1, 2>([&](int i, int j, int e, int r, int c) {
                r += r0;
                v[i][j][e] = U[r * LO + c] - (v[i][j][e] + g.sY[r * LO + c]);
                if (e & 1) {
                    *reinterpret_cast<float2 *>(g.sV + r * lv + c - 1) =  // e^D V'
                        make_float2(e_[C + r] * v[i][j][e - 1], e_[C + r] * v[i][j][e]);
                    *reinterpret_cast<float2 *>(rec + R.V + r * Dvp + j0 + c - 1) = make_float2(v[i][j][e - 1], v[i][j][e]);
                }
            });
        else if (n + 1 < p.Nc)
            stage(rec + R.size, n + 1);
        cp_async_commit_group();
        cp_async_wait<1>();  // K
        __syncthreads();
        if (own) {
            const float gamma = e_[C - 1];
            float add[1][2][4] = {};
            tf32::tile<1, 2, true, true, EX, false, 8>(add, g.K + m0, LD, g.sV, lv, C);
            tf32::each<1, 2>([&](int i, int j, int e, int r, int c) {
                S[i][j][e] = fmaf(gamma, S[i][j][e], add[i][j][e]);
                if (e & 1) *reinterpret_cast<float2 *>(g.sS + (m0 + r) * LO + c - 1) = make_float2(S[i][j][e - 1], S[i][j][e]);
            });
        }
    }
}

// dV' = M^T dO + e^D (K dS),  dS <- gamma dS + Q^T (e^G dO) - W^T dV', from the last chunk to the first; the two terms
// with dO are in the record, where their results take their place.
template <typename T, bool FULL>
__device__ __forceinline__ void chain_backward(const GbArgs &p, int64_t bh, int j0, float *sm) {
    constexpr bool EX = sizeof(T) == 2;
    constexpr int HT = NT_C / 2;
    const Stage<T> g(sm);
    const Chain q = chain_of(p, bh, j0);
    const Rec &R = q.R;
    const int m0 = q.m0, r0 = q.r0, Dkp = FULL ? 128 : q.Dkp, Dvp = q.Dvp;
    const bool own = FULL || m0 < Dkp, first = !q.half;
    const int ht = threadIdx.x & (HT - 1);
    auto stage = [&](const float *rec, int n) {  // K, M^T dO, e: by the second group of warps
        stage_block<HT, 32>(g.e + (n & 1) * 2 * C, 2 * C, rec + R.eG, 2 * C, 1, 2 * C, ht);
        stage_keys<HT>(p, q, g.K, n, ht);
        stage_block<HT, 4>(g.U + (n & 1) * C * LO, LO, rec + R.dV + j0, Dvp, C, VS, ht);
    };
    float dS[1][2][4] = {};
    tf32::each<1, 2>([&](int i, int j, int e, int r, int c) {
        r += m0;
        if (r < p.Dk && j0 + c < p.Dv && p.dST) dS[i][j][e] = p.dST[(bh * p.Dk + r) * p.Dv + j0 + c];
        if (own) g.sS[r * LO + c] = dS[i][j][e];
    });
    float *rec = const_cast<float *>(q.rec0) + (int64_t)(p.Nc - 1) * R.size;
    if (!first) stage(rec, p.Nc - 1);
    cp_async_commit_group();
    for (int n = p.Nc - 1; n >= 0; --n, rec -= R.size) {
        const float *e_ = g.e + (n & 1) * 2 * C, *U = g.U + (n & 1) * C * LO;
        cp_async_wait<0>();  // K
        __syncthreads();     // and dS; the last chunk's W and H are read
        stage_block<NT_C, 32>(g.W, LD, rec + R.W, Dkp, C, Dkp);
        stage_block<NT_C, 4>(g.H, LO, rec + R.dS + j0, Dvp, Dkp, VS);
        cp_async_commit_group();
        float x[1][2][4] = {};
        tf32::tile<1, 2, false, true, EX, false, 8>(x, g.K + r0 * LD + q.kh, LD, g.sS + q.kh * LO, LO, FULL ? C : q.kn);
        if (!first) tf32::each<1, 2>([&](int i, int j, int e, int r, int c) { g.sY[(r0 + r) * LO + c] = x[i][j][e]; });
        __syncthreads();  // the other half of the sum; K is read
        if (first)
            tf32::each<1, 2>([&](int i, int j, int e, int r, int c) {
                r += r0;
                x[i][j][e] = fmaf(e_[C + r], x[i][j][e] + g.sY[r * LO + c], U[r * LO + c]);
                if (e & 1) {
                    *reinterpret_cast<float2 *>(g.sV + r * LV + c - 1) = make_float2(-x[i][j][e - 1], -x[i][j][e]);
                    *reinterpret_cast<float2 *>(rec + R.dV + r * Dvp + j0 + c - 1) = make_float2(x[i][j][e - 1], x[i][j][e]);
                }
            });
        else if (n > 0)
            stage(rec - R.size, n - 1);
        cp_async_commit_group();
        cp_async_wait<1>();  // W and H
        __syncthreads();
        if (own) {
            tf32::each<1, 2>([&](int i, int j, int e, int r, int c) {  // the gradient of the state leaving the chunk
                if (!(e & 1))
                    *reinterpret_cast<float2 *>(rec + R.dS + (m0 + r) * Dvp + j0 + c) = make_float2(dS[i][j][e], dS[i][j][e + 1]);
            });
            const float gamma = e_[C - 1];
            float sub[1][2][4] = {};
            tf32::tile<1, 2, true, true, false, false, 8>(sub, g.W + m0, LD, g.sV, LV, C);
            tf32::each<1, 2>([&](int i, int j, int e, int r, int c) {
                dS[i][j][e] = fmaf(gamma, dS[i][j][e], g.H[(m0 + r) * LO + c] + sub[i][j][e]);
                if (e & 1) *reinterpret_cast<float2 *>(g.sS + (m0 + r) * LO + c - 1) = make_float2(dS[i][j][e - 1], dS[i][j][e]);
            });
        }
    }
    if (p.dS0 && in_bounds(p.dS0 + bh * p.Dk * p.Dv, (size_t)p.Dk * p.Dv * 4, p.dS0, p.ns_bytes, p.bounds))
        tf32::each<1, 2>([&](int i, int j, int e, int r, int c) {
            r += m0;
            if (r < p.Dk && j0 + c < p.Dv) p.dS0[(bh * p.Dk + r) * p.Dv + j0 + c] = dS[i][j][e];
        });
}

template <typename T, bool FULL>
__global__ void __launch_bounds__(NT_C, 2) gb_chain_kernel(const __grid_constant__ GbArgs p) {
    extern __shared__ __align__(16) uint8_t gb_sm[];
    // the backward ones first: they take longer, and an SM then holds one of each (16 heads: 228 us, alternating 244)
    const int64_t half = gridDim.x >> 1, job = blockIdx.x < half ? blockIdx.x : blockIdx.x - half, bh = job / p.nslice;
    const int j0 = (int)(job - bh * p.nslice) * VS;
    const Rec R = make_rec(p.Dk, p.Dv);
    if (!in_bounds(p.ws + bh * p.Nc * R.size, (size_t)p.Nc * R.size * 4, p.ws, p.ws_bytes, p.bounds)) return;
    float *sm = reinterpret_cast<float *>(gb_sm);
    if (blockIdx.x < half) chain_backward<T, FULL>(p, bh, j0, sm);
    else chain_forward<T, FULL>(p, bh, j0, sm);
}

// ---------------------------------------------------------------- per chunk: the gradients
// The products over the value channels (dQg, dKd, dW, dM, the first part of dT) are summed over pieces of 32 channels,
// whose operands arrive while the piece before them is used; fp32 inputs leave room for one set of them.
constexpr int LQ = 40;  // pitch of the pieces: 8 mod 32, and for bf16 pairs distinct banks
template <typename T> struct Piece {
    static constexpr int SETS = sizeof(T) == 2 ? 2 : 1;
    static constexpr size_t BYTES = sizeof(float) * (2 * 128 + 2 * C) * LQ + 2 * sizeof(T) * C * LQ;
    float *S, *dS, *dV, *V;  // [128][LQ], [64][LQ]
    T *dO, *v;
    __device__ Piece(uint8_t *base, int i) {
        S = reinterpret_cast<float *>(base + (SETS == 2 ? (i & 1) * BYTES : 0));
        dS = S + 128 * LQ;
        dV = dS + 128 * LQ;
        V = dV + C * LQ;
        dO = reinterpret_cast<T *>(V + C * LQ);
        v = dO + C * LQ;
    }
};
// what takes their place afterwards: dW and dV' [64][LD], dT and T^T dT [64][LC]
constexpr size_t AFTER_BYTES = sizeof(float) * (2 * C * LD + 2 * C * LC);
template <typename T> constexpr size_t grad_area() {
    return Piece<T>::SETS * Piece<T>::BYTES > AFTER_BYTES ? Piece<T>::SETS * Piece<T>::BYTES : AFTER_BYTES;
}
template <typename T> constexpr size_t grad_smem() {
    return sizeof(double) * C + sizeof(float) * (2 * C * LC + 3 * C + 32) + 2 * sizeof(T) * C * LD + grad_area<T>();
}

template <typename T>
__global__ void __launch_bounds__(NT_P, 1) gb_grad_kernel(const __grid_constant__ GbArgs p) {
    constexpr bool EX = sizeof(T) == 2;
    extern __shared__ __align__(16) uint8_t gb_sm[];
    double *sG = reinterpret_cast<double *>(gb_sm);
    float *sT = reinterpret_cast<float *>(sG + C), *sM = sT + C * LC;  // T, dM * E [64][LC]
    float *seG = sM + C * LC, *seD = seG + C, *sb = seD + C, *sred = sb + C;
    T *sK = reinterpret_cast<T *>(sred + 32), *sQ = sK + C * LD;        // [64][LD]
    uint8_t *area = reinterpret_cast<uint8_t *>(sQ + C * LD);
    float *sdW = reinterpret_cast<float *>(area), *sdV = sdW + C * LD, *sdT = sdV + C * LD, *sY = sdT + C * LC;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t4 = lane & 3;
    const int64_t bh = blockIdx.x / p.Nc;
    const int n = (int)(blockIdx.x - bh * p.Nc);
    const Unit u = unit_of(p, bh, n);
    const int Dk = p.Dk, Dv = p.Dv, Dkp = pad16(Dk), Dvp = pad32(Dv), len = u.len;
    const Rec R = make_rec(Dk, Dv);
    const float *rec = p.ws + (int64_t)blockIdx.x * R.size;
    if (!in_bounds(rec, (size_t)R.size * 4, p.ws, p.ws_bytes, p.bounds)) return;
    const int64_t rk = (int64_t)p.H * Dk, rv = (int64_t)p.H * Dv;
    const T *gv = (const T *)p.v + u.row0 * Dv, *gO = (const T *)p.dO + u.row0 * Dv;

    auto stage_cols = [&](T *dst, const T *src, int j0) {  // 32 columns of token rows
        if (p.wide_v) {
            constexpr int E = 16 / (int)sizeof(T), VPR = 32 / E;
            const int r = tid / VPR, c = tid % VPR * E;
            if (tid < C * VPR) {
                const bool in = r < len && j0 + c < Dv;
                cp_async16_fill(reinterpret_cast<float *>(dst + r * LQ + c),
                                reinterpret_cast<const float *>(src + (in ? r * rv + j0 + c : 0)), in);
            }
        } else {
            const int c = tid & 31;
#pragma unroll
            for (int r = tid >> 5; r < C; r += NT_P / 32)
                dst[r * LQ + c] = (r < len && j0 + c < Dv) ? src[r * rv + j0 + c] : T(0.f);
        }
    };
    auto stage = [&](int i) {
        const Piece<T> q(area, i);
        const int j0 = 32 * i;
        stage_block<NT_P, 8>(q.S, LQ, rec + R.S + j0, Dvp, Dkp, 32);
        stage_block<NT_P, 8>(q.dS, LQ, rec + R.dS + j0, Dvp, Dkp, 32);
        stage_block<NT_P, 8>(q.dV, LQ, rec + R.dV + j0, Dvp, C, 32);
        stage_block<NT_P, 8>(q.V, LQ, rec + R.V + j0, Dvp, C, 32);
        stage_cols(q.dO, gO, j0);
        stage_cols(q.v, gv, j0);
        cp_async_commit_group();
    };
    stage(0);
    stage_rows<T, NT_P>(sK, (const T *)p.k + u.row0 * Dk, rk, len, Dk, Dkp, p.wide_k);
    stage_rows<T, NT_P>(sQ, (const T *)p.q + u.row0 * Dk, rk, len, Dk, Dkp, p.wide_k);
    stage_block<NT_P, 16>(sT, LC, rec + R.T, C, C, C);
    cp_async_commit_group();
    if (tid < C) {
        sG[tid] = reinterpret_cast<const double *>(rec + R.G)[tid];
        seG[tid] = rec[R.eG + tid];
        seD[tid] = rec[R.eD + tid];
        sb[tid] = tid < len ? load_elem((const T *)p.beta, u.row0 + (int64_t)tid * p.H) : 0.f;
    }

    // every warp: 32 rows from r0; 16 columns from c0 of [64][D] results, 8 from c1 of [64][64] ones
    const int r0 = row_half(warp), ct = warp >> 1, c0 = 16 * ct, c1 = 8 * ct;
    const bool inK = c0 < Dkp, inV = c0 < Dvp, tri = c1 < r0 + 32;  // tri: the tile reaches below the diagonal
    float dq[2][2][4] = {}, dk[2][2][4] = {}, X[2][1][4] = {};
    float late[2][2] = {}, early[2][2] = {}, db[2][2] = {};  // row sums of this lane's rows 16 i + g + 8 half
    float dot = 0.f;                                          // <dS_next, S>
    {
        float w[2][2][4] = {}, m[2][1][4] = {}, d[2][1][4] = {};
        const int np = Dvp / 32;
        for (int i = 0; i < np; ++i) {
            if (i == 0) cp_async_wait<1>();  // the first piece; k, q and T may still be on their way
            else cp_async_wait<0>();
            __syncthreads();
            if (Piece<T>::SETS == 2 && i + 1 < np) stage(i + 1);
            const Piece<T> q(area, i);
            if (inK) {
                tf32::tile<2, 2, false, false, EX, false, 4>(dq, q.dO + r0 * LQ, LQ, q.S + c0 * LQ, LQ, 32);
                tf32::tile<2, 2, false, false, false, false, 4>(w, q.dV + r0 * LQ, LQ, q.S + c0 * LQ, LQ, 32);
            }
            if (tri) {
                tf32::tile<2, 1, false, false, EX, false, 4>(m, q.dO + r0 * LQ, LQ, q.V + c1 * LQ, LQ, 32);
                tf32::tile<2, 1, false, false, false, EX, 4>(d, q.dV + r0 * LQ, LQ, q.v + c1 * LQ, LQ, 32);
            }
            if (inK) tf32::tile<2, 2, false, false, false, false, 4>(dk, q.V + r0 * LQ, LQ, q.dS + c0 * LQ, LQ, 32);
            for (int r = tid >> 3, c = (tid & 7) * 4; r < Dkp; r += NT_P / 8) {
                const float4 x = *reinterpret_cast<const float4 *>(q.S + r * LQ + c);
                const float4 y = *reinterpret_cast<const float4 *>(q.dS + r * LQ + c);
                dot = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, dot))));
            }
            if (Piece<T>::SETS == 1 && i + 1 < np) {
                __syncthreads();
                stage(i + 1);
            }
        }
        float2 M[2][2];
        tf32::each<2, 1>([&](int i, int j, int e, int r, int c) {
            if (!(e & 1)) M[i][e >> 1] = *reinterpret_cast<const float2 *>(rec + R.M + (r0 + r) * C + c1 + c);
        });
        cp_async_wait<0>();
        __syncthreads();  // the pieces are read; k, q and T are there
        stage_block<NT_P, 32>(sdV, LD, rec + R.dV, Dvp, C, Dvp);
        cp_async_commit_group();
        if (inK)  // dq = e^G dQg, dk = e^D dKd, dW
            tf32::each<2, 2>([&](int i, int j, int e, int r, int c) {
                r += r0;
                c += c0;
                dq[i][j][e] *= seG[r];
                dk[i][j][e] *= seD[r];
                late[i][e >> 1] = fmaf(dq[i][j][e], load_elem(sQ, r * LD + c), late[i][e >> 1]);
                early[i][e >> 1] = fmaf(dk[i][j][e], load_elem(sK, r * LD + c), early[i][e >> 1]);
                if (e & 1) *reinterpret_cast<float2 *>(sdW + r * LD + c - 1) = make_float2(-w[i][j][e - 1], -w[i][j][e]);
            });
        tf32::each<2, 1>([&](int i, int j, int e, int r, int c) {  // dM (i <= r)
            r += r0;
            c += c1;
            const float x = c <= r ? m[i][j][e] : 0.f;
            sM[r * LC + c] = c <= r ? x * expf((float)(sG[r] - sG[c])) : 0.f;
            if (c < r) X[i][j][e] = x * (e & 1 ? M[i][e >> 1].y : M[i][e >> 1].x);
        });
        __syncthreads();
        // dT = dV' Bv^T + dW Bk^T, on and below the diagonal (T has nothing above it)
        float b[2][1][4] = {};
        if (tri) tf32::tile<2, 1, false, false, false, EX>(b, sdW + r0 * LD, LD, sK + c1 * LD, LD, Dkp);
        tf32::each<2, 1>([&](int i, int j, int e, int r, int c) {
            r += r0;
            c += c1;
            sdT[r * LC + c] = c <= r ? sb[c] * fmaf(seG[c], b[i][j][e], d[i][j][e]) : 0.f;
        });
    }
    float2 vv[2][2][2];  // this lane's pairs of v, on their way meanwhile
    tf32::each<2, 2>([&](int i, int j, int e, int r, int c) {
        if (!(e & 1)) vv[i][j][e >> 1] = row_pair(gv + (r0 + r) * rv, c0 + c, Dv, r0 + r < len, p.wide_v);
    });
    if (inK) {  // dBk = T^T dW
        float a[2][2][4] = {};
        tf32::tile<2, 2, true, true, false, false>(a, sT + r0 + r0 * LC, LC, sdW + c0 + r0 * LD, LD, C - r0);
        tf32::each<2, 2>([&](int i, int j, int e, int r, int c) {
            r += r0;
            const float x = a[i][j][e] * seG[r], xk = x * load_elem(sK, r * LD + c0 + c);
            db[i][e >> 1] += xk;
            late[i][e >> 1] = fmaf(sb[r], xk, late[i][e >> 1]);
            dk[i][j][e] = fmaf(sb[r], x, dk[i][j][e]);
        });
    }
    cp_async_wait<0>();  // dV'
    __syncthreads();
    if (inV) {  // dBv = T^T dV'
        float a[2][2][4] = {};
        tf32::tile<2, 2, true, true, false, false>(a, sT + r0 + r0 * LC, LC, sdV + c0 + r0 * LD, LD, C - r0);
        tf32::each<2, 2>([&](int i, int j, int e, int r, int c) {
            r += r0;
            c += c0;
            db[i][e >> 1] = fmaf(a[i][j][e], e & 1 ? vv[i][j][e >> 1].y : vv[i][j][e >> 1].x, db[i][e >> 1]);
            store_pair(p.dv, p.nv_bytes, p.bounds, (u.row0 + (int64_t)r * p.H) * Dv, c - (e & 1), Dv, r < len && (e & 1),
                       p.pair_v, sb[r] * a[i][j][e & 2], sb[r] * a[i][j][e | 1]);
        });
    }
    {
        float y[2][1][4] = {};  // T^T dT
        tf32::tile<2, 1, true, true, false, false>(y, sT + r0 + r0 * LC, LC, sdT + c1 + r0 * LC, LC, C - r0);
        tf32::each<2, 1>([&](int i, int j, int e, int r, int c) { sY[(r0 + r) * LC + c1 + c] = y[i][j][e]; });
    }
    float2 Pp[2][2];
    tf32::each<2, 1>([&](int i, int j, int e, int r, int c) {
        if (!(e & 1)) Pp[i][e >> 1] = *reinterpret_cast<const float2 *>(rec + R.P + (r0 + r) * C + c1 + c);
    });
    __syncthreads();
    float *sdP = sdW;  // [64][LC]; dW is read
    {  // dA = -(T^T dT) T^T (i < r);  dP' = beta dA E
        float a[2][1][4] = {};
        if (tri) tf32::tile<2, 1, false, false, false, false>(a, sY + r0 * LC, LC, sT + c1 * LC, LC, c1 + 8);
        tf32::each<2, 1>([&](int i, int j, int e, int r, int c) {
            r += r0;
            c += c1;
            float x = 0.f;
            if (c < r) {
                const float P = e & 1 ? Pp[i][e >> 1].y : Pp[i][e >> 1].x;
                db[i][e >> 1] = fmaf(-a[i][j][e], P, db[i][e >> 1]);
                x = -a[i][j][e] * sb[r];
                X[i][j][e] = fmaf(x, P, X[i][j][e]);
                x *= expf((float)(sG[r] - sG[c]));
            }
            sdP[r * LC + c] = x;
        });
    }
    __syncthreads();
    if (inK) {
        tf32::tile<2, 2, false, true, false, EX>(dq, sM + r0 * LC, LC, sK + c0, LD, r0 + 32);
        tf32::tile<2, 2, false, true, false, EX>(dk, sdP + r0 * LC, LC, sK + c0, LD, r0 + 32);
        tf32::tile<2, 2, true, true, false, EX>(dk, sdP + r0 + r0 * LC, LC, sK + c0 + r0 * LD, LD, C - r0);
        tf32::tile<2, 2, true, true, false, EX>(dk, sM + r0 + r0 * LC, LC, sQ + c0 + r0 * LD, LD, C - r0);
        tf32::each<2, 2>([&](int i, int j, int e, int r, int c) {
            r += r0;
            c += c0;
            const int64_t row = (u.row0 + (int64_t)r * p.H) * Dk;
            const bool in = r < len && (e & 1);
            store_pair(p.dq, p.nk_bytes, p.bounds, row, c - (e & 1), Dk, in, p.pair_k, dq[i][j][e & 2], dq[i][j][e | 1]);
            store_pair(p.dk, p.nk_bytes, p.bounds, row, c - (e & 1), Dk, in, p.pair_k, dk[i][j][e & 2], dk[i][j][e | 1]);
        });
    }
    // the sums over rows and pairs, in the places of T^T dT and dV', which are read
    float *sX = sY, *part = sdV;  // part: [late, early, db][8 column groups][64]
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
            float s[3] = {late[i][hh], early[i][hh], db[i][hh]};
#pragma unroll
            for (int k = 0; k < 3; ++k) {
                s[k] += __shfl_xor_sync(0xffffffffu, s[k], 1);
                s[k] += __shfl_xor_sync(0xffffffffu, s[k], 2);
                if (t4 == 0) part[(k * 8 + ct) * C + r0 + 16 * i + 8 * hh + g] = s[k];
            }
        }
    tf32::each<2, 1>([&](int i, int j, int e, int r, int c) { sX[(r0 + r) * LC + c1 + c] = X[i][j][e]; });
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, m);
    if (lane == 0) sred[warp] = dot;
    __syncthreads();
    // sX[r][t] <- sum over i <= t of row r (a warp per four rows, two columns per lane)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float *row = sX + (4 * warp + i) * LC + 2 * lane;
        const float a = row[0], b = row[1];
        float s = a + b;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const float o = __shfl_up_sync(0xffffffffu, s, m);
            if (lane >= m) s += o;
        }
        row[0] = s - b;
        row[1] = s;
    }
    float *sums = part + 24 * C;  // late, early, db [64] each
    if (tid < 3 * C) {
        const int k = tid / C, r = tid % C;
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) s += part[(k * 8 + w) * C + r];
        sums[tid] = s;
    }
    __syncthreads();
    {  // eight lanes per token share its sums
        const int t = tid >> 3, part = tid & 7;
        float dg = 0.f;
#pragma unroll
        for (int i = 0; i < C / 8; ++i) {
            const int r = part + 8 * i;
            if (r >= t) dg += sums[r] + (t > 0 ? sX[r * LC + t - 1] : 0.f);
            else dg += sums[C + r];
        }
        float d = sred[part] + sred[part + 8];
#pragma unroll
        for (int m = 4; m > 0; m >>= 1) {
            dg += __shfl_xor_sync(0xffffffffu, dg, m);
            d += __shfl_xor_sync(0xffffffffu, d, m);
        }
        dg = fmaf(seG[C - 1], d, dg);
        if (part) return;
        if (t < len) {
            const int64_t at = u.row0 + (int64_t)t * p.H;
            if (in_bounds(p.dbeta + at, 4, p.dbeta, p.nb_bytes, p.bounds)) p.dbeta[at] = sums[2 * C + t];
            if (!in_bounds(p.dz + at, 4, p.dz, p.nb_bytes, p.bounds)) return;
            if (p.log_decay) {  // a clamped input has no gradient
                const float x = p.log_decay[at];
                p.dz[at] = (x >= p.g_min && x <= 0.f) ? dg : 0.f;
            } else {  // d sigmoid(z)/dz = e / (1 + e)^2, e = e^{-|z|}: no cancellation where sigmoid is near 1
                const float e = expf(-fabsf(load_elem((const T *)p.z, at)));
                p.dz[at] = dg * p.g_min * e / ((1.f + e) * (1.f + e));
            }
        }
    }
}

// ---------------------------------------------------------------- host side
size_t gdn_bwd_workspace(int64_t B, int64_t S, int H, int Dk, int Dv) {
    return (size_t)B * H * ((S + C - 1) / C) * (size_t)make_rec(Dk, Dv).size * sizeof(float);
}

template <typename T>
kda_status_t gb_launch(GbArgs p, int64_t nbh, cudaStream_t st) {
    const int64_t units = nbh * p.Nc, jobs = 2 * nbh * p.nslice;
    cudaFuncSetAttribute(gb_prep_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)prep_smem<T>());
    const auto chain = pad16(p.Dk) == 128 ? gb_chain_kernel<T, true> : gb_chain_kernel<T, false>;
    cudaFuncSetAttribute(chain, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)chain_smem<T>());
    cudaFuncSetAttribute(gb_grad_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)grad_smem<T>());
    p.wide_k = p.Dk * (int)sizeof(T) % 16 == 0 && aligned_to(p.q, 16) && aligned_to(p.k, 16);
    p.wide_v = p.Dv * (int)sizeof(T) % 16 == 0 && aligned_to(p.v, 16) && aligned_to(p.dO, 16);
    p.pair_k = p.Dk % 2 == 0 && aligned_to(p.dq, 8) && aligned_to(p.dk, 8);
    p.pair_v = p.Dv % 2 == 0 && aligned_to(p.dv, 8);
    gb_prep_kernel<T><<<(unsigned)units, prep_nt<T>(), prep_smem<T>(), st>>>(p);
    KDA_TRY(check_launch("gb_prep_kernel"));
    chain<<<(unsigned)jobs, NT_C, chain_smem<T>(), st>>>(p);
    KDA_TRY(check_launch("gb_chain_kernel"));
    gb_grad_kernel<T><<<(unsigned)units, NT_P, grad_smem<T>(), st>>>(p);
    return check_launch("gb_grad_kernel");
}

kda_status_t gb_validate(const kda_recurrent_bwd_args *a) {
    if (!a) return fail(KDA_ERR_INVALID_ARG, "args is NULL");
    KDA_TRY(check_dtype(a->dtype));
    KDA_TRY(check_gmin(a->g_min));
    if (a->B < 0 || a->S < 0 || a->H < 1 || a->D_k < 1 || a->D_v < 1)
        return fail(KDA_ERR_INVALID_ARG, "bad sizes B=%lld S=%lld H=%d D_k=%d D_v=%d", (long long)a->B, (long long)a->S,
                    a->H, a->D_k, a->D_v);
    if (a->D_k > 128 || a->D_v > 128)
        return fail(KDA_ERR_UNSUPPORTED, "D_k and D_v must be <= 128 (got %d, %d)", a->D_k, a->D_v);
    // one CTA per (b, h, chunk), and two per (b, h, 16 value columns)
    const int64_t nc = a->S / C + (a->S % C != 0), most = nc > 16 ? nc : 16;
    if (a->B > 0 && (a->B > 0x7fffffffLL / a->H || a->B * a->H > 0x7fffffffLL / most))
        return fail(KDA_ERR_UNSUPPORTED, "gdn backward: B*H*max(chunks, 16) exceeds 2^31 - 1");
    return KDA_OK;
}

}  // namespace

}  // namespace kda

using namespace kda;

extern "C" {

kda_status_t kda_gdn_chunk_bwd_workspace_size(const kda_recurrent_bwd_args *a, size_t *bytes) {
    clear_error();
    if (!bytes) return fail(KDA_ERR_INVALID_ARG, "bytes is NULL");
    KDA_TRY(gb_validate(a));
    *bytes = gdn_bwd_workspace(a->B, a->S, a->H, a->D_k, a->D_v);
    return KDA_OK;
}

kda_status_t kda_gdn_chunk_bwd(const kda_recurrent_bwd_args *a) {
    clear_error();
    KDA_TRY(gb_validate(a));
    if (a->B == 0) return KDA_OK;
    const size_t need = gdn_bwd_workspace(a->B, a->S, a->H, a->D_k, a->D_v);
    KDA_TRY(bwd_check_buffers(a, need, true));
    cudaStream_t st = (cudaStream_t)a->stream;
    const int64_t nbh = a->B * a->H;
    GbArgs p;
    p.S = a->S;
    p.H = a->H;
    p.Dk = a->D_k;
    p.Dv = a->D_v;
    p.Nc = (int)((a->S + C - 1) / C);
    p.nslice = pad32(a->D_v) / VS;
    p.q = a->q; p.k = a->k; p.v = a->v; p.z = a->z; p.beta = a->beta; p.dO = a->d_o;
    p.log_decay = a->log_decay;
    p.g_min = a->g_min;
    p.S0 = a->initial_state;
    p.dST = a->d_final_state;
    p.dq = a->dq; p.dk = a->dk; p.dv = a->dv; p.dbeta = a->dbeta; p.dz = a->dz; p.dS0 = a->d_initial_state;
    p.ws = reinterpret_cast<float *>(a->workspace);
    const size_t ns = (size_t)nbh * a->D_k * a->D_v * 4, nb = (size_t)nbh * a->S * 4;
    p.ws_bytes = checked_size(need);
    p.ns_bytes = checked_size(ns);
    p.nk_bytes = checked_size(nb * a->D_k);
    p.nv_bytes = checked_size(nb * a->D_v);
    p.nb_bytes = checked_size(nb);
    p.bounds = device_bounds_counter();
    if (a->S == 0) {  // no token: the state's gradient passes through
        if (a->d_initial_state) {
            const cudaError_t e = a->d_final_state
                                      ? cudaMemcpyAsync(a->d_initial_state, a->d_final_state, ns,
                                                        cudaMemcpyDeviceToDevice, st)
                                      : cudaMemsetAsync(a->d_initial_state, 0, ns, st);
            if (e != cudaSuccess) return fail(KDA_ERR_CUDA, "gdn backward: %s", cudaGetErrorString(e));
        }
        return KDA_OK;
    }
    return a->dtype == KDA_F32 ? gb_launch<float>(p, nbh, st) : gb_launch<__nv_bfloat16>(p, nbh, st);
}

}  // extern "C"
