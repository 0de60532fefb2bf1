// The dense product with its epilogue, Z = X W^T + b, Y = act(Z) + R, and its gradients.
//
// Three kernels:
//   * linear_gemm_kernel: tensor-core tiles.  D = A B^T with 128 x BN output tiles; one thread
//     feeds shared memory with TMA (128-byte-swizzled boxes of 64 x 64), one issues tcgen05.mma
//     into one of two fp32 accumulators in TMEM, four warps drain the other one: bias, activation
//     and residual are applied in fp32 registers and the output is rounded once.  Persistent CTAs
//     walk the tiles, so the epilogue of a tile runs under the products of the next.  Either
//     operand may lie along the contraction (rows of K) or across it (the gradients' transposed
//     operands): only the boxes' order and two descriptor bits differ, nothing is transposed in
//     memory.  One launch takes up to two products (dX = dZ W and dW = dZ^T X).
//   * linear_rows_kernel: a few rows.  A warp per output column streams that column's weights once
//     for all rows.
//   * linear_dz_kernel: dZ = dY act'(Z) and the column sums behind db.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "norm.cuh"
#include "tcgen05_ptx.cuh"

namespace fe {

enum { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3, kActSwiglu = 4 };

// Device-side problems of the entry points without a handle (kDevTcTimeout).
__device__ uint32_t g_op_status;

FE_DEV float phi_cdf(float z) { return 0.5f * (1.0f + erff(z * 0.70710678118654752f)); }

FE_DEV float act_fwd(int act, float z)
{
    if (act == kActRelu) return z > 0.0f ? z : (z == z ? 0.0f : z);
    if (act == kActGelu) return z * phi_cdf(z);
    if (act == kActSilu) return z * sigmoidf(z);
    return z;
}

// act'(z) of the elementwise activations.
FE_DEV float act_bwd(int act, float z)
{
    if (act == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
    if (act == kActGelu) return phi_cdf(z) + z * __expf(-0.5f * z * z) * 0.39894228040143268f;
    if (act == kActSilu) {
        const float q = sigmoidf(z);
        return q * (1.0f + z * (1.0f - q));
    }
    return 1.0f;
}

// ---- tensor-core tiles ---------------------------------------------------------------

constexpr int kLinThreads = 256;   // warp 0: TMA, 1: MMA, 2: TMEM, 4-7: epilogue
constexpr int kLinM = 128;
constexpr uint32_t kLinBox = 64 * 128;   // one TMA box: 64 rows of 128 bytes
constexpr unsigned long long kLinTimeoutNs = 2000ull * 1000 * 1000;

__host__ __device__ constexpr int lin_stages(int BN) { return BN == 256 ? 4 : 6; }
__host__ __device__ constexpr uint32_t lin_stage_bytes(int BN) { return kLinM * 128 + BN * 128; }
__host__ __device__ constexpr uint32_t lin_smem_bytes(int BN)
{
    return 1024 + lin_stages(BN) * lin_stage_bytes(BN) + 8 * (2 * lin_stages(BN) + 4) + 16;
}

struct LinProblem {
    CUtensorMap ta, tb;      // boxes of 64 x 64, 128-byte swizzle
    int M, N, K;             // D [M][N] = A [M][K] B [N][K]^T
    int a_mn, b_mn;          // operand stored across the contraction: A as [K][M], B as [K][N]
    int tiles_m, tiles_n;
    int act;
    int cols;                // output columns: N, or N / 2 for swiglu
    const uint16_t* bias;    // [N] or null
    const uint16_t* res;     // [M][ldr] or null
    int64_t ldr;
    uint16_t* out;           // [M][ldo]
    int64_t ldo;
    uint16_t* z;             // [M][N] or null
    int vec;                 // out, res and z rows take 16-byte accesses
};

struct LinParams {
    LinProblem p[2];
    int tiles0, tiles;       // tiles of p[0], of both
};

FE_DEV void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// Descriptor of an operand stored across the contraction: boxes of 64 (M or N) x 64 k, one 128-byte
// row per k, 8-k groups 1024 bytes apart, the next 64 of M or N one box further.
FE_DEV uint64_t lin_desc_mn(uint32_t saddr)
{
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(kLinBox >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

FE_DEV void tc_ld32(uint32_t taddr, uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// 32 consecutive columns from c0 of one row: dst[c0 + j] = bf16(v[j]) for c0 + j < cols.
FE_DEV void lin_store32(uint16_t* dst, int c0, int cols, bool vec, const float (&v)[32])
{
    if (vec && c0 + 32 <= cols) {
        uint4* d = reinterpret_cast<uint4*>(dst + c0);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            d[q] = make_uint4(bf16x2_rn(v[8 * q], v[8 * q + 1]), bf16x2_rn(v[8 * q + 2], v[8 * q + 3]),
                              bf16x2_rn(v[8 * q + 4], v[8 * q + 5]), bf16x2_rn(v[8 * q + 6], v[8 * q + 7]));
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (c0 + j < cols) dst[c0 + j] = (uint16_t)(bf16x2_rn(v[j], 0.0f) & 0xffffu);
    }
}

// v[j] += src[c0 + j] (bf16) for c0 + j < cols.
FE_DEV void lin_add32(const uint16_t* src, int c0, int cols, bool vec, float (&v)[32])
{
    if (vec && c0 + 32 <= cols) {
        const uint4* s = reinterpret_cast<const uint4*>(src + c0);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint4 w = s[q];
            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * q + 2 * j] += __uint_as_float(a[j] << 16);
                v[8 * q + 2 * j + 1] += __uint_as_float(a[j] & 0xffff0000u);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 32; ++j)
            if (c0 + j < cols) v[j] += bf16_bits_to_f32(src[c0 + j]);
    }
}

template <int BN>
__global__ void __launch_bounds__(kLinThreads, 1) linear_gemm_kernel(const __grid_constant__ LinParams P)
{
    constexpr int S = lin_stages(BN);
    constexpr uint32_t kStage = lin_stage_bytes(BN);
    extern __shared__ uint8_t lin_dyn[];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t base0 = tc_saddr(lin_dyn);
    uint8_t* sm = lin_dyn + ((1024u - (base0 & 1023u)) & 1023u);
    const uint32_t ring = tc_saddr(sm);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S * kStage);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 4);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t bar0 = tc_saddr(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };
    auto empty = [&](int s) { return bar0 + 8u * (S + s); };
    auto accfull = [&](int s) { return bar0 + 8u * (2 * S + s); };
    auto accempty = [&](int s) { return bar0 + 8u * (2 * S + 2 + s); };
    if (tid == 0) {
        for (int s = 0; s < S; ++s) {
            tc_mbar_init(full(s), 1);
            tc_mbar_init(empty(s), 1);
        }
        for (int s = 0; s < 2; ++s) {
            tc_mbar_init(accfull(s), 1);
            tc_mbar_init(accempty(s), 4);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        *abort = 0;
    }
    if (warp == 2) {
        tc_alloc(tc_saddr(tmem_slot), 2 * BN);
        tc_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();

    if (warp == 0) {
        if (lane == 0) {
            // ---- producer: boxes of A and B into the ring ------------------------------------
            uint32_t it = 0;
            for (int tile = blockIdx.x; tile < P.tiles && !*abort; tile += gridDim.x) {
                const LinProblem& p = P.p[tile >= P.tiles0];
                const int ti = tile >= P.tiles0 ? tile - P.tiles0 : tile;
                const int m0 = ti / p.tiles_n * kLinM, tn = ti % p.tiles_n;
                const int nk = (p.K + 63) / 64;
                for (int k = 0; k < nk; ++k, ++it) {
                    const int s = it % S;
                    if (it >= S && !tc_mbar_wait(empty(s), (it / S - 1) & 1, kLinTimeoutNs)) {
                        *abort = 1;
                        break;
                    }
                    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(full(s)), "r"(kStage)
                                 : "memory");
                    const uint32_t a = ring + s * kStage, b = a + kLinM * 128;
#pragma unroll
                    for (int i = 0; i < kLinM / 64; ++i) {
                        const int m = m0 + 64 * i;
                        tma_load_2d(a + i * kLinBox, &p.ta, p.a_mn ? m : 64 * k, p.a_mn ? 64 * k : m, full(s));
                    }
#pragma unroll
                    for (int i = 0; i < BN / 64; ++i) {
                        // swiglu: the first half of the tile's columns are gate rows of W, the
                        // second the up rows of the same output columns
                        int n = tn * BN + 64 * i;
                        if (p.act == kActSwiglu)
                            n = tn * (BN / 2) + 64 * (i % (BN / 128)) + (i >= BN / 128 ? p.cols : 0);
                        tma_load_2d(b + i * kLinBox, &p.tb, p.b_mn ? n : 64 * k, p.b_mn ? 64 * k : n, full(s));
                    }
                }
            }
            // no copy outlives the loop (only short of the consumer's waits after an abort)
            for (uint32_t j = it > S ? it - S : 0; j < it; ++j)
                tc_mbar_wait(full(j % S), (j / S) & 1, kLinTimeoutNs);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            // ---- MMA issue -----------------------------------------------------------------
            uint32_t it = 0, done = 0;
            for (int tile = blockIdx.x; tile < P.tiles && !*abort; tile += gridDim.x, ++done) {
                const LinProblem& p = P.p[tile >= P.tiles0];
                const int nk = (p.K + 63) / 64;
                const int acc = done & 1;
                // f32 accumulator, bf16 operands, transposed operands' bits, N and M
                const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)p.a_mn << 15) |
                                       ((uint32_t)p.b_mn << 16) | ((uint32_t)(BN >> 3) << 17) |
                                       ((uint32_t)(kLinM >> 4) << 24);
                if (done >= 2 && !tc_mbar_wait(accempty(acc), (done / 2 - 1) & 1, kLinTimeoutNs)) *abort = 1;
                tc_fence_after();
                for (int k = 0; k < nk && !*abort; ++k, ++it) {
                    const int s = it % S;
                    if (!tc_mbar_wait(full(s), (it / S) & 1, kLinTimeoutNs)) {
                        *abort = 1;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a = ring + s * kStage, b = a + kLinM * 128;
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint64_t ad = p.a_mn ? lin_desc_mn(a + 2048 * ks) : tc_smem_desc(a + 32 * ks);
                        const uint64_t bd = p.b_mn ? lin_desc_mn(b + 2048 * ks) : tc_smem_desc(b + 32 * ks);
                        tc_mma_f16(tmem + BN * acc, ad, bd, idesc, (k > 0 || ks > 0) ? 1u : 0u);
                    }
                    tc_commit(empty(s));
                }
                tc_commit(accfull(acc));
            }
            // never leave with MMAs in flight: they read shared memory and write TMEM
            for (uint32_t j = done > 2 ? done - 2 : 0; j < done; ++j)
                if (!tc_mbar_wait(accfull(j & 1), (j / 2) & 1, kLinTimeoutNs)) *abort = 1;
        }
        __syncwarp();
    } else if (warp >= 4) {
        // ---- epilogue: a thread per row, 32 columns at a time ----------------------------------
        uint32_t done = 0;
        for (int tile = blockIdx.x; tile < P.tiles; tile += gridDim.x, ++done) {
            const LinProblem& p = P.p[tile >= P.tiles0];
            const int ti = tile >= P.tiles0 ? tile - P.tiles0 : tile;
            const int acc = done & 1;
            const int64_t row = (int64_t)(ti / p.tiles_n) * kLinM + 32 * (warp - 4) + lane;
            const bool on = row < p.M, vec = p.vec != 0;
            if (!tc_mbar_wait(accfull(acc), (done / 2) & 1, kLinTimeoutNs)) *abort = 1;
            if (__any_sync(0xffffffffu, *abort != 0)) break;
            tc_fence_after();
            const uint32_t t0 = tmem + ((uint32_t)(32 * (warp - 4)) << 16) + BN * acc;
            if (p.act == kActSwiglu) {
                const int n0 = ti % p.tiles_n * (BN / 2);
#pragma unroll 1
                for (int c = 0; c < BN / 2; c += 32) {
                    uint32_t rg[32], ru[32];
                    tc_ld32(t0 + c, rg);
                    tc_ld32(t0 + BN / 2 + c, ru);
                    tc_wait_ld();
                    float g[32], u[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        g[j] = __uint_as_float(rg[j]);
                        u[j] = __uint_as_float(ru[j]);
                    }
                    const int c0 = n0 + c;
                    if (p.bias) {
                        lin_add32(p.bias, c0, p.cols, false, g);
                        lin_add32(p.bias + p.cols, c0, p.cols, false, u);
                    }
                    if (on && p.z) {
                        lin_store32(p.z + (size_t)row * p.N, c0, p.cols, vec, g);
                        lin_store32(p.z + (size_t)row * p.N + p.cols, c0, p.cols, vec, u);
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) g[j] = g[j] * sigmoidf(g[j]) * u[j];
                    if (on) {
                        if (p.res) lin_add32(p.res + (size_t)row * p.ldr, c0, p.cols, vec, g);
                        lin_store32(p.out + (size_t)row * p.ldo, c0, p.cols, vec, g);
                    }
                }
            } else {
                const int n0 = ti % p.tiles_n * BN;
#pragma unroll 1
                for (int c = 0; c < BN; c += 32) {
                    uint32_t r[32];
                    tc_ld32(t0 + c, r);
                    tc_wait_ld();
                    float v[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
                    const int c0 = n0 + c;
                    if (p.bias) lin_add32(p.bias, c0, p.cols, false, v);
                    if (on && p.z) lin_store32(p.z + (size_t)row * p.N, c0, p.cols, vec, v);
                    if (p.act != kActNone)
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = act_fwd(p.act, v[j]);
                    if (on) {
                        if (p.res) lin_add32(p.res + (size_t)row * p.ldr, c0, p.cols, vec, v);
                        lin_store32(p.out + (size_t)row * p.ldo, c0, p.cols, vec, v);
                    }
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(accempty(acc)) : "memory");
        }
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort) atomicOr(&g_op_status, kDevTcTimeout);
    if (warp == 2) {
        tc_fence_after();
        tc_dealloc(tmem, 2 * BN);
    }
}

// ---- a few rows ------------------------------------------------------------------------

struct LinRowsParams {
    const uint16_t* x;
    int64_t ldx;
    const uint16_t* w;
    const uint16_t* bias;
    const uint16_t* res;
    int64_t ldr;
    uint16_t* y;
    int64_t ldy;
    uint16_t* z;
    int M, N, K, act, cols;
};

FE_DEV void fma8(const uint4& a, const uint4& b, float& acc)
{
    const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        acc = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), acc);
        acc = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), acc);
    }
}

constexpr int kLinRowsWarps = 4;

// A warp per output column (two weight rows for swiglu), MR rows of x.
template <int MR, bool GLU>
__global__ void __launch_bounds__(32 * kLinRowsWarps) linear_rows_kernel(LinRowsParams p)
{
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int c = blockIdx.x * kLinRowsWarps + (threadIdx.x >> 5);
    if (c >= p.cols) return;
    const uint16_t* w0 = p.w + (size_t)c * p.K;
    const uint16_t* w1 = p.w + (size_t)(c + p.cols) * p.K;   // read for swiglu only
    float acc[2][MR];
#pragma unroll
    for (int m = 0; m < MR; ++m) acc[0][m] = acc[1][m] = 0.0f;
#pragma unroll 4
    for (int k = 8 * lane; k < p.K; k += 256) {
        const uint4 a = ldg_stream(w0 + k);
        uint4 b = make_uint4(0, 0, 0, 0);
        if (GLU) b = ldg_stream(w1 + k);
#pragma unroll
        for (int m = 0; m < MR; ++m) {
            if (m >= p.M) break;
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(p.x + (size_t)m * p.ldx + k));
            fma8(a, x, acc[0][m]);
            if (GLU) fma8(b, x, acc[1][m]);
        }
    }
#pragma unroll
    for (int m = 0; m < MR; ++m) {
        if (m >= p.M) break;
        float z0 = warp_sum(acc[0][m]), z1 = GLU ? warp_sum(acc[1][m]) : 0.0f;
        if (lane != 0) continue;
        if (p.bias) {
            z0 += bf16_bits_to_f32(p.bias[c]);
            if (GLU) z1 += bf16_bits_to_f32(p.bias[c + p.cols]);
        }
        if (p.z) {
            p.z[(size_t)m * p.N + c] = (uint16_t)(bf16x2_rn(z0, 0.0f) & 0xffffu);
            if (GLU) p.z[(size_t)m * p.N + c + p.cols] = (uint16_t)(bf16x2_rn(z1, 0.0f) & 0xffffu);
        }
        float v = GLU ? z0 * sigmoidf(z0) * z1 : act_fwd(p.act, z0);
        if (p.res) v += bf16_bits_to_f32(p.res[(size_t)m * p.ldr + c]);
        p.y[(size_t)m * p.ldy + c] = (uint16_t)(bf16x2_rn(v, 0.0f) & 0xffffu);
    }
}

// ---- dZ and its column sums ----------------------------------------------------------------

struct LinDzParams {
    const uint16_t* dy;   // [M][lddy]
    int64_t lddy;
    const uint16_t* z;    // [M][N], null for no activation
    uint16_t* dz;         // [M][lddz] or null
    int64_t lddz;
    float* part;          // [gridDim.y][N] or null
    int64_t M, rows_per_cta;
    int N, cols, act;
};

// VEC consecutive bf16 values (16-byte aligned when VEC is 8).
template <int VEC>
FE_DEV void dz_load(const uint16_t* p, float (&v)[VEC])
{
    if (VEC == 8) {
        const uint4 q = *reinterpret_cast<const uint4*>(p);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    } else {
        v[0] = bf16_bits_to_f32(*p);
    }
}

template <int VEC>
FE_DEV void dz_store(uint16_t* p, const float (&v)[VEC])
{
    if (VEC == 8)
        *reinterpret_cast<uint4*>(p) = make_uint4(bf16x2_rn(v[0], v[1 % VEC]), bf16x2_rn(v[2 % VEC], v[3 % VEC]),
                                                  bf16x2_rn(v[4 % VEC], v[5 % VEC]), bf16x2_rn(v[6 % VEC], v[7 % VEC]));
    else
        *p = (uint16_t)(bf16x2_rn(v[0], 0.0f) & 0xffffu);
}

// Block 32 x 8: a thread owns VEC columns, 8 threads share the rows of a chunk.
template <int VEC>
__global__ void __launch_bounds__(256) linear_dz_kernel(LinDzParams p)
{
    __shared__ float red[8][2 * VEC][33];
    griddep_wait();
    const int x = threadIdx.x & 31, yy = threadIdx.x >> 5;
    const int c = (blockIdx.x * 32 + x) * VEC;
    const int64_t r0 = (int64_t)blockIdx.y * p.rows_per_cta, r1 = min(p.M, r0 + p.rows_per_cta);
    const bool glu = p.act == kActSwiglu;
    float s0[VEC], s1[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) s0[j] = s1[j] = 0.0f;
    if (c < p.cols) {
        for (int64_t r = r0 + yy; r < r1; r += 8) {
            float g[VEC], z0[VEC], z1[VEC];
            dz_load<VEC>(p.dy + r * p.lddy + c, g);
            if (p.act != kActNone) dz_load<VEC>(p.z + r * p.N + c, z0);
            if (glu) dz_load<VEC>(p.z + r * p.N + p.cols + c, z1);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float d0, d1 = 0.0f;
                if (glu) {
                    const float q = sigmoidf(z0[j]);
                    d1 = g[j] * z0[j] * q;
                    d0 = g[j] * z1[j] * q * (1.0f + z0[j] * (1.0f - q));
                } else {
                    d0 = p.act == kActNone ? g[j] : g[j] * act_bwd(p.act, z0[j]);
                }
                s0[j] += d0;
                s1[j] += d1;
                z0[j] = d0;
                z1[j] = d1;
            }
            if (p.dz) {
                dz_store<VEC>(p.dz + r * p.lddz + c, z0);
                if (glu) dz_store<VEC>(p.dz + r * p.lddz + p.cols + c, z1);
            }
        }
    }
    if (!p.part) return;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
        red[yy][j][x] = s0[j];
        red[yy][VEC + j][x] = s1[j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * VEC * (glu ? 2 : 1); i += 256) {
        const int h = i / (32 * VEC), j = (i / 32) % VEC, xx = i & 31;
        const int col = (blockIdx.x * 32 + xx) * VEC + j;
        if (col >= p.cols) continue;
        float v = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) v += red[q][h * VEC + j][xx];
        p.part[(size_t)blockIdx.y * p.N + h * p.cols + col] = v;
    }
}

}  // namespace fe
