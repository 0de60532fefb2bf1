// The dense product with its epilogue, Z = X W^T + b, Y = act(Z) + R, and its gradients.
//
// Its kernels, by what bounds the product:
//   * linear_gemm_kernel, many tiles, bound by the tensor cores: D = A B^T in 256 x BN tiles by pairs of
//     CTAs; in each a warp feeds shared memory with TMA (128-byte-swizzled boxes), in the leader one
//     issues tcgen05.mma for both into one of two fp32 accumulators in TMEM, and eight warps drain the
//     other one: bias, activation and residual are applied in fp32 registers and the output is
//     rounded once.  Persistent pairs walk the tiles, so the epilogue of a tile runs under the
//     products of the next.  Either operand may lie along the contraction (rows of K) or across it
//     (the gradients' transposed operands): only the boxes' order and two descriptor bits differ,
//     nothing is transposed in memory.  One launch takes up to two products (dX = dZ W and dW = dZ^T X).
//     16384 x 1536 at K = 2048 with swiglu: 70 to 72 us, 1450 TFLOP/s; dX and dW of 4096 rows 39 us.  (All figures
//     here: launches of one kind in a captured graph, operands in turn.)
//   * linear_split_kernel, fewer tiles than SMs, bound by what an SM takes in: 128 x 64 or 128 x 128 tiles,
//     the contraction split over a cluster.  64 x 2048 at K = 768: 4.2 us; 1024 x 1000 at K = 2048: 9.0 us.
//   * linear_skinny_kernel, 2 to 16 rows, and linear_rows_kernel, one row: bound by one pass over the
//     weights.  1536 x 2048 with swiglu: 4.0 us for 16 rows, 2.8 us (2.2 TB/s) for one.
//   * linear_dz_kernel, memory: dZ = dY act'(Z) and the column sums behind db.  4096 x 1536 with swiglu:
//     7.2 us with the sums' launch.
#pragma once

#include <cuda.h>

#include "cluster.cuh"
#include "common.cuh"
#include "norm.cuh"
#include "tcgen05_ptx.cuh"

namespace fe {

enum { kActNone = 0, kActRelu = 1, kActGelu = 2, kActSilu = 3, kActSwiglu = 4 };

// Phi(z) and exp(-z^2 / 2), two at a time.  The tail is Q(|z|) = erfc(x) / 2 with x = |z| / sqrt 2, and
// erfc(x) = exp(-x^2) t p(t) with t = 1 / (1 + 0.43 x): erfc(x) exp(x^2) / t is smooth in t and p its
// polynomial of degree 7, fitted by reweighted least squares to 2e-7 relative for x up to 12, so the small
// tail keeps its digits.  One exponential, shared with the density, one reciprocal, the polynomial in
// paired instructions: with erff a tile's epilogue took as long as its products at K = 2048.
FE_DEV float2 phi_cdf2(float2 z, float2& e)
{
    const float2 y = make_float2(fabsf(z.x), fabsf(z.y));
    const float2 u = fma2(y, make_float2(0.304055916f, 0.304055916f), make_float2(1.0f, 1.0f));   // 0.43 / sqrt 2
    const float2 t = make_float2(rcp_ftz(u.x), rcp_ftz(u.y));
    const float2 w = mul2(mul2(z, z), make_float2(-0.5f * kLog2e, -0.5f * kLog2e));
    e = make_float2(ex2_ftz(w.x), ex2_ftz(w.y));
    constexpr float c[8] = {0.121269358f, 0.121994241f, 0.103734795f, 0.119104225f, -0.0344093589f, 0.182367387f, -0.149515733f, 0.0354549963f};   // p / 2
    float2 q = make_float2(c[7], c[7]);
#pragma unroll
    for (int i = 6; i >= 0; --i) q = fma2(q, t, make_float2(c[i], c[i]));
    q = mul2(q, mul2(t, e));
    return make_float2(z.x < 0.0f ? q.x : 1.0f - q.x, z.y < 0.0f ? q.y : 1.0f - q.y);
}

FE_DEV float phi_cdf(float z, float& e)
{
    float2 e2;
    const float2 c = phi_cdf2(make_float2(z, z), e2);
    e = e2.x;
    return c.x;
}

FE_DEV float act_fwd(int act, float z)
{
    if (act == kActRelu) return z > 0.0f ? z : (z == z ? 0.0f : z);
    if (act == kActGelu) {
        float e;
        return z * phi_cdf(z, e);
    }
    if (act == kActSilu) return z * sigmoidf(z);
    return z;
}

// act'(z) of the elementwise activations.
FE_DEV float act_bwd(int act, float z)
{
    if (act == kActRelu) return z > 0.0f ? 1.0f : 0.0f;
    if (act == kActGelu) {
        float e;
        const float c = phi_cdf(z, e);
        return c + z * e * 0.39894228040143268f;
    }
    if (act == kActSilu) {
        const float q = sigmoidf(z);
        return q * (1.0f + z * (1.0f - q));
    }
    return 1.0f;
}

// act over an array, the choice made once.
template <int N>
FE_DEV void act_all(int act, float (&v)[N])
{
    if (act == kActNone) return;
    if (act == kActRelu) {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = act_fwd(kActRelu, v[j]);
    } else if (act == kActGelu) {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            float2 e;
            const float2 c = phi_cdf2(make_float2(v[j], v[j + 1]), e);
            v[j] *= c.x;
            v[j + 1] *= c.y;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = act_fwd(kActSilu, v[j]);
    }
}

// act' over an array.
template <int ACT, int N>
FE_DEV void act_bwd_all(float (&v)[N])
{
    if (N % 2 == 0 && ACT == kActGelu) {
#pragma unroll
        for (int j = 0; j < N; j += 2) {
            float2 e;
            const float2 z = make_float2(v[j], v[N > 1 ? j + 1 : j]), c = phi_cdf2(z, e);
            v[j] = c.x + z.x * e.x * 0.39894228040143268f;
            v[N > 1 ? j + 1 : j] = c.y + z.y * e.y * 0.39894228040143268f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; ++j) v[j] = act_bwd(ACT, v[j]);
    }
}

// ---- tensor-core tiles ---------------------------------------------------------------

constexpr unsigned long long kLinTimeoutNs = 2000ull * 1000 * 1000;
constexpr int kLinThreads = 384;         // warp 0: TMA, 1: MMA, 2: TMEM, 4-11: epilogue
constexpr int kLinM = 256;               // rows of a tile: 128 in each CTA of the pair
constexpr uint32_t kLinABytes = 128 * 128;   // one k step of 64: 128 rows of 128 bytes
constexpr uint32_t kLinSlotBytes = 32 * 64;  // output staging: 32 rows x 32 columns of bf16
constexpr int kLinMaxPairs = 128;
// A stage: A, and BN / 2 columns' rows of 128 bytes, in boxes of 64 columns where B lies across.  What the
// staging leaves of shared memory is the ring's.
__host__ __device__ constexpr uint32_t lin_stage(int BN) { return kLinABytes + (BN / 2 + 63) / 64 * 8192; }
__host__ __device__ constexpr int lin_slots(bool plain) { return plain ? 2 : 4; }   // of each of the 8 epilogue warps
__host__ __device__ constexpr int lin_stages(int BN, bool plain)
{
    return (227 * 1024 - 1024 - 8 * lin_slots(plain) * (int)kLinSlotBytes - 8 * 20 - 16) / ((int)lin_stage(BN) + 16);
}
__host__ __device__ constexpr int lin_bars(int BN, bool plain) { return 2 * lin_stages(BN, plain) + 4 + 16; }
__host__ __device__ constexpr uint32_t lin_smem(int BN, bool plain)
{
    return 1024 + lin_stages(BN, plain) * lin_stage(BN) + 8 * lin_slots(plain) * kLinSlotBytes + 8 * lin_bars(BN, plain) + 16;
}

static_assert(lin_smem(128, true) <= 227 * 1024 && lin_smem(128, false) <= 227 * 1024 && lin_smem(192, true) <= 227 * 1024 &&
                  lin_smem(192, false) <= 227 * 1024 && lin_smem(256, true) <= 227 * 1024 && lin_smem(256, false) <= 227 * 1024,
              "a CTA's shared memory");

struct LinProblem {
    CUtensorMap ta, tb;      // operand boxes: 64 of k x rows (K-major), 64 x 64 of k (across)
    CUtensorMap to, tr, tz;  // out, res and z: boxes of 32 columns x 32 rows
    int M, N, K;             // D [M][N] = A [M][K] B [N][K]^T
    int a_mn, b_mn;          // operand stored across the contraction: A as [K][M], B as [K][N]
    int tiles_n, tiles;
    int act;
    int cols;                // output columns: N, or N / 2 for swiglu
    const uint16_t* bias;    // [N] or null
    const uint16_t* res;     // [M][ldr] or null
    int64_t ldr;
    uint16_t* out;           // [M][ldo]
    int64_t ldo;
    uint16_t* z;             // [M][N] or null
    int vec_out, vec_res, vec_z;   // rows suit TMA (16-byte aligned base and stride)
};

struct LinParams {
    LinProblem p[2];
    int n;                   // problems
    int start[2][kLinMaxPairs + 1];   // n == 2: pair c takes tiles [start[i][c], start[i][c + 1]) of problem i
};

FE_DEV void tma_load_2d(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cta.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// The same, completing on a barrier of either CTA of the pair.
FE_DEV void tma_load_2d_pair(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

FE_DEV void tma_store_2d(const CUtensorMap* map, int x, int y, uint32_t src)
{
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%1, %2}], [%3];\n\t"
                 "cp.async.bulk.commit_group;" ::"l"(map), "r"(x), "r"(y), "r"(src)
                 : "memory");
}

FE_DEV void prefetch_tensormap(const CUtensorMap* map) { asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory"); }

template <int N>
FE_DEV void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(N) : "memory"); }

// Bounded wait for phase `parity` of an mbarrier by a thread that suspends meanwhile: the products run
// at the power limit, where polling warps cost clocks.
FE_DEV bool lin_wait(uint32_t bar, uint32_t parity, unsigned long long limit_ns = kLinTimeoutNs)
{
    unsigned long long t0 = 0;
    for (int it = 0;; ++it) {
        uint32_t ok;
        asm volatile(
            "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity), "r"(20000u)
            : "memory");
        if (ok) return true;
        if (it == 0) t0 = globaltimer_ns();
        else if (globaltimer_ns() - t0 > limit_ns) return false;
    }
}

// The same by every lane of a warp, with one answer.
FE_DEV bool lin_wait_warp(uint32_t bar, uint32_t parity, unsigned long long limit_ns = kLinTimeoutNs)
{
    return __all_sync(0xffffffffu, lin_wait(bar, parity, limit_ns));
}

// One lane of a converged warp.  The producer and MMA warps run their loops with every lane and pick
// the issuing one only around the instruction, so that addresses and descriptors stay warp-uniform: a
// loop entered by lane 0 alone took 720 cycles per k step whatever the tile's width.
FE_DEV bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Position in a ring of S stages: the stage and the parity of its current round.
struct RingPos {
    uint32_t s, parity;
    bool full_round;   // the ring has been filled once
    FE_DEV RingPos() : s(0), parity(0), full_round(false) {}
    FE_DEV void next(uint32_t S)
    {
        if (++s == S) {
            s = 0;
            parity ^= 1;
            full_round = true;
        }
    }
};

FE_DEV void expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

// Descriptor of an operand stored across the contraction: boxes of 64 (M or N) x 64 k, one 128-byte
// row per k, 8-k groups 1024 bytes apart, the next 64 of M or N one box further.
FE_DEV uint64_t lin_desc_mn(uint32_t saddr)
{
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
    d |= (uint64_t)(8192u >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// f32 accumulator, bf16 operands, which of them lie across the contraction, N and M.
FE_DEV uint32_t lin_idesc(int a_mn, int b_mn, int M, int N)
{
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

FE_DEV void tc_mma_pair(uint32_t tmem_d, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_d),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

// Arrives on the barrier at this offset in both CTAs once the MMAs so far are done.
FE_DEV void tc_commit_pair(uint32_t mbar)
{
    asm volatile(
        "{\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\t"
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(mbar)
        : "memory");
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

// v[j] += bias[c0 + j] for c0 + j < cols; every lane has the same columns.
FE_DEV void lin_add_bias(const uint16_t* bias, int c0, int cols, float (&v)[32])
{
    const uint16_t* b = bias + c0;
    if (c0 + 32 <= cols && (reinterpret_cast<uintptr_t>(b) & 15) == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint4 w = __ldg(reinterpret_cast<const uint4*>(b) + q);
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
            if (c0 + j < cols) v[j] += bf16_bits_to_f32(b[j]);
    }
}

// A staging slot holds 32 rows of 32 bf16 (64 bytes) in TMA's 64-byte swizzle: 16-byte chunk c of row
// r is stored at chunk c ^ (r / 2 % 4), so the eight rows of an access phase use every bank once.
FE_DEV uint32_t lin_slot_chunk(int r, int c) { return (uint32_t)r * 64u + (uint32_t)((c ^ ((r >> 1) & 3)) << 4); }

// The epilogue's view of one warp's staging: 32 x 32 blocks of bf16 go out (or a residual comes in)
// through slots, by TMA where the matrix suits it, else row by row with the lanes along a row.
struct LinStage {
    uint8_t* base;
    uint32_t saddr;
    uint32_t ny;   // slots given out to y

    // A slot may be written again once at most `pending` of the latest stores still read theirs.
    template <int PENDING>
    FE_DEV void settle() const
    {
        if ((threadIdx.x & 31) == 0) bulk_wait_read<PENDING>();
        __syncwarp();
    }

    FE_DEV void put(int slot, int lane, const float (&v)[32]) const
    {
        uint8_t* p = base + slot * kLinSlotBytes;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            *reinterpret_cast<uint4*>(p + lin_slot_chunk(lane, q)) =
                make_uint4(bf16x2_rn(v[8 * q], v[8 * q + 1]), bf16x2_rn(v[8 * q + 2], v[8 * q + 3]),
                           bf16x2_rn(v[8 * q + 4], v[8 * q + 5]), bf16x2_rn(v[8 * q + 6], v[8 * q + 7]));
    }

    FE_DEV void add(int slot, int lane, float (&v)[32]) const
    {
        const uint8_t* p = base + slot * kLinSlotBytes;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint4 w = *reinterpret_cast<const uint4*>(p + lin_slot_chunk(lane, q));
            const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[8 * q + 2 * j] += __uint_as_float(a[j] << 16);
                v[8 * q + 2 * j + 1] += __uint_as_float(a[j] & 0xffff0000u);
            }
        }
    }

    FE_DEV uint16_t* at(int slot, int r, int col) const
    {
        return reinterpret_cast<uint16_t*>(base + slot * kLinSlotBytes + lin_slot_chunk(r, col >> 3)) + (col & 7);
    }

    // Block (row0, col0) of a matrix with row stride ld from a slot; columns from `limit` on are not the block's: a
    // swiglu z's other half begins there, or the matrix ends (`ends`: after whole 16-byte pieces, where TMA
    // stops by itself; within a piece it would write the rest of the piece too).
    FE_DEV void flush(int slot, int lane, const CUtensorMap* map, bool vec, bool ends, uint16_t* m, int64_t ld, int row0,
                      int rows, int col0, int limit) const
    {
        if (vec && (ends || col0 + 32 <= limit)) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) tma_store_2d(map, col0, row0, saddr + slot * kLinSlotBytes);
        } else {
            __syncwarp();
            if (col0 + lane < limit)
                for (int r = 0; r < 32 && row0 + r < rows; ++r) m[(size_t)(row0 + r) * ld + col0 + lane] = *at(slot, r, lane);
            __syncwarp();
            // a group for this block as well: settle() counts blocks
            if (vec && lane == 0) asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }

    FE_DEV void fill(int slot, int lane, const uint16_t* m, int64_t ld, int row0, int rows, int col0, int cols) const
    {
        for (int r = 0; r < 32; ++r)
            *at(slot, r, lane) = row0 + r < rows && col0 + lane < cols ? m[(size_t)(row0 + r) * ld + col0 + lane] : 0;
        __syncwarp();
    }
};

// The tiles of problem i that a CTA pair works on: round robin over a single problem, its share of two.
struct LinRange {
    int t, end, step;
    FE_DEV LinRange(const LinParams& P, int i, int pair, int pairs)
        : t(P.n == 1 ? pair : P.start[i][pair]), end(P.n == 1 ? P.p[i].tiles : P.start[i][pair + 1]), step(P.n == 1 ? pairs : 1)
    {
    }
};

// 256 x BN output tiles by pairs of CTAs (one MMA over two SMs: each holds 128 rows of A and half of
// B's columns, so a k step moves 32 KB into each SM for 512 cycles of products; a single CTA's
// 128 x 256 tile would move 48 KB and measured 20 % slower).  Counters at 16384 x 1536, K = 2048: tensor
// pipe 85 % of cycles, 81 MB of DRAM for 99 MB of operands and output.  What is left: the first tile's loads and
// the last one's epilogue, 4 us a launch, and power.
template <int BN, bool PLAIN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kLinThreads, 1)
    linear_gemm_kernel(const __grid_constant__ LinParams P)
{
    constexpr int S = lin_stages(BN, PLAIN), kLinBars = lin_bars(BN, PLAIN), kLinSlots = lin_slots(PLAIN);
    constexpr uint32_t kLinStage = lin_stage(BN);
    constexpr int kAccStride = 256;
    constexpr uint32_t kTmemCols = BN > 128 ? 512 : 256;
    constexpr uint32_t kAccCol = BN > 128 ? kAccStride : 128;
    extern __shared__ uint8_t lin_dyn[];
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const uint32_t rank = cluster_rank();
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    const uint32_t base0 = tc_saddr(lin_dyn);
    uint8_t* sm = lin_dyn + ((1024u - (base0 & 1023u)) & 1023u);
    const uint32_t ring = tc_saddr(sm);
    uint8_t* staging = sm + S * kLinStage;
    uint64_t* bars = reinterpret_cast<uint64_t*>(staging + 8 * kLinSlots * kLinSlotBytes);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kLinBars);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t bar0 = tc_saddr(bars);
    auto full = [&](int s) { return bar0 + 8u * s; };                   // pair's leader: bytes of both CTAs landed
    auto empty = [&](int s) { return bar0 + 8u * (S + s); };            // both: the stage's MMAs are done
    auto accfull = [&](int s) { return bar0 + 8u * (2 * S + s); };      // both: a tile's products are done
    auto accempty = [&](int s) { return bar0 + 8u * (2 * S + 2 + s); }; // leader: both CTAs drained it
    auto resfull = [&](int w, int s) { return bar0 + 8u * (2 * S + 4 + 2 * w + s); };
    if (tid < kLinBars) {
        tc_mbar_init(bar0 + 8u * tid, tid == 2 * S + 2 || tid == 2 * S + 3 ? 16 : 1);   // accempty: both CTAs' 8 warps
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 64) *abort = 0;
    if (tid >= 96 && tid < 96 + 2 * P.n) prefetch_tensormap(tid & 1 ? &P.p[(tid - 96) >> 1].tb : &P.p[(tid - 96) >> 1].ta);
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc_saddr(tmem_slot)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();   // both CTAs' barriers are ready before either signals the other
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();
    griddep_launch();   // the next launch's CTAs start as these end

    if (warp == 0) {
        // ---- producer: this CTA's boxes of A and B into its ring, reported to the leader ------------
        RingPos at;
        uint32_t loads = 0;
        for (int i = 0; i < P.n; ++i) {
            const LinProblem& p = P.p[i];
            const int nk = (p.K + 63) / 64, tiles_n = p.tiles_n, a_mn = p.a_mn, b_mn = p.b_mn, cols = p.cols;
            const bool glu = p.act == kActSwiglu;
            const CUtensorMap *ta = &p.ta, *tb = &p.tb;
            const uint32_t bytes = 2 * (kLinABytes + (b_mn ? (BN / 2 + 63) / 64 * 8192u : BN / 2 * 128u));
            for (LinRange g(P, i, pair, pairs); g.t < g.end && !*abort; g.t += g.step) {
                const int m0 = g.t / tiles_n * kLinM + 128 * rank, tn = g.t % tiles_n;
                // swiglu: the leader's columns are gate rows of W, the other's the up rows of the same
                // output columns
                const int n0 = glu ? tn * (BN / 2) + (rank ? cols : 0) : tn * BN + (BN / 2) * rank;
                for (int k = 0; k < nk; ++k, at.next(S), ++loads) {
                    const uint32_t s = at.s;
                    if (at.full_round && !lin_wait_warp(empty(s), at.parity ^ 1)) {
                        *abort = 1;
                        break;
                    }
                    if (elect_one()) {
                        if (rank == 0) expect_tx(full(s), bytes);
                        const uint32_t bar = cluster_map(full(s), 0);
                        const uint32_t a = ring + s * kLinStage, b = a + kLinABytes;
                        if (a_mn) {
                            tma_load_2d_pair(a, ta, m0, 64 * k, bar);
                            tma_load_2d_pair(a + 8192, ta, m0 + 64, 64 * k, bar);
                        } else {
                            tma_load_2d_pair(a, ta, 64 * k, m0, bar);
                        }
                        if (b_mn) {
#pragma unroll
                            for (int j = 0; j < (BN / 2 + 63) / 64; ++j)
                                tma_load_2d_pair(b + j * 8192, tb, n0 + 64 * j, 64 * k, bar);
                        } else {
                            tma_load_2d_pair(b, tb, 64 * k, n0, bar);
                        }
                    }
                    __syncwarp();
                }
            }
        }
        // no copy outlives the loop: the leader sees those of both CTAs land
        if (rank == 0)
            for (uint32_t j = loads > S ? loads - S : 0; j < loads; ++j) lin_wait_warp(full(j % S), (j / S) & 1);
    } else if (warp == 1) {
        if (rank == 0) {
            // ---- MMA issue, for both CTAs ------------------------------------------------------------
            RingPos at;
            uint32_t done = 0;
            for (int i = 0; i < P.n; ++i) {
                const LinProblem& p = P.p[i];
                const int nk = (p.K + 63) / 64, a_mn = p.a_mn, b_mn = p.b_mn;
                const uint32_t idesc = lin_idesc(a_mn, b_mn, kLinM, BN);
                const uint64_t a0 = a_mn ? lin_desc_mn(ring) : tc_smem_desc(ring);
                const uint64_t b0 = b_mn ? lin_desc_mn(ring + kLinABytes) : tc_smem_desc(ring + kLinABytes);
                const uint32_t as = a_mn ? 2048 / 16 : 32 / 16, bs = b_mn ? 2048 / 16 : 32 / 16;   // 16 of k further
                for (LinRange g(P, i, pair, pairs); g.t < g.end && !*abort; g.t += g.step, ++done) {
                    const int acc = done & 1;
                    if (done >= 2 && !lin_wait_warp(accempty(acc), (done / 2 - 1) & 1)) *abort = 1;
                    tc_fence_after();
                    for (int k = 0; k < nk && !*abort; ++k, at.next(S)) {
                        const uint32_t s = at.s;
                        if (!lin_wait_warp(full(s), at.parity)) {
                            *abort = 1;
                            break;
                        }
                        tc_fence_after();
                        if (elect_one()) {
                            const uint64_t a = a0 + s * (kLinStage >> 4), b = b0 + s * (kLinStage >> 4);
#pragma unroll
                            for (int ks = 0; ks < 4; ++ks)
                                tc_mma_pair(tmem + kAccCol * acc, a + ks * as, b + ks * bs, idesc, (k > 0 || ks > 0) ? 1u : 0u);
                            tc_commit_pair(empty(s));
                        }
                        __syncwarp();
                    }
                    if (elect_one()) tc_commit_pair(accfull(acc));
                    __syncwarp();
                }
            }
            // never leave with MMAs in flight: they read shared memory and write TMEM
            for (uint32_t j = done > 2 ? done - 2 : 0; j < done; ++j)
                if (!lin_wait_warp(accfull(j & 1), (j / 2) & 1)) *abort = 1;
        }
    } else if (warp >= 4) {
        // ---- epilogue: a thread per row, blocks of 32 columns through the staging slots; the two
        // warps of a TMEM quarter take every other block (with one warp an SM sub-partition had
        // nothing to run under its latencies: 1300 cycles a block)
        const int ew = warp - 4, quarter = ew & 3, half = ew >> 2;
        LinStage st{staging + ew * kLinSlots * kLinSlotBytes, tc_saddr(staging + ew * kLinSlots * kLinSlotBytes), 0};
        uint32_t done = 0, nres = 0;
        bool stop = false;
        for (int i = 0; i < P.n && !stop; ++i) {
            const LinProblem& p = P.p[i];
            // operands in registers: the loops' memory clobbers would reload them each time
            const int act = p.act, M = p.M, N = p.N, cols = p.cols, tiles_n = p.tiles_n;
            const bool vec_out = p.vec_out, vec_z = p.vec_z, vec_res = p.vec_res;
            const uint16_t *bias = p.bias, *res = p.res;
            uint16_t *out = p.out, *zo = p.z;
            const int64_t ldr = p.ldr, ldo = p.ldo;
            const CUtensorMap *to = &p.to, *tr = &p.tr, *tz = &p.tz;
            const bool glu = !PLAIN && act == kActSwiglu, ends = cols % 8 == 0;
            const int tile_cols = glu ? BN / 2 : BN;
            st.settle<0>();   // the problem before may have used the slots another way
            for (LinRange g(P, i, pair, pairs); g.t < g.end; g.t += g.step, ++done) {
                const int acc = done & 1;
                const int row0 = g.t / tiles_n * kLinM + 128 * rank + 32 * quarter, n0 = g.t % tiles_n * tile_cols;
                const int chunks = min(tile_cols, cols - n0 + 31) / 32;   // blocks with a column to write
                const bool live = row0 < M;
                // a residual block is fetched one block ahead; nres counts the fetches by TMA
                const bool has_res = !PLAIN && res && live, tma_res = has_res && vec_res;
                auto fetch = [&](int c) {
                    const int slot = st.ny++ & 1;
                    st.settle<0>();
                    if (tma_res) {
                        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                        __syncwarp();
                        if (lane == 0) {
                            expect_tx(resfull(ew, nres & 1), kLinSlotBytes);
                            tma_load_2d(st.saddr + slot * kLinSlotBytes, tr, n0 + 32 * c, row0, resfull(ew, nres & 1));
                        }
                        ++nres;
                    } else {
                        st.fill(slot, lane, res, ldr, row0, M, n0 + 32 * c, cols);
                    }
                    return slot;
                };
                int slot = 0;
                if (has_res && half < chunks) slot = fetch(half);
                // a whole tile's products: a dW's run over every row, some 200 ns per k step
                if (!lin_wait_warp(accfull(acc), (done / 2) & 1, kLinTimeoutNs + 1000ull * ((p.K + 63) / 64))) *abort = 1;
                stop = __any_sync(0xffffffffu, *abort != 0);
                tc_fence_after();
                const uint32_t t0 = tmem + ((uint32_t)(32 * quarter) << 16) + kAccCol * acc;
#pragma unroll 1
                for (int c = half; c < chunks; c += 2) {
                    uint32_t r[32];
                    float v[32];
                    tc_ld32(t0 + 32 * c, r);
                    const int c0 = n0 + 32 * c;
                    tc_wait_ld();
#pragma unroll
                    for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
                    if (!PLAIN) {
                        if (glu) {
                            tc_ld32(t0 + BN / 2 + 32 * c, r);
                            tc_wait_ld();
                            float u[32];
#pragma unroll
                            for (int j = 0; j < 32; ++j) u[j] = __uint_as_float(r[j]);
                            if (bias) {
                                lin_add_bias(bias, c0, cols, v);
                                lin_add_bias(bias + cols, c0, cols, u);
                            }
                            if (zo && live && !stop) {   // slots 2 and 3 are z's
                                st.settle<0>();
                                st.put(2, lane, v);
                                st.flush(2, lane, tz, vec_z, false, zo, N, row0, M, c0, cols);
                                st.put(3, lane, u);
                                st.flush(3, lane, tz, vec_z, true, zo, N, row0, M, c0 + cols, N);
                            }
#pragma unroll
                            for (int j = 0; j < 32; ++j) v[j] = v[j] * sigmoidf(v[j]) * u[j];
                        } else {
                            if (bias) lin_add_bias(bias, c0, cols, v);
                            if (zo && live && !stop) {
                                st.settle<0>();
                                st.put(2, lane, v);
                                st.flush(2, lane, tz, vec_z, true, zo, N, row0, M, c0, cols);
                            }
                            act_all<32>(act, v);
                        }
                        if (has_res) {
                            const uint32_t turn = nres - 1;   // this block's fetch
                            if (tma_res && !lin_wait_warp(resfull(ew, turn & 1), (turn >> 1) & 1)) {
                                *abort = 1;
                                lin_wait_warp(resfull(ew, turn & 1), (turn >> 1) & 1);   // it must not outlive the slot
                            }
                            st.add(slot, lane, v);
                            // the next block's residual goes to the other slot, whose store has been read by then
                            if (c + 2 < chunks) {
                                const int ahead = fetch(c + 2);
                                if (live && !stop) {
                                    st.put(slot, lane, v);
                                    st.flush(slot, lane, to, vec_out, ends, out, ldo, row0, M, c0, cols);
                                }
                                slot = ahead;
                                continue;
                            }
                        }
                    }
                    if (live && !stop) {
                        if (!has_res) {
                            // the slots go round, or two beside z's: all later stores but the one before last may be reading
                            if (!PLAIN && zo) {
                                slot = st.ny++ & 1;
                                st.settle<0>();
                            } else {
                                slot = st.ny++ & (kLinSlots - 1);
                                st.settle<kLinSlots - 1>();
                            }
                        }
                        st.put(slot, lane, v);
                        st.flush(slot, lane, to, vec_out, ends, out, ldo, row0, M, c0, cols);
                    }
                }
                // the accumulator is read: the products after the next may begin
                tc_fence_before();
                __syncwarp();
                if (lane == 0)   // nothing in memory goes with it: a release to the cluster would wait for the stores
                    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_map(accempty(acc), 0)) : "memory");
                if (stop) break;
            }
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (tid == 0 && *abort) atomicOr(&g_op_status, kDevTcTimeout);
    cluster_sync();   // the pair's shared memory and TMEM are in use until both are here
    if (warp == 2) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

// ---- few tiles: the contraction split over a cluster --------------------------------------

constexpr int kSplMaxStages = 7;
constexpr int kSplThreads = 256;              // warp 0: TMA, 1: MMA, 2: TMEM, 4-7: residual; then all finish
// A tile's columns are BN (64 or 128): for swiglu half of them gate columns, half their up columns.
__host__ __device__ constexpr uint32_t spl_stage(int BN) { return 128 * 128 + BN * 128; }
__host__ __device__ constexpr int spl_ld(int BN) { return BN + 4; }   // fp32 rows: 16-byte accesses of 8 rows hit every bank
__host__ __device__ constexpr uint32_t spl_part(int BN) { return 128 * spl_ld(BN) * 4; }   // [splits][128 / splits] partial rows
// Shared memory for `stages` stages: short contractions take few, so that CTAs of consecutive launches fit
// an SM together.  res: bytes of the finished rows' residual.
__host__ __device__ constexpr uint32_t spl_smem(int BN, int stages, uint32_t res)
{
    return 1024 + stages * spl_stage(BN) + spl_part(BN) + res + 8 * (2 * stages + 1) + 16;
}

struct LinSplitParams {
    CUtensorMap ta, tb;      // x: boxes of 64 k x 128 rows; w: 64 k x BN / 2 rows
    int M, N, K, splits, stages, act, cols;
    int vec_res;             // residual rows in 16-byte pieces
    uint32_t res_bytes;      // of shared memory for the residual
    const uint16_t* bias;
    const uint16_t* res;
    int64_t ldr;
    uint16_t* out;
    int64_t ldo;
    uint16_t* z;
};

// A thread's four columns of a row: consecutive ones where rows are 8-byte aligned (VEC), else `step` apart, so
// that the lanes of a row write consecutive halfwords.
template <bool VEC>
FE_DEV void spl_store4(uint16_t* o, int step, int left, const float (&v)[4])
{
    const uint32_t a = bf16x2_rn(v[0], v[1]), b = bf16x2_rn(v[2], v[3]);
    if (VEC) {
        *reinterpret_cast<uint2*>(o) = make_uint2(a, b);
    } else {
        o[0] = (uint16_t)a;
        if (left > step) o[step] = (uint16_t)(a >> 16);
        if (left > 2 * step) o[2 * step] = (uint16_t)b;
        if (left > 3 * step) o[3 * step] = (uint16_t)(b >> 16);
    }
}

// v += four bf16, the same way.
template <bool VEC>
FE_DEV void spl_add4(const uint16_t* s, int step, int left, float (&v)[4])
{
    if (VEC) {
        const uint2 q = *reinterpret_cast<const uint2*>(s);
        v[0] += __uint_as_float(q.x << 16);
        v[1] += __uint_as_float(q.x & 0xffff0000u);
        v[2] += __uint_as_float(q.y << 16);
        v[3] += __uint_as_float(q.y & 0xffff0000u);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (left > j * step) v[j] += bf16_bits_to_f32(s[j * step]);
    }
}

template <bool VEC>
FE_DEV void spl_sum4(const float* s, int step, float (&v)[4])
{
    if (VEC) {
        const float4 q = *reinterpret_cast<const float4*>(s);
        v[0] += q.x; v[1] += q.y; v[2] += q.z; v[3] += q.w;
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] += s[j * step];
    }
}

// The rows that a CTA of the cluster finishes: their partials added in rank order, then the epilogue, several rows
// of a thread at a time so that their loads do not wait for each other's stores.
template <bool GLU, int BN, bool VEC>
FE_DEV void spl_finish(const LinSplitParams& p, const float* part, const uint16_t* res, int m0, int tn, int rows, int rank)
{
    constexpr int W = GLU ? BN / 2 : BN, TPR = W / 4, LD = spl_ld(BN), STEP = VEC ? 1 : TPR, R = BN / 32, ROWS = kSplThreads / TPR;
    const int tid = threadIdx.x, lg = 31 - __clz(p.splits), per = 128 >> lg;
    const int cc = (VEC ? 4 : 1) * (tid % TPR), col0 = tn * W + cc, left = p.cols - col0;
    if (left <= 0) return;
    // a thread's columns are the same in every row: the bias once
    float bv[4] = {0, 0, 0, 0}, bu[4] = {0, 0, 0, 0};
    if (p.bias) {
        spl_add4<false>(p.bias + col0, STEP, left, bv);
        if (GLU) spl_add4<false>(p.bias + p.cols + col0, STEP, left, bu);
    }
#pragma unroll 1
    for (int i0 = tid / TPR; i0 < per && (i0 << lg) + rank < rows; i0 += R * ROWS) {
        float v[R][4], u[R][4];
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[r][j] = bv[j];
                u[r][j] = bu[j];
            }
#pragma unroll 1
        for (int s = 0; s < p.splits; ++s) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float* from = part + (s * per + min(i0 + r * ROWS, per - 1)) * LD + cc;
                spl_sum4<VEC>(from, STEP, v[r]);
                if (GLU) spl_sum4<VEC>(from + W, STEP, u[r]);
            }
        }
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int i = i0 + r * ROWS, row = (i << lg) + rank;
            if (i >= per || row >= rows) break;
            const size_t grow = (size_t)(m0 + row);
            if (p.z) {
                spl_store4<VEC>(p.z + grow * p.N + col0, STEP, left, v[r]);
                if (GLU) spl_store4<VEC>(p.z + grow * p.N + p.cols + col0, STEP, left, u[r]);
            }
            if (GLU) {
#pragma unroll
                for (int j = 0; j < 4; ++j) v[r][j] *= sigmoidf(v[r][j]) * u[r][j];
            } else {
                act_all<4>(p.act, v[r]);
            }
            if (p.res) spl_add4<VEC>(res + i * W + cc, STEP, left, v[r]);
            spl_store4<VEC>(p.out + grow * p.ldo + col0, STEP, left, v[r]);
        }
    }
}

// One 128 x BN tile per cluster of `splits` CTAs (a power of two), each over its share of the k steps.
// Row i of a CTA's partial tile goes through distributed shared memory to CTA i % splits, which adds
// that row's partials in rank order and finishes it.  For products of so few tiles that whole tiles
// would leave most SMs idle while the operands stream through the rest.  Rows are sent, not fetched: a
// store needs no answer, and nothing is read across CTAs after the one barrier (fetching cost 3 us a
// launch).  The finish is a short loop: code that runs once is bound by fetching its instructions.  The
// residual of the finished rows is brought into shared memory while the products run.
template <bool GLU, int BN, bool VEC>
__global__ void __launch_bounds__(kSplThreads) linear_split_kernel(const __grid_constant__ LinSplitParams p)
{
    constexpr uint32_t kSplStage = spl_stage(BN);
    constexpr int LD = spl_ld(BN), W = GLU ? BN / 2 : BN;
    const uint32_t S = p.stages;
    extern __shared__ uint8_t lin_dyn[];
    const int tid = threadIdx.x, lane = tid & 31, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    const int m0 = blockIdx.y * 128, tn = blockIdx.x;
    const uint32_t rank = blockIdx.z;
    const int nk = (p.K + 63) / 64;
    const int k0 = (int)((int64_t)nk * rank / p.splits), k1 = (int)((int64_t)nk * (rank + 1) / p.splits);
    const uint32_t base0 = tc_saddr(lin_dyn);
    uint8_t* sm = lin_dyn + ((1024u - (base0 & 1023u)) & 1023u);
    const uint32_t ring = tc_saddr(sm);
    float* part = reinterpret_cast<float*>(sm + S * kSplStage);
    uint16_t* res = reinterpret_cast<uint16_t*>(sm + S * kSplStage + spl_part(BN));   // [128 / splits][W]
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + S * kSplStage + spl_part(BN) + p.res_bytes);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S + 1);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t bar0 = tc_saddr(bars);
    auto full = [&](uint32_t s) { return bar0 + 8u * s; };
    auto empty = [&](uint32_t s) { return bar0 + 8u * (S + s); };
    const uint32_t accfull = bar0 + 8u * 2 * S;
    const int rows = min(128, p.M - m0), lg = 31 - __clz(p.splits), per = 128 >> lg;
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");   // this CTA runs: its memory may be written
    if (tid <= 2 * (int)S) {
        tc_mbar_init(bar0 + 8u * tid, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (tid == 32) *abort = 0;
    if (tid >= 96 && tid < 98) prefetch_tensormap(tid == 96 ? &p.ta : &p.tb);
    if (warp == 2) {
        tc_alloc(tc_saddr(tmem_slot), BN);
        tc_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    griddep_wait();
    griddep_launch();
    if (warp == 0) {
        const int n0 = tn * W, n1 = GLU ? n0 + p.cols : n0 + BN / 2;
        RingPos ri;
        uint32_t i = 0;
        for (int k = k0; k < k1; ++k, ++i, ri.next(S)) {
            const uint32_t s = ri.s;
            if (ri.full_round && !lin_wait_warp(empty(s), ri.parity ^ 1)) {
                *abort = 1;
                break;
            }
            if (elect_one()) {
                expect_tx(full(s), kSplStage);
                const uint32_t a = ring + s * kSplStage, b = a + 128 * 128;
                tma_load_2d(a, &p.ta, 64 * k, m0, full(s));
                tma_load_2d(b, &p.tb, 64 * k, n0, full(s));
                tma_load_2d(b + BN / 2 * 128, &p.tb, 64 * k, n1, full(s));
            }
            __syncwarp();
        }
        for (uint32_t j = i > S ? i - S : 0; j < i; ++j) lin_wait_warp(full(j % S), (j / S) & 1);
    } else if (warp == 1) {
        const uint32_t idesc = lin_idesc(0, 0, 128, BN);
        const uint64_t a0 = tc_smem_desc(ring), b0 = tc_smem_desc(ring + 128 * 128);
        RingPos ri;
        for (int k = k0; k < k1; ++k, ri.next(S)) {
            const uint32_t s = ri.s;
            if (!lin_wait_warp(full(s), ri.parity)) {
                *abort = 1;
                break;
            }
            tc_fence_after();
            if (elect_one()) {
                const uint64_t a = a0 + s * (kSplStage >> 4), b = b0 + s * (kSplStage >> 4);
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
                    tc_mma_f16(tmem, a + 2 * ks, b + 2 * ks, idesc, (k > k0 || ks > 0) ? 1u : 0u);
                tc_commit(empty(s));
            }
            __syncwarp();
        }
        if (elect_one()) tc_commit(accfull);
        __syncwarp();
        if (!lin_wait_warp(accfull, 0)) *abort = 1;
    } else if (warp >= 4 && p.res) {
        const int left = min(W, p.cols - tn * W);   // this tile's columns
        const uint16_t* src = p.res + (size_t)m0 * p.ldr + tn * W;
        if (p.vec_res) {
            constexpr int C = W / 8;
#pragma unroll 4
            for (int i = tid - 128; i < per * C; i += 128) {
                const int row = ((i / C) << lg) + rank, c = 8 * (i % C);
                if (row < rows && c < left)
                    *reinterpret_cast<uint4*>(res + 8 * i) = *reinterpret_cast<const uint4*>(src + (size_t)row * p.ldr + c);
            }
        } else {
#pragma unroll 8
            for (int i = tid - 128; i < per * W; i += 128) {
                const int row = ((i / W) << lg) + rank, c = i % W;
                if (row < rows && c < left) res[i] = src[(size_t)row * p.ldr + c];
            }
        }
    }
    __syncthreads();   // the products are done
    tc_fence_after();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");   // every CTA of the cluster runs
#pragma unroll
    for (int h = 0; h < BN / 64; ++h) {
        const int row = 32 * (warp & 3) + lane, c = 32 * (warp >> 2) + 64 * h;
        uint32_t r[32];
        tc_ld32(tmem + ((uint32_t)(32 * (warp & 3)) << 16) + c, r);
        tc_wait_ld();
        if (row < rows) {
            const uint32_t to = cluster_map(tc_saddr(part + (rank * per + (row >> lg)) * LD + c), row & (p.splits - 1));
#pragma unroll
            for (int q = 0; q < 8; ++q)
                asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + 16 * q), "r"(r[4 * q]),
                             "r"(r[4 * q + 1]), "r"(r[4 * q + 2]), "r"(r[4 * q + 3])
                             : "memory");
        }
    }
    tc_fence_before();
    cluster_sync();
    if (warp == 2) {
        tc_fence_after();
        tc_dealloc(tmem, BN);
    }
    spl_finish<GLU, BN, VEC>(p, part, res, m0, tn, rows, rank);
    if (tid == 0 && *abort) atomicOr(&g_op_status, kDevTcTimeout);
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

// One row of x: a warp per output column (two weight rows for swiglu).  A second row's loads would take the
// registers that keep this one's weights in flight; from two rows on the kernel below is faster.
template <bool GLU>
__global__ void __launch_bounds__(32 * kLinRowsWarps) linear_rows_kernel(LinRowsParams p)
{
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31;
    const int c = blockIdx.x * kLinRowsWarps + (threadIdx.x >> 5);
    if (c >= p.cols) return;
    const uint16_t* w0 = p.w + (size_t)c * p.K;
    const uint16_t* w1 = p.w + (size_t)(c + p.cols) * p.K;   // read for swiglu only
    float z0 = 0.0f, z1 = 0.0f;
#pragma unroll 4
    for (int k = 8 * lane; k < p.K; k += 256) {
        const uint4 a = ldg_stream(w0 + k);
        uint4 b = make_uint4(0, 0, 0, 0);
        if (GLU) b = ldg_stream(w1 + k);
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(p.x + k));
        fma8(a, x, z0);
        if (GLU) fma8(b, x, z1);
    }
    z0 = warp_sum(z0);
    if (GLU) z1 = warp_sum(z1);
    if (lane != 0) return;
    if (p.bias) {
        z0 += bf16_bits_to_f32(p.bias[c]);
        if (GLU) z1 += bf16_bits_to_f32(p.bias[c + p.cols]);
    }
    if (p.z) {
        p.z[c] = (uint16_t)(bf16x2_rn(z0, 0.0f) & 0xffffu);
        if (GLU) p.z[c + p.cols] = (uint16_t)(bf16x2_rn(z1, 0.0f) & 0xffffu);
    }
    float v = GLU ? z0 * sigmoidf(z0) * z1 : act_fwd(p.act, z0);
    if (p.res) v += bf16_bits_to_f32(p.res[c]);
    p.y[c] = (uint16_t)(bf16x2_rn(v, 0.0f) & 0xffffu);
}

// ---- a small batch ---------------------------------------------------------------------

// Rows to which the kernel below is taken.  Every CTA reads all of x, so that more rows are faster in tiles: N = 1536,
// K = 2048 takes 4.0 us at 16 rows (tiles 5.0), 8.8 at 32 (tiles 5.4); N = 4096, K = 1024 4.0 at 16 (tiles 6.0), 3.0 at 2
// (6.2).  A warp walks the contraction 512 of k at a time, so a long one is faster in tiles as well, which split it: N =
// 512, K = 4096 takes 6.1 us at 16 rows (tiles 4.3) and 5.0 at 2 (tiles 4.1); the rule does not look at K.
constexpr int kSkinnyMaxM = 16;

FE_DEV void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A CTA per 16 rows of W (swiglu: 8 gate rows and their up rows) against up to 8 NT rows of x: W's rows
// are the M side of m16n8k16, x's the N side.  The warps share the contraction, 64 of k at a time, and
// add their sums through shared memory in warp order.  A lane feeds both operands from 16-byte runs of
// a row, so the MMAs see k in another order, the same for both.  What bounds it is the latency of one
// pass over the weights: everything a warp needs of its share is in flight at once, and no tile, TMA or
// cluster set-up stands before it.
template <int NT, bool GLU>
__global__ void __launch_bounds__(256) linear_skinny_kernel(LinRowsParams p)
{
    constexpr int LD = 8 * NT + 1, C = GLU ? 8 : 16;
    __shared__ float red[8][16][LD];
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int c0 = blockIdx.x * C;
    const bool lo_on = c0 + g < p.cols, hi_on = GLU ? lo_on : c0 + 8 + g < p.cols;
    const uint16_t* wlo = p.w + (size_t)(lo_on ? c0 + g : 0) * p.K;
    const uint16_t* whi = p.w + (size_t)(hi_on ? (GLU ? p.cols + c0 + g : c0 + 8 + g) : 0) * p.K;
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll(NT <= 2 ? 4 : 2)
    for (int kb = 64 * warp; kb < p.K; kb += 512) {
        uint4 lo[2], hi[2], x[2][NT];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int k = kb + 32 * h + 8 * t;
            const bool in = k < p.K;   // K is a multiple of 8
            lo[h] = in && lo_on ? ldg_stream(wlo + k) : zero;
            hi[h] = in && hi_on ? ldg_stream(whi + k) : zero;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int m = 8 * n + g;
                x[h][n] = in && m < p.M ? __ldg(reinterpret_cast<const uint4*>(p.x + (size_t)m * p.ldx + k)) : zero;
            }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                mma_bf16(acc[n], lo[h].x, hi[h].x, lo[h].y, hi[h].y, x[h][n].x, x[h][n].y);
                mma_bf16(acc[n], lo[h].z, hi[h].z, lo[h].w, hi[h].w, x[h][n].z, x[h][n].w);
            }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
        float* r = &red[warp][g][8 * n + 2 * t];
        r[0] = acc[n][0];
        r[1] = acc[n][1];
        r[8 * LD] = acc[n][2];
        r[8 * LD + 1] = acc[n][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < C * p.M; i += 256) {
        const int c = i % C, m = i / C, col = c0 + c;
        if (col >= p.cols) continue;
        float z0 = 0.0f, z1 = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            z0 += red[w][c][m];
            if (GLU) z1 += red[w][c + 8][m];
        }
        if (p.bias) {
            z0 += bf16_bits_to_f32(p.bias[col]);
            if (GLU) z1 += bf16_bits_to_f32(p.bias[col + p.cols]);
        }
        if (p.z) {
            p.z[(size_t)m * p.N + col] = (uint16_t)(bf16x2_rn(z0, 0.0f) & 0xffffu);
            if (GLU) p.z[(size_t)m * p.N + col + p.cols] = (uint16_t)(bf16x2_rn(z1, 0.0f) & 0xffffu);
        }
        float v = GLU ? z0 * sigmoidf(z0) * z1 : act_fwd(p.act, z0);
        if (p.res) v += bf16_bits_to_f32(p.res[(size_t)m * p.ldr + col]);
        p.y[(size_t)m * p.ldy + col] = (uint16_t)(bf16x2_rn(v, 0.0f) & 0xffffu);
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
    int N, cols;
};

template <int VEC>
struct DzWord {
    using T = uint16_t;
};
template <>
struct DzWord<8> {
    using T = uint4;
};

template <int VEC>
FE_DEV void dz_unpack(const typename DzWord<VEC>::T& q, float (&v)[VEC])
{
    if constexpr (VEC == 8) {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < VEC; ++j) v[j] = __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    } else {
        v[0] = bf16_bits_to_f32(q);
    }
}

template <int VEC>
FE_DEV void dz_store(uint16_t* p, const float (&v)[VEC])
{
    if constexpr (VEC == 8)
        *reinterpret_cast<uint4*>(p) =
            make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
    else
        *p = (uint16_t)(bf16x2_rn(v[0], 0.0f) & 0xffffu);
}

constexpr int kDzRows = 2;   // rows a thread has in flight

// Block 32 x 8: a thread owns VEC columns, 8 threads share the rows of a chunk.  Bound by memory: dY and
// Z are read once, dZ written once, so a thread keeps two rows' loads in flight and an SM 16 warps.
template <int VEC, int ACT>
__global__ void __launch_bounds__(256, 2) linear_dz_kernel(LinDzParams p)
{
    using W = typename DzWord<VEC>::T;
    __shared__ float red[8][2 * VEC][33];
    griddep_wait();
    griddep_launch();
    const int x = threadIdx.x & 31, yy = threadIdx.x >> 5;
    const int c = (blockIdx.x * 32 + x) * VEC;
    const int64_t r0 = (int64_t)blockIdx.y * p.rows_per_cta, r1 = min(p.M, r0 + p.rows_per_cta);
    constexpr bool glu = ACT == kActSwiglu;
    float s0[VEC], s1[VEC];
#pragma unroll
    for (int j = 0; j < VEC; ++j) s0[j] = s1[j] = 0.0f;
    if (c < p.cols) {
        for (int64_t r = r0 + yy; r < r1; r += 8 * kDzRows) {
            W wg[kDzRows], w0[kDzRows], w1[kDzRows];
#pragma unroll
            for (int i = 0; i < kDzRows; ++i) {
                const int64_t q = r + 8 * i;
                if (q >= r1) break;
                wg[i] = *reinterpret_cast<const W*>(p.dy + q * p.lddy + c);
                if (ACT != kActNone) w0[i] = *reinterpret_cast<const W*>(p.z + q * p.N + c);
                if (glu) w1[i] = *reinterpret_cast<const W*>(p.z + q * p.N + p.cols + c);
            }
#pragma unroll
            for (int i = 0; i < kDzRows; ++i) {
                const int64_t q = r + 8 * i;
                if (q >= r1) break;
                float g[VEC], z0[VEC], z1[VEC];
                dz_unpack<VEC>(wg[i], g);
                if (ACT != kActNone) dz_unpack<VEC>(w0[i], z0);
                if (glu) dz_unpack<VEC>(w1[i], z1);
                if (!glu && ACT != kActNone) act_bwd_all<ACT>(z0);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    float d0, d1 = 0.0f;
                    if (glu) {
                        const float sg = sigmoidf(z0[j]);
                        d1 = g[j] * z0[j] * sg;
                        d0 = g[j] * z1[j] * sg * (1.0f + z0[j] * (1.0f - sg));
                    } else {
                        d0 = ACT == kActNone ? g[j] : g[j] * z0[j];
                    }
                    s0[j] += d0;
                    s1[j] += d1;
                    z0[j] = d0;
                    z1[j] = d1;
                }
                if (p.dz) {
                    dz_store<VEC>(p.dz + q * p.lddz + c, z0);
                    if (glu) dz_store<VEC>(p.dz + q * p.lddz + p.cols + c, z1);
                }
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
