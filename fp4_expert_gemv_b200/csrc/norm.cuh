// The norms around a block, with its gate and residual, in one pass over the row:
//
//   m  = y * rho_y,  rho_y = 1 / sqrt(mean(y^2) + eps),  v = w_post * m   (or v = y)
//   r' = r + s * a(g) * v                                                  (a: identity or sigmoid)
//   u  = w_pre * r' * rho,  rho = 1 / sqrt(mean(r'^2) + eps)
//
// r' leaves one block, u enters the next: at a block boundary both norms, the gate and the
// residual sum are one launch that reads r and y once and writes r' and u once.  A row lives in
// the registers of its group of threads; the two sums of squares are the only exchanges.
// Everything is fp32 between the loads and the single rounding of each output; u is taken from
// the unrounded r'.
#pragma once

#include "bulk.cuh"
#include "cluster.cuh"
#include "common.cuh"

namespace fe {

// Device-side problems of the entry points without a handle: kDevTcTimeout, and FE_DEVICE_LOAD_TIMEOUT's bit (a copy
// into shared memory never completed).
constexpr uint32_t kOpLoadTimeout = 0x8;
__device__ uint32_t g_op_status;

constexpr int kNormMaxH = 16384;   // 1024 threads x 2 chunks of 8

enum { kGateNone = 0, kGateChannel = 1, kGateToken = 2, kGateFull = 3 };

struct NormParams {
    const void* r;            // [T][H] bf16 or fp32
    const uint16_t* y;        // [T][H] or null
    const uint16_t* w_post;   // [H] or null
    const uint16_t* gate;     // [H], [T] or [T][H]
    const uint16_t* w_pre;    // [H] or null
    int gate_kind, gate_sigmoid;
    float scale, eps;
    int64_t T;
    int H;
    void* r_out;              // or null
    uint16_t* u;              // or null
};

struct NormBwdParams {
    NormParams f;
    const void* dr_out;       // [T][H] like r, or null
    const uint16_t* du;       // [T][H] or null
    void* dr;                 // or null
    uint16_t* dy;             // or null
    void* dgate;              // channel: null (through part), token: float [T], full: bf16 [T][H]
    float* part;              // [grid][3][H] column sums (dw_post, dw_pre, dgate per channel), or null
};

// 2^x and 1 / x to 2 ulp, one instruction each: no scaling around results below 2^-126, which are zero.  exp(x) as
// 2^(x log2 e) with one rounded product is off by |x| 2^-23 of itself besides (2^-16 at x = -87, the last one that
// is not zero): a sigmoid far from 0 and a softmax's small p are rounded so by choice, what they are added to is
// larger by as much, and a product in two parts would cost two more instructions an element.
FE_DEV float ex2_ftz(float x)
{
    float v;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(v) : "f"(x));
    return v;
}

FE_DEV float rcp_ftz(float x)
{
    float v;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(v) : "f"(x));
    return v;
}

constexpr float kLog2e = 1.4426950408889634f;

FE_DEV float sigmoidf(float x) { return rcp_ftz(1.0f + ex2_ftz(x * -kLog2e)); }

// Two fp32 fused multiply-adds in one instruction, and products.
FE_DEV float2 fma2(float2 a, float2 b, float2 c)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, c, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
        "fma.rn.f32x2 d, a, b, c;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

FE_DEV float2 mul2(float2 a, float2 b)
{
    float2 d;
    asm("{\n\t.reg .b64 a, b, d;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmul.rn.f32x2 d, a, b;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

// A thread's chunk c of 8 elements of a row: consecutive (VEC 8, 16-byte accesses) or strided by
// the group's threads (VEC 1: any width and alignment, still coalesced).
template <int VEC>
FE_DEV int norm_elem(int c, int j, int t, int tpr)
{
    return VEC == 8 ? (c * tpr + t) * 8 + j : (c * 8 + j) * tpr + t;
}

template <int VEC>
FE_DEV void norm_load(const uint16_t* row, int c, int t, int tpr, int H, bool on, float (&v)[8])
{
    if (VEC == 8) {
        const int e = norm_elem<8>(c, 0, t, tpr);
        uint4 q = make_uint4(0, 0, 0, 0);
        if (on && e < H) q = *reinterpret_cast<const uint4*>(row + e);
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[2 * j] = __uint_as_float(w[j] << 16);
            v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = norm_elem<1>(c, j, t, tpr);
            v[j] = on && e < H ? bf16_bits_to_f32(row[e]) : 0.0f;
        }
    }
}

template <int VEC>
FE_DEV void norm_load(const float* row, int c, int t, int tpr, int H, bool on, float (&v)[8])
{
    if (VEC == 8) {
        const int e = norm_elem<8>(c, 0, t, tpr);
        float4 a = make_float4(0, 0, 0, 0), b = a;
        if (on && e < H) {
            a = *reinterpret_cast<const float4*>(row + e);
            b = *reinterpret_cast<const float4*>(row + e + 4);
        }
        v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
        v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = norm_elem<1>(c, j, t, tpr);
            v[j] = on && e < H ? row[e] : 0.0f;
        }
    }
}

template <int VEC>
FE_DEV void norm_store(uint16_t* row, int c, int t, int tpr, int H, const float (&v)[8])
{
    if (VEC == 8) {
        const int e = norm_elem<8>(c, 0, t, tpr);
        if (e < H)
            *reinterpret_cast<uint4*>(row + e) =
                make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = norm_elem<1>(c, j, t, tpr);
            if (e < H) row[e] = (uint16_t)(bf16x2_rn(v[j], 0.0f) & 0xffffu);
        }
    }
}

template <int VEC>
FE_DEV void norm_store(float* row, int c, int t, int tpr, int H, const float (&v)[8])
{
    if (VEC == 8) {
        const int e = norm_elem<8>(c, 0, t, tpr);
        if (e < H) {
            *reinterpret_cast<float4*>(row + e) = make_float4(v[0], v[1], v[2], v[3]);
            *reinterpret_cast<float4*>(row + e + 4) = make_float4(v[4], v[5], v[6], v[7]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = norm_elem<1>(c, j, t, tpr);
            if (e < H) row[e] = v[j];
        }
    }
}

// Sums of N values over the tpr threads of a row's group, every thread gets them.  tpr is a power
// of two from 32 to 1024; groups of one warp need no barrier.  `buf` alternates between two halves
// from one call to the next: a half is written again only after the barrier of the call between.
template <int N>
FE_DEV void group_sum(float (&v)[N], int tpr, float (*buf)[32][N])
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    if (tpr == 32) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wpg = tpr >> 5, first = warp & ~(wpg - 1);
    if (lane == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) (*buf)[warp][i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        float s = (*buf)[first + (lane & (wpg - 1))][i];
        for (int o = wpg >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        v[i] = s;
    }
}

// One group of tpr threads per row, blockDim.x / tpr rows per CTA.
template <int VEC, int C, bool R32>
__global__ void __launch_bounds__(1024) block_norm_kernel(NormParams p, int tpr)
{
    using RT = typename std::conditional<R32, float, uint16_t>::type;
    __shared__ float red[2][32][1];
    griddep_wait();
    griddep_launch();
    const int t = threadIdx.x & (tpr - 1);
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    const bool on = row < p.T;
    const size_t base = (size_t)(on ? row : 0) * p.H;
    float r[C][8], y[C][8], a[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) norm_load<VEC>(static_cast<const RT*>(p.r) + base, c, t, tpr, p.H, on, r[c]);
    if (p.y) {
        float g1 = 1.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) norm_load<VEC>(p.y + base, c, t, tpr, p.H, on, y[c]);
        if (p.gate_kind == kGateChannel || p.gate_kind == kGateFull) {
            const uint16_t* g = p.gate + (p.gate_kind == kGateFull ? base : 0);
#pragma unroll
            for (int c = 0; c < C; ++c) norm_load<VEC>(g, c, t, tpr, p.H, on, a[c]);
        } else if (p.gate_kind == kGateToken && on) {
            g1 = bf16_bits_to_f32(p.gate[row]);
            if (p.gate_sigmoid) g1 = sigmoidf(g1);
        }
        float k = p.scale * g1;
        if (p.w_post) {
            float s[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) s[0] += y[c][j] * y[c][j];
            group_sum<1>(s, tpr, &red[0]);
            k *= rsqrtf(s[0] / (float)p.H + p.eps);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float w[8];
            if (p.w_post) norm_load<VEC>(p.w_post, c, t, tpr, p.H, true, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float v = k * y[c][j];
                if (p.w_post) v *= w[j];
                if (p.gate_kind == kGateChannel || p.gate_kind == kGateFull)
                    v *= p.gate_sigmoid ? sigmoidf(a[c][j]) : a[c][j];
                r[c][j] += v;
            }
        }
        if (p.r_out && on) {
#pragma unroll
            for (int c = 0; c < C; ++c) norm_store<VEC>(static_cast<RT*>(p.r_out) + base, c, t, tpr, p.H, r[c]);
        }
    }
    if (!p.u) return;
    float s[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool in = VEC == 8 || norm_elem<VEC>(c, j, t, tpr) < p.H;
            s[0] += in ? r[c][j] * r[c][j] : 0.0f;
        }
    group_sum<1>(s, tpr, &red[1]);
    const float rho = rsqrtf(s[0] / (float)p.H + p.eps);
    if (!on) return;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float w[8];
        norm_load<VEC>(p.w_pre, c, t, tpr, p.H, true, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) w[j] *= r[c][j] * rho;
        norm_store<VEC>(p.u + base, c, t, tpr, p.H, w);
    }
}

// ---- many rows: the rows stream through shared memory ------------------------------------------
// With one row per group at a time a group loads, waits, reduces, waits and stores, and most of its time
// nothing is on its way from memory.  Here every group of tpr threads walks its rows with the next
// ones already being copied (cp.async.bulk) into its own ring of stages, synchronises alone (a named
// barrier per group) and keeps what belongs to its columns in registers: weights, channel gate, the
// sums over rows.
// One exchange per row: with q = scale w_post a(g) y the second norm's sum is
//   sum r'^2 = sum r^2 + 2 rho_y sum r q + rho_y^2 sum q^2,
// and the backward pass's other sums follow from seven products of the operands as they lie in memory
// (block_norm_backward_ring_kernel), so the sums of all of them travel together and a second walk over
// the stage writes every output.  Where r' is small next to what cancels in it (sum r'^2 below an
// eighth of its positive parts, or not finite), the group takes the sums of the rounded r' itself,
// which costs that row two more exchanges; the backward pass also where a product of y before its norm with a
// gradient leaves fp32 though the norm's own does not.  With an exchange per norm and one for dm, the group's
// warps spent 10,000 cycles a row in latencies: 44 us for T = 4096, H = 2048 backward, where memory
// needs 16.  Now it takes 26.5 us there and 85 us at T = 16384 (4.7 TB/s) without the weights' gradients, 6 us
// more with them (their last partials and the launch that adds them); forward with fp32 rows 21.2 us (4.75
// TB/s).  What bounds it is one group's exchange per row, with 16 warps on an SM.
// A thread has 16 columns: the exchange is paid per thread and row, and with 8 columns it was half of all
// instructions.  What varies per element is a template parameter or a neutral factor, never a branch.

FE_DEV void group_bar(int group, int tpr)
{
    if (tpr == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
}

constexpr int kRedSums = 7;   // sums per exchange, at most

__host__ __device__ constexpr int norm_red_floats(int tpr) { return kRedSums * (tpr / 32 < 4 ? 4 : tpr / 32); }

// Sums over the group's threads; red: [N][max(4, warps)] floats of the group's own, zero where there is no
// warp, in one of two halves that alternate from call to call (the barrier between separates
// a half's readers from its next writers).
template <int N>
FE_DEV void ring_sum(float (&v)[N], int group, int tpr, float* red)
{
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = warp_sum(v[i]);
    if (tpr == 32) {
        __syncwarp();
        return;
    }
    const int wpg = tpr >> 5, slots = max(wpg, 4);
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) red[i * slots + ((threadIdx.x >> 5) & (wpg - 1))] = v[i];
    group_bar(group, tpr);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float4* q = reinterpret_cast<const float4*>(red + i * slots);
        float4 f = q[0];
        float sum = (f.x + f.y) + (f.z + f.w);
        for (int w = 1; w < slots / 4; ++w) {
            f = q[w];
            sum += (f.x + f.y) + (f.z + f.w);
        }
        v[i] = sum;
    }
}

FE_DEV void unpack8(const uint4& q, float (&v)[8])
{
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(w[j] << 16);
        v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}

// Chunk `ch` of 8 of the row of bf16 (fp32) at shared address `row`.
template <bool F32>
FE_DEV void ring_get(uint32_t row, int ch, float (&v)[8])
{
    if constexpr (F32) {
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                     : "r"(row + 32 * ch));
        asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                     : "r"(row + 32 * ch + 16));
    } else {
        uint4 q;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w)
                     : "r"(row + 16 * ch));
        unpack8(q, v);
    }
}

FE_DEV void put8(uint16_t* p, const float (&v)[8])
{
    *reinterpret_cast<uint4*>(p) =
        make_uint4(bf16x2_rn(v[0], v[1]), bf16x2_rn(v[2], v[3]), bf16x2_rn(v[4], v[5]), bf16x2_rn(v[6], v[7]));
}

FE_DEV void put8(float* p, const float (&v)[8])
{
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}

constexpr unsigned long long kNormTimeoutNs = 2000ull * 1000 * 1000;

// Shared memory of a group besides its stages: reduction space (two halves), then a barrier per stage.
__host__ __device__ inline uint32_t norm_group_extra(int tpr, int stages)
{
    return (4u * 2 * norm_red_floats(tpr) + 8u * stages + 127u) / 128u * 128u;
}

// Bytes of a row's operands in a stage.
__host__ __device__ inline uint32_t norm_fwd_stage(int H, bool r32, bool y, bool full)
{
    return (uint32_t)H * ((r32 ? 4 : 2) + (y ? 2 : 0) + (full ? 2 : 0));
}
__host__ __device__ inline uint32_t norm_bwd_stage(int H, bool r32, bool full)
{
    return (uint32_t)H * ((r32 ? 8 : 4) + 4 + (full ? 2 : 0));
}

// A thread's 16 columns: chunks t and t + tpr of 8.
constexpr int kRingC = 2;

FE_DEV float2 pair(const float (&a)[8], int j) { return make_float2(a[j], a[j + 1]); }
FE_DEV void put2(float (&d)[8], int j, float2 v)
{
    d[j] = v.x;
    d[j + 1] = v.y;
}

// Over 8 columns: d = a b + c, d = a b, and the same with one factor for all.
FE_DEV void vfma(float (&d)[8], const float (&a)[8], const float (&b)[8], const float (&c)[8])
{
#pragma unroll
    for (int j = 0; j < 8; j += 2) put2(d, j, fma2(pair(a, j), pair(b, j), pair(c, j)));
}
FE_DEV void vfma(float (&d)[8], float a, const float (&b)[8], const float (&c)[8])
{
#pragma unroll
    for (int j = 0; j < 8; j += 2) put2(d, j, fma2(make_float2(a, a), pair(b, j), pair(c, j)));
}
FE_DEV void vmul(float (&d)[8], const float (&a)[8], const float (&b)[8])
{
#pragma unroll
    for (int j = 0; j < 8; j += 2) put2(d, j, mul2(pair(a, j), pair(b, j)));
}
FE_DEV void vmul(float (&d)[8], float a, const float (&b)[8])
{
#pragma unroll
    for (int j = 0; j < 8; j += 2) put2(d, j, mul2(make_float2(a, a), pair(b, j)));
}

// s += sum of a[j] b[j], in two chains that the caller adds at the end.
FE_DEV void vdot(float (&s)[2], const float (&a)[8], const float (&b)[8])
{
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float2 v = fma2(pair(a, j), pair(b, j), make_float2(s[0], s[1]));
        s[0] = v.x;
        s[1] = v.y;
    }
}

// After a wait that ran out: the copies under way, of up to n rows from stage s on, get the same time again, each, so
// that none outlives the CTA's shared memory.
FE_DEV void ring_drain(uint32_t bar, int s, uint32_t parity, int stages, int64_t n)
{
    for (int j = 0; j < stages && j < n; ++j) {
        mbar_wait(bar + 8 * s, parity, kNormTimeoutNs);
        if (++s == stages) {
            s = 0;
            parity ^= 1;
        }
    }
}

// How the gate enters a row: one factor, a factor per column, or one per element.
enum { kByRow = 0, kByColumn = 1, kByElement = 2 };

// Whether the expanded sum of squares lost too much, given its positive parts (also if it is not finite).
FE_DEV bool sum_cancelled(float sum, float parts) { return !(sum >= 0.125f * parts) || isinf(sum); }

// Whether a sum of products with y before its norm left fp32 (or met a NaN), though the sum it stands for may not.
FE_DEV bool sum_overflowed(float sum) { return !(fabsf(sum) <= 3.402823466e38f); }

// Copies of a row's operands: lane k of the group's first warp holds operand k.
struct RowCopies {
    const char* src;
    uint32_t off, bytes;
    int n;

    FE_DEV RowCopies() : src(nullptr), off(0), bytes(0), n(0) {}
    FE_DEV void add(int t, const void* p, uint32_t at, uint32_t nb)
    {
        if (t == n) {
            src = static_cast<const char*>(p);
            off = at;
            bytes = nb;
        }
        ++n;
    }
    // Row `row` into the stage at dst; by the group's first warp, converged.  Nothing more once a wait of its has run out.
    FE_DEV void fill(int t, int64_t row, int64_t rows, uint32_t dst, uint32_t stage, uint32_t bar, bool dead = false) const
    {
        if (t >= 32 || row >= rows || __any_sync(0xffffffffu, dead)) return;
        if (t == 0) mbar_expect_tx(bar, stage);
        __syncwarp();
        if (t < n) bulk_g2s(dst + off, src + (size_t)row * bytes, bytes, bar);
    }
};

template <bool R32, int GATE, bool Y>
__global__ void __launch_bounds__(512) block_norm_ring_kernel(NormParams p, int tpr, int stages)
{
    using RT = typename std::conditional<R32, float, uint16_t>::type;
    constexpr int C = kRingC;
    extern __shared__ __align__(128) uint8_t norm_dyn[];
    const int t = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = blockDim.x / tpr;
    const int H = p.H;
    const bool token = p.gate_kind == kGateToken, has_u = p.u != nullptr, has_r = p.r_out != nullptr;
    const uint32_t stage = norm_fwd_stage(H, R32, Y, GATE == kByElement);
    const uint32_t oy = H * sizeof(RT), og = oy + 2 * H;
    uint8_t* base = norm_dyn + (size_t)group * (stages * stage + norm_group_extra(tpr, stages));
    float* red = reinterpret_cast<float*>(base + stages * stage);
    const uint32_t bar = smem_addr(red + 2 * norm_red_floats(tpr));
    for (int i = t; i < 2 * norm_red_floats(tpr); i += tpr) red[i] = 0.0f;
    if (t == 0)
        for (int s = 0; s < stages; ++s) mbar_init(bar + 8 * s, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    griddep_wait();
    griddep_launch();
    const int64_t step = (int64_t)gridDim.x * groups, first = (int64_t)blockIdx.x * groups + group;
    RowCopies rc;
    rc.add(t, p.r, 0, H * sizeof(RT));
    if (Y) rc.add(t, p.y, oy, 2 * H);
    if (GATE == kByElement) rc.add(t, p.gate, og, 2 * H);
    const uint32_t base_a = smem_addr(base);
    for (int s = 0; s < stages; ++s) rc.fill(t, first + s * step, p.T, base_a + s * stage, stage, bar + 8 * s);
    // cw: scale * w_post (* the column's gate); neutral factors for what is not there
    float cw[C][8];
    uint4 qpre[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int ch = t + c * tpr;
        const bool mine = ch * 8 < H;
        float g[8];
        qpre[c] = mine && has_u ? reinterpret_cast<const uint4*>(p.w_pre)[ch] : make_uint4(0, 0, 0, 0);
        unpack8(mine && p.w_post ? reinterpret_cast<const uint4*>(p.w_post)[ch] : make_uint4(0, 0, 0, 0), cw[c]);
        if (GATE == kByColumn) unpack8(mine ? reinterpret_cast<const uint4*>(p.gate)[ch] : make_uint4(0, 0, 0, 0), g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!p.w_post) cw[c][j] = 1.0f;
            cw[c][j] *= p.scale;
            if (GATE == kByColumn) cw[c][j] *= p.gate_sigmoid ? sigmoidf(g[j]) : g[j];
        }
    }
    int s = 0, half = 0;
    uint32_t parity = 0;
    bool dead = false;
    uint16_t graw = token && first < p.T ? p.gate[first] : 0;   // the coming row's gate
    const float inv_h = 1.0f / (float)H;
    for (int64_t row = first; row < p.T; row += step) {
        if (!dead && !mbar_wait(bar + 8 * s, parity, kNormTimeoutNs)) {
            dead = true;
            if (t < 32) ring_drain(bar, s, parity, stages, (p.T - row + step - 1) / step);
        }
        const uint32_t src = base_a + s * stage;
        float k = 1.0f;
        if (token) {
            k = bf16_bits_to_f32(graw);
            if (p.gate_sigmoid) k = sigmoidf(k);
            if (row + step < p.T) graw = p.gate[row + step];
        }
        // the row's chunks of r, and q = cw a y
        float r[C][8], q[C][8], syy[2] = {0, 0}, srr[2] = {0, 0}, srq[2] = {0, 0}, sqq[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int ch = t + c * tpr;
            if (ch * 8 < H) {
                ring_get<R32>(src, ch, r[c]);
                vdot(srr, r[c], r[c]);
                if (Y) {
                    ring_get<false>(src + oy, ch, q[c]);
                    vdot(syy, q[c], q[c]);
                    vmul(q[c], q[c], cw[c]);
                    if (GATE == kByElement) {
                        float a[8];
                        ring_get<false>(src + og, ch, a);
                        if (p.gate_sigmoid) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) a[j] = sigmoidf(a[j]);
                        }
                        vmul(q[c], q[c], a);
                    }
                    vdot(srq, r[c], q[c]);
                    vdot(sqq, q[c], q[c]);
                }
            }
        }
        float ss;
        if (Y) {
            float sum[4] = {srr[0] + srr[1], syy[0] + syy[1], srq[0] + srq[1], sqq[0] + sqq[1]};
            ring_sum<4>(sum, group, tpr, red + half * norm_red_floats(tpr));   // also: everyone has read the stage
            half ^= 1;
            if (p.w_post) k *= rsqrtf(sum[1] * inv_h + p.eps);
            const float parts = sum[0] + k * k * sum[3];
            ss = parts + 2.0f * k * sum[2];
            rc.fill(t, row + stages * step, p.T, src, stage, bar + 8 * s, dead);
            if (has_u && sum_cancelled(ss, parts)) {   // the same for the whole group
                float d[2] = {0, 0}, v[8];
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if ((t + c * tpr) * 8 < H) {
                        vfma(v, k, q[c], r[c]);
                        vdot(d, v, v);
                    }
                float one[1] = {d[0] + d[1]};
                ring_sum<1>(one, group, tpr, red + half * norm_red_floats(tpr));
                half ^= 1;
                ss = one[0];
            }
        } else {
            float one[1] = {srr[0] + srr[1]};
            ring_sum<1>(one, group, tpr, red + half * norm_red_floats(tpr));
            half ^= 1;
            rc.fill(t, row + stages * step, p.T, src, stage, bar + 8 * s, dead);
            ss = one[0];
        }
        const float rho = has_u ? rsqrtf(ss * inv_h + p.eps) : 0.0f;
        const size_t at = (size_t)row * H;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int ch = t + c * tpr;
            if (ch * 8 < H && !dead) {
                if (Y) {
                    vfma(r[c], k, q[c], r[c]);   // r'
                    if (has_r) put8(static_cast<RT*>(p.r_out) + at + 8 * ch, r[c]);
                }
                if (has_u) {
                    float w[8];
                    unpack8(qpre[c], w);
                    vmul(w, rho, w);
                    vmul(w, w, r[c]);
                    put8(p.u + at + 8 * ch, w);
                }
            }
        }
        if (++s == stages) {
            s = 0;
            parity ^= 1;
        }
    }
    if (dead) atomicOr(&g_op_status, kOpLoadTimeout);
}

// The gradients.  With n = r' rho and x = du w_pre:
//   D  = dr' + rho (x - n mean(x n))              gradient at r', and at r
//   dv = s a D,  dg = s v D a'(g),  dm = dv w_post
//   dy = rho_y (dm - m mean(dm m))                (dy = dv without w_post)
//   dw_pre = sum_t du n,  dw_post = sum_t dv m,  dg summed over what the gate was broadcast to
// r' is rebuilt in fp32 from r and y, which the gradients need anyway, so the forward pass saves
// nothing.  Every row sum follows from y y, r r, r q, q q, x r, x q and dr' q (q = s a w_post y): with
// k = rho mean(x n),
//   sum x r' = sum x r + rho_y sum x q,
//   sum dm m = rho_y (sum dr' q + rho sum x q - k rho (sum r q + rho_y sum q q)).
// With e = D m, dw_post and a channel gate's gradient are column factors times the same sum of e over
// rows.  The sums over rows stay in the registers of the thread that owns the column; one partial per
// CTA, added in a fixed order by column_sum_kernel.
// Two kernels: block_norm_backward_ring_kernel for rows of whole aligned 16-byte chunks with y, du and dr' there, up
// to the width whose stages fit; block_norm_backward_any_kernel for any other width, alignment and set of
// operands, straight from memory.
template <bool R32, int GATE>
__global__ void __launch_bounds__(512) block_norm_backward_ring_kernel(NormBwdParams q, int tpr, int stages)
{
    using RT = typename std::conditional<R32, float, uint16_t>::type;
    constexpr int C = kRingC;
    extern __shared__ __align__(128) uint8_t norm_dyn[];
    const NormParams& p = q.f;
    const int t = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = blockDim.x / tpr;
    const int H = p.H;
    const bool token = p.gate_kind == kGateToken, w_post = p.w_post != nullptr;
    const uint32_t stage = norm_bwd_stage(H, R32, GATE == kByElement);
    const uint32_t oy = H * sizeof(RT), odr = oy + 2 * H, odu = odr + H * sizeof(RT), og = odu + 2 * H;
    uint8_t* base = norm_dyn + (size_t)group * (stages * stage + norm_group_extra(tpr, stages));
    float* red = reinterpret_cast<float*>(base + stages * stage);
    const uint32_t bar = smem_addr(red + 2 * norm_red_floats(tpr));
    for (int i = t; i < 2 * norm_red_floats(tpr); i += tpr) red[i] = 0.0f;
    if (t == 0)
        for (int s = 0; s < stages; ++s) mbar_init(bar + 8 * s, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    griddep_wait();
    griddep_launch();
    const int64_t step = (int64_t)gridDim.x * groups, first = (int64_t)blockIdx.x * groups + group;
    RowCopies rc;
    rc.add(t, p.r, 0, H * sizeof(RT));
    rc.add(t, p.y, oy, 2 * H);
    rc.add(t, q.dr_out, odr, H * sizeof(RT));
    rc.add(t, q.du, odu, 2 * H);
    if (GATE == kByElement) rc.add(t, p.gate, og, 2 * H);
    const uint32_t base_a = smem_addr(base);
    for (int s = 0; s < stages; ++s) rc.fill(t, first + s * step, p.T, base_a + s * stage, stage, bar + 8 * s);
    // cw: scale * w_post (* the column's gate), wq: w_pre; the sums over rows
    float cw[C][8], E[C][8], gw_pre[C][8];
    uint4 wq[C];   // in bf16: 16 registers less than two chunks of fp32
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float g[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            cw[c][j] = 1.0f;
            E[c][j] = gw_pre[c][j] = g[j] = 0.0f;
        }
        if (w_post) norm_load<8>(p.w_post, c, t, tpr, H, true, cw[c]);
        norm_load<8>(p.w_pre, c, t, tpr, H, true, g);
        wq[c] = make_uint4(bf16x2_rn(g[0], g[1]), bf16x2_rn(g[2], g[3]), bf16x2_rn(g[4], g[5]), bf16x2_rn(g[6], g[7]));
        if (GATE == kByColumn) norm_load<8>(p.gate, c, t, tpr, H, true, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            cw[c][j] *= p.scale;
            if (GATE == kByColumn) cw[c][j] *= p.gate_sigmoid ? sigmoidf(g[j]) : g[j];
        }
    }
    int s = 0, half = 0;
    uint32_t parity = 0;
    bool dead = false;
    uint16_t graw = token && first < p.T ? p.gate[first] : 0;   // the coming row's gate
    const float inv_h = 1.0f / (float)H;
    for (int64_t row = first; row < p.T; row += step) {
        if (!dead && !mbar_wait(bar + 8 * s, parity, kNormTimeoutNs)) {
            dead = true;
            // the row before has not been replaced yet
            if (t < 32) ring_drain(bar, s, parity, stages, min((p.T - row + step - 1) / step, (int64_t)stages - (row != first)));
        }
        const uint32_t src = base_a + s * stage;
        const size_t at = (size_t)row * H;
        // chunk c of an operand of the row, for chunks inside it
        auto inside = [&](int c) { return (t + c * tpr) * 8 < H; };
        auto get_r = [&](int c, float (&v)[8]) { ring_get<R32>(src, t + c * tpr, v); };
        auto get_y = [&](int c, float (&v)[8]) { ring_get<false>(src + oy, t + c * tpr, v); };
        auto get_dr = [&](int c, float (&v)[8]) { ring_get<R32>(src + odr, t + c * tpr, v); };
        auto get_du = [&](int c, float (&v)[8]) { ring_get<false>(src + odu, t + c * tpr, v); };
        auto get_a = [&](int c, float (&v)[8]) {
            ring_get<false>(src + og, t + c * tpr, v);
            if (p.gate_sigmoid) {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[j] = sigmoidf(v[j]);
            }
        };
        auto put = [&](auto* global, int c, const float (&v)[8]) { put8(global + at + 8 * (t + c * tpr), v); };
        float g1 = 1.0f, d1 = 1.0f;
        if (token) {
            g1 = bf16_bits_to_f32(graw);
            if (row + step < p.T) graw = p.gate[row + step];
            if (p.gate_sigmoid) {
                g1 = sigmoidf(g1);
                d1 = g1 * (1.0f - g1);
            }
        }
        // ---- first walk: the seven sums (a row gate stays out of q: it is a factor of the row) -----------
        float syy[2] = {0, 0}, srr[2] = {0, 0}, srq[2] = {0, 0}, sqq[2] = {0, 0}, sxr[2] = {0, 0}, sxq[2] = {0, 0},
              sdq[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (!inside(c)) continue;
            float r[8], y[8], x[8], f[8];
            get_y(c, y);
            get_r(c, r);
            get_du(c, x);
            get_dr(c, f);
            vdot(syy, y, y);
            vmul(y, y, cw[c]);
            if (GATE == kByElement) {
                float a[8];
                get_a(c, a);
                vmul(y, y, a);
            }
            vdot(sdq, f, y);
            vdot(srr, r, r);
            vdot(srq, r, y);
            vdot(sqq, y, y);
            unpack8(wq[c], f);
            vmul(x, x, f);
            vdot(sxr, x, r);
            vdot(sxq, x, y);
        }
        float sum[7] = {syy[0] + syy[1], srr[0] + srr[1], srq[0] + srq[1], sqq[0] + sqq[1],
                        sxr[0] + sxr[1], sxq[0] + sxq[1], sdq[0] + sdq[1]};
        ring_sum<7>(sum, group, tpr, red + half * norm_red_floats(tpr));
        half ^= 1;
        // everyone is past the row before: its stage takes the row that follows the ones under way
        if (row != first) {
            const int sp = s == 0 ? stages - 1 : s - 1;
            rc.fill(t, row + (stages - 1) * step, p.T, base_a + sp * stage, stage, bar + 8 * sp, dead);
        }
        const float rho_y = w_post ? rsqrtf(sum[0] * inv_h + p.eps) : 1.0f;
        const float k1 = g1 * rho_y;   // v's factor of q
        const float parts = sum[1] + k1 * k1 * sum[3];
        float ss = parts + 2.0f * k1 * sum[2], sx = sum[4] + k1 * sum[5];
        const bool direct = sum_cancelled(ss, parts) || sum_overflowed(sx);   // the same for the whole group
        if (direct) {
            float d0[2] = {0, 0}, d1s[2] = {0, 0};
#pragma unroll 1
            for (int c = 0; c < C; ++c) {
                if (!inside(c)) continue;
                float r[8], y[8], x[8], f[8];
                get_y(c, y);
                get_r(c, r);
                get_du(c, x);
#pragma unroll
                for (int cc = 0; cc < C; ++cc)
                    if (cc == c) {
                        vmul(f, rho_y, y);
                        vmul(y, f, cw[cc]);
                        unpack8(wq[cc], f);
                    }
                vmul(x, x, f);
                if (GATE == kByElement) {
                    get_a(c, f);
                    vmul(y, y, f);
                }
                vfma(r, g1, y, r);
                vdot(d0, r, r);
                vdot(d1s, x, r);
            }
            float two[2] = {d0[0] + d0[1], d1s[0] + d1s[1]};
            ring_sum<2>(two, group, tpr, red + half * norm_red_floats(tpr));
            half ^= 1;
            ss = two[0];
            sx = two[1];
        }
        const float rho = rsqrtf(ss * inv_h + p.eps);
        const float rk = sx * inv_h * rho * rho * rho;   // rho mean(x n) rho
        const float dq = sum[6] + rho * sum[5] - rk * (sum[2] + k1 * sum[3]);
        float sdm = k1 * dq;   // sum dm m; over d1 / g1: dg of a token
        float sdg = rho_y * dq;
        if (direct || sum_overflowed(dq)) {
            float d0[2] = {0, 0};
#pragma unroll 1
            for (int c = 0; c < C; ++c) {
                if (!inside(c)) continue;
                float r[8], y[8], x[8], f[8], D[8];
                get_y(c, y);
                get_r(c, r);
                get_du(c, x);
                get_dr(c, D);
#pragma unroll
                for (int cc = 0; cc < C; ++cc)
                    if (cc == c) {
                        vmul(f, rho_y, y);
                        vmul(y, f, cw[cc]);
                        unpack8(wq[cc], f);
                    }
                vmul(x, x, f);
                if (GATE == kByElement) {
                    get_a(c, f);
                    vmul(y, y, f);
                }
                vfma(r, g1, y, r);
                vfma(D, -rk, r, D);
                vfma(D, rho, x, D);
                vdot(d0, D, y);
            }
            float one[1] = {d0[0] + d0[1]};
            ring_sum<1>(one, group, tpr, red + half * norm_red_floats(tpr));
            half ^= 1;
            sdg = one[0];
            sdm = g1 * sdg;
        }
        if (token && q.dgate && t == 0 && !dead) static_cast<float*>(q.dgate)[row] = sdg * d1;
        const float kd = w_post ? sdm * inv_h : 0.0f;
        // ---- second walk: every output ---------------------------------------------------------------
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (!inside(c)) continue;
            float r[8], m[8], D[8], f[8], a[8];
            get_y(c, m);
            get_r(c, r);
            get_dr(c, D);
            vmul(m, rho_y, m);
            if (GATE == kByElement) {
                get_a(c, a);
                vmul(f, cw[c], a);
            } else if (GATE == kByRow) {
                vmul(f, g1, cw[c]);
            } else {
                vmul(f, 1.0f, cw[c]);
            }
            float x[8], e[8];
            vfma(r, f, m, r);   // r'
            get_du(c, x);
            vmul(x, rho, x);
            vfma(gw_pre[c], x, r, gw_pre[c]);
            vfma(D, -rk, r, D);
            unpack8(wq[c], e);
            vfma(D, x, e, D);
            if (q.dr && !dead) put(static_cast<RT*>(q.dr), c, D);
            vmul(e, D, m);
            if (GATE == kByRow) vfma(E[c], g1, e, E[c]);
            else if (GATE == kByColumn) vfma(E[c], 1.0f, e, E[c]);
            else vfma(E[c], a, e, E[c]);
            if (GATE == kByElement && q.dgate && !dead) {
                vmul(e, cw[c], e);
                if (p.gate_sigmoid) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) e[j] *= a[j] * (1.0f - a[j]);
                }
                put(static_cast<uint16_t*>(q.dgate), c, e);
            }
            if (q.dy && !dead) {
                vmul(D, f, D);        // dm
                vfma(D, -kd, m, D);
                vmul(D, rho_y, D);
                put(q.dy, c, D);
            }
        }
        if (++s == stages) {
            s = 0;
            parity ^= 1;
        }
    }
    if (dead) atomicOr(&g_op_status, kOpLoadTimeout);
    if (!q.part) return;
    // the CTA's groups join over the stages (every copy has landed and been read): each leaves its column
    // sums, then they are added in group order, one partial per CTA
    __syncthreads();
    float* cols = reinterpret_cast<float*>(norm_dyn);   // [groups][3][H]
    float* own = cols + (size_t)group * 3 * H;
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float ga[8], wp[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) ga[j] = wp[j] = 1.0f;
        if (GATE == kByColumn) {
            norm_load<8>(p.gate, c, t, tpr, H, true, ga);
            if (w_post) norm_load<8>(p.w_post, c, t, tpr, H, true, wp);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float da = 1.0f;
            if (GATE == kByColumn && p.gate_sigmoid) {
                ga[j] = sigmoidf(ga[j]);
                da = ga[j] * (1.0f - ga[j]);
            }
            wp[j] *= p.scale * da * E[c][j];
            E[c][j] *= p.scale * ga[j];
        }
        norm_store<8>(own, c, t, tpr, H, E[c]);
        norm_store<8>(own + H, c, t, tpr, H, gw_pre[c]);
        if (GATE == kByColumn) norm_store<8>(own + 2 * H, c, t, tpr, H, wp);
    }
    __syncthreads();
    float* out = q.part + (size_t)blockIdx.x * 3 * H;
    for (int e = threadIdx.x; e < (GATE == kByColumn ? 3 : 2) * H; e += blockDim.x) {
        float v = cols[e];
        for (int g = 1; g < groups; ++g) v += cols[(size_t)g * 3 * H + e];
        out[e] = v;
    }
}

// Any width, alignment and set of operands: the same sums and the same two walks, over memory.  A thread has four
// columns 32 apart at a time (a warp 128 beside each other), the group's next batch lies 4 tpr columns further; the
// second walk goes backwards, so that the four it begins with are still held in registers (a whole row of
// up to 2048 columns), and the rest of the row is found in L1.  The next row is asked for into L2 while this
// one is summed.  What bounds it is issuing instructions, two bytes a load: one address serves a thread's four
// columns (columns a row's threads apart took a third more time), and a batch within the row checks no
// ends.  16384 x 1999 with a full gate takes 224 us, 2.3 TB/s; 1237 x 1999 29.2 us.  The sums over rows lie in
// shared memory, where each column has one thread per group.
template <typename OT>
FE_DEV float any_get(const OT* p, size_t i)
{
    if constexpr (std::is_same<OT, float>::value) return p[i];
    else return bf16_bits_to_f32(p[i]);
}

// Asks for `bytes` from p into L2, a 128-byte line per thread of the group.
FE_DEV void any_prefetch(const void* p, size_t bytes, int t, int tpr)
{
    if (!p) return;
    const char* b = static_cast<const char*>(p);
    for (size_t o = (size_t)t * 128; o < bytes; o += (size_t)tpr * 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(b + o));
}

template <bool R32, int GATE, bool ALL>
__global__ void __launch_bounds__(512, 2) block_norm_backward_any_kernel(NormBwdParams q, int tpr)
{
    using RT = typename std::conditional<R32, float, uint16_t>::type;
    extern __shared__ __align__(128) uint8_t norm_dyn[];
    const NormParams& p = q.f;
    const int t = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = blockDim.x / tpr;
    const int H = p.H;
    // ALL: every operand and output is there
    const bool has_y = ALL || p.y != nullptr, has_du = ALL || q.du != nullptr, has_dr = ALL || q.dr_out != nullptr;
    const bool token = p.gate_kind == kGateToken, w_post = ALL || p.w_post != nullptr, sig = p.gate_sigmoid != 0;
    // [groups] reduction halves, then [groups][2][H] sums over rows: of e (times the row's or element's
    // gate) and of du n
    float* red = reinterpret_cast<float*>(norm_dyn) + (size_t)group * 2 * norm_red_floats(tpr);
    float* sums = reinterpret_cast<float*>(norm_dyn) + (size_t)groups * 2 * norm_red_floats(tpr);
    float* E = sums + (size_t)group * 2 * H;
    float* gw_pre = E + H;
    for (int i = t; i < 2 * norm_red_floats(tpr); i += tpr) red[i] = 0.0f;
    for (int e = t; e < 2 * H; e += tpr) E[e] = 0.0f;
    __syncthreads();
    griddep_wait();
    griddep_launch();
    const RT* pr = static_cast<const RT*>(p.r);
    const RT* pdr = static_cast<const RT*>(q.dr_out);
    const int64_t step = (int64_t)gridDim.x * groups, first = (int64_t)blockIdx.x * groups + group;
    const float inv_h = 1.0f / (float)H;
    // a warp has the 32 U columns from U times its place, a thread U of them, 32 apart
    constexpr int U = 4;
    const int col0 = U * (t & ~31) + (t & 31);
    int half = 0;
    for (int64_t row = first; row < p.T; row += step) {
        const size_t at = (size_t)row * H;
        float g1 = 1.0f, d1 = 1.0f;
        if (token) {
            g1 = bf16_bits_to_f32(p.gate[row]);
            if (sig) {
                g1 = sigmoidf(g1);
                d1 = g1 * (1.0f - g1);
            }
        }
        if (row + step < p.T) {
            const size_t next = (size_t)(row + step) * H;
            any_prefetch(pr + next, sizeof(RT) * H, t, tpr);
            if (has_dr) any_prefetch(pdr + next, sizeof(RT) * H, t, tpr);
            if (has_y) any_prefetch(p.y + next, 2 * H, t, tpr);
            if (has_du) any_prefetch(q.du + next, 2 * H, t, tpr);
            if (GATE == kByElement) any_prefetch(p.gate + next, 2 * H, t, tpr);
        }
        // the gate of column e and scale w_post (a row gate stays out of both)
        auto gate_at = [&](int e) {
            if (GATE == kByRow) return 1.0f;
            const float g = bf16_bits_to_f32(p.gate[GATE == kByElement ? at + e : (size_t)e]);
            return sig ? sigmoidf(g) : g;
        };
        auto cw_at = [&](int e) { return p.scale * (w_post ? bf16_bits_to_f32(p.w_post[e]) : 1.0f); };
        auto x_at = [&](int e) { return has_du ? bf16_bits_to_f32(q.du[at + e]) * bf16_bits_to_f32(p.w_pre[e]) : 0.0f; };
        auto y_at = [&](int e) { return has_y ? bf16_bits_to_f32(p.y[at + e]) : 0.0f; };
        auto d_at = [&](int e) { return has_dr ? any_get(pdr, at + e) : 0.0f; };
        // columns e0, e0 + 32, ... of the row: one address per operand; IN: all of them are in the row
        float y[U], r[U], du[U], d[U], ga[U];
        auto load = [&](auto in, int e0) {
            constexpr bool IN = decltype(in)::value;
            const uint16_t *py = p.y + at + e0, *pu = q.du + at + e0, *pg = p.gate + (GATE == kByElement ? at + e0 : (size_t)e0);
            const RT *prr = pr + at + e0, *pd = pdr + at + e0;
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (!IN && e0 + 32 * j >= H) break;
                y[j] = has_y ? bf16_bits_to_f32(py[32 * j]) : 0.0f;
                r[j] = any_get(prr, 32 * j);
                du[j] = has_du ? bf16_bits_to_f32(pu[32 * j]) : 0.0f;
                d[j] = has_dr ? any_get(pd, 32 * j) : 0.0f;
                if (GATE != kByRow) ga[j] = bf16_bits_to_f32(pg[32 * j]);
            }
            if (GATE != kByRow && sig) {
#pragma unroll
                for (int j = 0; j < U; ++j) {
                    if (!IN && e0 + 32 * j >= H) break;
                    ga[j] = sigmoidf(ga[j]);
                }
            }
        };
        float sum[7] = {0, 0, 0, 0, 0, 0, 0};
        auto add = [&](auto in, int e0) {
            constexpr bool IN = decltype(in)::value;
            load(in, e0);
            const uint16_t *pw = p.w_post + e0, *pq = p.w_pre + e0;
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (!IN && e0 + 32 * j >= H) break;
                float f = p.scale * y[j];
                if (w_post) f *= bf16_bits_to_f32(pw[32 * j]);
                if (GATE != kByRow) f *= ga[j];
                const float x = has_du ? du[j] * bf16_bits_to_f32(pq[32 * j]) : 0.0f;
                sum[0] = fmaf(y[j], y[j], sum[0]);
                sum[1] = fmaf(r[j], r[j], sum[1]);
                sum[2] = fmaf(r[j], f, sum[2]);
                sum[3] = fmaf(f, f, sum[3]);
                sum[4] = fmaf(x, r[j], sum[4]);
                sum[5] = fmaf(x, f, sum[5]);
                sum[6] = fmaf(d[j], f, sum[6]);
            }
        };
        int e0 = col0;
        for (;; e0 += U * tpr) {
            if (e0 + 32 * (U - 1) < H) add(std::true_type{}, e0);
            else add(std::false_type{}, e0);
            if (e0 - col0 + U * tpr >= H) break;
        }
        ring_sum<7>(sum, group, tpr, red + half * norm_red_floats(tpr));
        half ^= 1;
        const float rho_y = w_post ? rsqrtf(sum[0] * inv_h + p.eps) : 1.0f;
        const float k1 = g1 * rho_y;
        const float parts = sum[1] + k1 * k1 * sum[3];
        float ss = parts + 2.0f * k1 * sum[2], sx = sum[4] + k1 * sum[5];
        const bool direct = sum_cancelled(ss, parts) || sum_overflowed(sx);
        if (direct) {
            float two[2] = {0, 0};
#pragma unroll 1
            for (int e = t; e < H; e += tpr) {
                const float r = any_get(pr, at + e) + cw_at(e) * gate_at(e) * g1 * (rho_y * y_at(e));
                two[0] = fmaf(r, r, two[0]);
                two[1] = fmaf(x_at(e), r, two[1]);
            }
            ring_sum<2>(two, group, tpr, red + half * norm_red_floats(tpr));
            half ^= 1;
            ss = two[0];
            sx = two[1];
        }
        const float rho = has_du ? rsqrtf(ss * inv_h + p.eps) : 0.0f;
        const float rk = has_du ? sx * inv_h * rho * rho * rho : 0.0f;
        const float dq = sum[6] + rho * sum[5] - rk * (sum[2] + k1 * sum[3]);
        float sdg = rho_y * dq;
        if (direct || sum_overflowed(dq)) {
            float one[1] = {0};
#pragma unroll 1
            for (int e = t; e < H; e += tpr) {
                const float f = cw_at(e) * gate_at(e), m = rho_y * y_at(e);
                const float r = any_get(pr, at + e) + f * g1 * m;
                one[0] = fmaf(d_at(e) + rho * x_at(e) - rk * r, f * m, one[0]);
            }
            ring_sum<1>(one, group, tpr, red + half * norm_red_floats(tpr));
            half ^= 1;
            sdg = one[0];
        }
        if (token && q.dgate && t == 0) static_cast<float*>(q.dgate)[row] = sdg * d1;
        const float kd = w_post ? sdg * g1 * inv_h : 0.0f;
        auto write = [&](auto in, int e0) {
            constexpr bool IN = decltype(in)::value;
            const uint16_t *pw = p.w_post + e0, *pq = p.w_pre + e0;
            RT* odr = static_cast<RT*>(q.dr) + at + e0;
            uint16_t *ody = q.dy + at + e0, *odg = static_cast<uint16_t*>(q.dgate) + at + e0;
            float *sE = E + e0, *sw = gw_pre + e0;
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (!IN && e0 + 32 * j >= H) break;
                const float m = rho_y * y[j], a = GATE == kByRow ? 1.0f : ga[j];
                const float cw = p.scale * (w_post ? bf16_bits_to_f32(pw[32 * j]) : 1.0f), f = cw * a * g1;
                const float ro = fmaf(f, m, r[j]);   // r'
                const float u = du[j] * rho;
                const float D = d[j] + (has_du ? u * bf16_bits_to_f32(pq[32 * j]) : 0.0f) - rk * ro;
                if (has_du) sw[32 * j] = fmaf(u, ro, sw[32 * j]);
                if (ALL || q.dr) {
                    if constexpr (R32) odr[32 * j] = D;
                    else odr[32 * j] = (uint16_t)(bf16x2_rn(D, 0.0f) & 0xffffu);
                }
                const float em = D * m;
                sE[32 * j] = fmaf(GATE == kByRow ? g1 : GATE == kByElement ? a : 1.0f, em, sE[32 * j]);
                if (GATE == kByElement && (ALL || q.dgate))
                    odg[32 * j] = (uint16_t)(bf16x2_rn(cw * em * (sig ? a * (1.0f - a) : 1.0f), 0.0f) & 0xffffu);
                if (ALL || q.dy) ody[32 * j] = (uint16_t)(bf16x2_rn(rho_y * (D * f - kd * m), 0.0f) & 0xffffu);
            }
        };
        for (bool held = true; e0 >= 0; e0 -= U * tpr, held = false) {
            if (e0 + 32 * (U - 1) < H) {
                if (!held) load(std::true_type{}, e0);
                write(std::true_type{}, e0);
            } else {
                if (!held) load(std::false_type{}, e0);
                write(std::false_type{}, e0);
            }
        }
    }
    if (!q.part) return;
    __syncthreads();
    float* out = q.part + (size_t)blockIdx.x * 3 * H;
    for (int e = threadIdx.x; e < H; e += blockDim.x) {
        float v = 0.0f, g = 0.0f;
        for (int k = 0; k < groups; ++k) {
            v += sums[(size_t)k * 2 * H + e];
            g += sums[(size_t)k * 2 * H + H + e];
        }
        float a = 1.0f, da = 1.0f;
        if (GATE == kByColumn) {
            a = bf16_bits_to_f32(p.gate[e]);
            if (sig) {
                a = sigmoidf(a);
                da = a * (1.0f - a);
            }
            out[2 * H + e] = p.scale * (w_post ? bf16_bits_to_f32(p.w_post[e]) : 1.0f) * da * v;
        }
        out[e] = p.scale * a * v;
        out[H + e] = g;
    }
}

// out_i[c] = sum over g of part[g][i][c], i < 3, c < W: 32 columns per CTA, 32 threads per column
// each adding every 32nd partial, then the 32 sums in order.  A fixed order: no atomics.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* part, int G, int W, int segs, float* o0,
                                                          float* o1, float* o2)
{
    __shared__ float s[32][33];
    griddep_wait();
    griddep_launch();
    const int x = threadIdx.x & 31, yy = threadIdx.x >> 5;
    const int seg = blockIdx.y, c = blockIdx.x * 32 + x;
    float* out = seg == 0 ? o0 : seg == 1 ? o1 : o2;
    if (!out) return;
    float v = 0.0f;
    if (c < W)
        for (int g0 = yy; g0 < G; g0 += 32 * 5) {   // 160 partials asked for at once
            float w[5];
#pragma unroll
            for (int j = 0; j < 5; ++j) w[j] = g0 + 32 * j < G ? part[((size_t)(g0 + 32 * j) * segs + seg) * W + c] : 0.0f;
#pragma unroll
            for (int j = 0; j < 5; ++j) v += w[j];
        }
    s[yy][x] = v;
    __syncthreads();
    v = warp_sum(s[x][yy]);   // lane x holds partial x of column yy
    const int col = blockIdx.x * 32 + yy;
    if (x == 0 && col < W) out[col] = v;
}

}  // namespace fe
