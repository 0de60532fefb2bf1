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

// Device-side problems of the entry points without a handle (kDevTcTimeout, kDevLoadTimeout).
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

FE_DEV float sigmoidf(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }

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
// ones already being copied (cp.async.bulk, one thread) into its own ring of stages, synchronises alone (a
// named barrier per group) and keeps what belongs to its columns in registers: weights, channel gate,
// the sums over rows.  A thread has 16 columns: the sums' shuffles and barriers are paid per thread
// and row, and with 8 columns they were half of all instructions.  What varies per element is a
// template parameter or a neutral factor, never a branch: the instruction count bounds these kernels
// next to memory (the first backward pass spent 114 instructions per element and 82 us at T = 4096,
// H = 2048, where memory needs 16).

FE_DEV void group_bar(int group, int tpr)
{
    if (tpr == 32) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory");
}

constexpr int kRedSums = 2;   // sums per exchange, at most

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

FE_DEV void ring_get(const uint16_t* row, int chunk, float (&v)[8]) { unpack8(reinterpret_cast<const uint4*>(row)[chunk], v); }

FE_DEV void ring_get(const float* row, int chunk, float (&v)[8])
{
    const float4 a = reinterpret_cast<const float4*>(row)[2 * chunk], b = reinterpret_cast<const float4*>(row)[2 * chunk + 1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
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
__host__ __device__ inline uint32_t norm_bwd_stage(int H, bool r32, bool y, bool full, bool dr, bool du)
{
    return (uint32_t)H * ((r32 ? 4 : 2) * (dr ? 2 : 1) + (y ? 2 : 0) + (full ? 2 : 0) + (du ? 2 : 0));
}

// A thread's 16 columns: chunks t and t + tpr of 8.
constexpr int kRingC = 2;

// How the gate enters a row: one factor, a factor per column, or one per element.
enum { kByRow = 0, kByColumn = 1, kByElement = 2 };

template <bool R32, int GATE>
__global__ void __launch_bounds__(512) block_norm_ring_kernel(NormParams p, int tpr, int stages)
{
    using RT = typename std::conditional<R32, float, uint16_t>::type;
    constexpr int C = kRingC;
    extern __shared__ __align__(128) uint8_t norm_dyn[];
    const int t = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = blockDim.x / tpr;
    const int H = p.H;
    const bool has_y = p.y != nullptr, token = p.gate_kind == kGateToken, has_u = p.u != nullptr, has_r = p.r_out != nullptr;
    const uint32_t stage = norm_fwd_stage(H, R32, has_y, GATE == kByElement);
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
    auto fill = [&](int64_t row, int s) {
        if (t != 0 || row >= p.T) return;
        const uint32_t dst = smem_addr(base + s * stage), b = bar + 8 * s;
        mbar_expect_tx(b, stage);
        const size_t at = (size_t)row * H;
        bulk_g2s(dst, static_cast<const RT*>(p.r) + at, H * sizeof(RT), b);
        if (has_y) bulk_g2s(dst + H * sizeof(RT), p.y + at, 2 * H, b);
        if (GATE == kByElement) bulk_g2s(dst + H * sizeof(RT) + 2 * H, p.gate + at, 2 * H, b);
    };
    for (int s = 0; s < stages; ++s) fill(first + s * step, s);
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
    float gate1 = token && first < p.T ? bf16_bits_to_f32(p.gate[first]) : 1.0f;
    const float inv_h = 1.0f / (float)H;
    for (int64_t row = first; row < p.T; row += step) {
        if (!dead && !mbar_wait(bar + 8 * s, parity, kNormTimeoutNs)) dead = true;
        const uint8_t* src = base + s * stage;
        float r[C][8], y[C][8];
        float k = 1.0f;
        if (token) {
            k = p.gate_sigmoid ? sigmoidf(gate1) : gate1;
            gate1 = row + step < p.T ? bf16_bits_to_f32(p.gate[row + step]) : 0.0f;   // the next row's
        }
        const size_t at = (size_t)row * H;
        if (has_y) {
            float sum[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int ch = t + c * tpr;
                if (ch * 8 < H) ring_get(reinterpret_cast<const uint16_t*>(src + H * sizeof(RT)), ch, y[c]);
                else
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[c][j] = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[0] = fmaf(y[c][j], y[c][j], sum[0]);
            }
            if (p.w_post) {
                ring_sum<1>(sum, group, tpr, red + half * norm_red_floats(tpr));
                half ^= 1;
                k *= rsqrtf(sum[0] * inv_h + p.eps);
            }
        }
        float sq[1] = {0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int ch = t + c * tpr;
            const bool mine = ch * 8 < H;
            if (mine) ring_get(reinterpret_cast<const RT*>(src), ch, r[c]);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) r[c][j] = 0.0f;
            if (has_y) {
                if (GATE == kByElement) {
                    float a[8];
                    unpack8(mine ? reinterpret_cast<const uint4*>(src + H * sizeof(RT) + 2 * H)[ch] : make_uint4(0, 0, 0, 0), a);
                    if (p.gate_sigmoid) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) a[j] = sigmoidf(a[j]);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[c][j] *= a[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) r[c][j] = fmaf(cw[c][j] * k, y[c][j], r[c][j]);
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sq[0] = fmaf(r[c][j], r[c][j], sq[0]);
            if (has_r && mine && !dead) norm_store<8>(static_cast<RT*>(p.r_out) + at, c, t, tpr, H, r[c]);
        }
        ring_sum<1>(sq, group, tpr, red + half * norm_red_floats(tpr));   // also: everyone has read the stage
        half ^= 1;
        fill(row + stages * step, s);
        if (has_u) {
            const float rho = rsqrtf(sq[0] * inv_h + p.eps);
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float w[8];
                unpack8(qpre[c], w);
#pragma unroll
                for (int j = 0; j < 8; ++j) w[j] *= r[c][j] * rho;
                if ((t + c * tpr) * 8 < H && !dead) norm_store<8>(p.u + at, c, t, tpr, H, w);
            }
        }
        if (++s == stages) {
            s = 0;
            parity ^= 1;
        }
    }
    if (dead) atomicOr(&g_op_status, kDevLoadTimeout);
}

// The gradients.  With n = r' rho and dn = du w_pre:
//   D  = dr' + rho (dn - n mean(dn n))            gradient at r', and at r
//   dv = s a D,  dg = s v D a'(g),  dm = dv w_post
//   dy = rho_y (dm - m mean(dm m))                (dy = dv without w_post)
//   dw_pre = sum_t du n,  dw_post = sum_t dv m,  dg summed over what the gate was broadcast to
// r' is rebuilt in fp32 from r and y, which the gradients need anyway, so the forward pass saves
// nothing.  With e = D m, dw_post and a channel gate's gradient are column factors times the same sum
// of e over rows.  The sums over rows stay in the registers of the thread that owns the column; one
// partial per CTA, added in a fixed order by column_sum_kernel.
// RING: rows of whole 16-byte chunks, through the ring, two chunks of 8 columns per thread (C = 2), or 1
// where a row needs no more; otherwise any width and alignment, the row's operands in registers, one
// chunk of columns t, t + tpr, ... per thread (C = 2 beyond 8192 columns).
template <bool R32, int GATE, bool RING, int C, int MAXT>
__global__ void __launch_bounds__(MAXT) block_norm_backward_kernel(NormBwdParams q, int tpr, int stages)
{
    using RT = typename std::conditional<R32, float, uint16_t>::type;
    constexpr int VEC = RING ? 8 : 1;
    extern __shared__ __align__(128) uint8_t norm_dyn[];
    const NormParams& p = q.f;
    const int t = threadIdx.x & (tpr - 1), group = threadIdx.x / tpr, groups = blockDim.x / tpr;
    const int H = p.H;
    const bool has_y = p.y != nullptr, has_du = q.du != nullptr, has_dr = q.dr_out != nullptr;
    const bool token = p.gate_kind == kGateToken, w_post = p.w_post != nullptr;
    const uint32_t stage = RING ? norm_bwd_stage(H, R32, has_y, GATE == kByElement, has_dr, has_du) : 0;
    const uint32_t oy = H * sizeof(RT), odr = oy + (has_y ? 2 * H : 0), odu = odr + (has_dr ? H * sizeof(RT) : 0),
                   og = odu + (has_du ? 2 * H : 0);
    uint8_t* base = norm_dyn + (size_t)group * (stages * stage + norm_group_extra(tpr, stages));
    float* red = reinterpret_cast<float*>(base + stages * stage);
    const uint32_t bar = smem_addr(red + 2 * norm_red_floats(tpr));
    for (int i = t; i < 2 * norm_red_floats(tpr); i += tpr) red[i] = 0.0f;
    if (RING && t == 0)
        for (int s = 0; s < stages; ++s) mbar_init(bar + 8 * s, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    griddep_wait();
    griddep_launch();
    const int64_t step = (int64_t)gridDim.x * groups, first = (int64_t)blockIdx.x * groups + group;
    auto fill = [&](int64_t row, int s) {
        if (t != 0 || row >= p.T) return;
        const uint32_t dst = smem_addr(base + s * stage), b = bar + 8 * s;
        mbar_expect_tx(b, stage);
        const size_t at = (size_t)row * H;
        bulk_g2s(dst, static_cast<const RT*>(p.r) + at, H * sizeof(RT), b);
        if (has_y) bulk_g2s(dst + oy, p.y + at, 2 * H, b);
        if (has_dr) bulk_g2s(dst + odr, static_cast<const RT*>(q.dr_out) + at, H * sizeof(RT), b);
        if (has_du) bulk_g2s(dst + odu, q.du + at, 2 * H, b);
        if (GATE == kByElement) bulk_g2s(dst + og, p.gate + at, 2 * H, b);
    };
    if (RING)
        for (int s = 0; s < stages; ++s) fill(first + s * step, s);
    // cw: scale * w_post (* the column's gate), wq: w_pre; the sums over rows
    float cw[C][8], wq[C][8], E[C][8], gw_pre[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c) {
        float g[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            cw[c][j] = 1.0f;
            wq[c][j] = E[c][j] = gw_pre[c][j] = 0.0f;
        }
        if (w_post) norm_load<VEC>(p.w_post, c, t, tpr, H, true, cw[c]);
        if (has_du) norm_load<VEC>(p.w_pre, c, t, tpr, H, true, wq[c]);
        if (GATE == kByColumn) norm_load<VEC>(p.gate, c, t, tpr, H, true, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            cw[c][j] *= p.scale;
            if (GATE == kByColumn) cw[c][j] *= p.gate_sigmoid ? sigmoidf(g[j]) : g[j];
        }
    }
    int s = 0, half = 0;
    uint32_t parity = 0;
    bool dead = false;
    float gate1 = token && first < p.T ? bf16_bits_to_f32(p.gate[first]) : 1.0f;
    const float inv_h = 1.0f / (float)H;
    for (int64_t row = first; row < p.T; row += step) {
        if (RING && !dead && !mbar_wait(bar + 8 * s, parity, kNormTimeoutNs)) dead = true;
        const uint8_t* src = base + s * stage;
        const size_t at = (size_t)row * H;
        // chunk c of an operand, from the stage or from memory
        auto get = [&](const auto* global, uint32_t off, int c, float (&v)[8]) {
            if constexpr (RING) {
                using OT = typename std::remove_const<typename std::remove_pointer<decltype(global)>::type>::type;
                if ((t + c * tpr) * 8 < H) ring_get(reinterpret_cast<const OT*>(src + off), t + c * tpr, v);
                else
#pragma unroll
                    for (int j = 0; j < 8; ++j) v[j] = 0.0f;
            } else {
                norm_load<1>(global + at, c, t, tpr, H, true, v);
            }
        };
        const RT* gr = static_cast<const RT*>(p.r);
        const RT* gdr = static_cast<const RT*>(q.dr_out);
        float r[C][8], y[C][8], dn[C][8], D[C][8], a[C][8];
        if (!RING) {   // everything on its way at once
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (has_y) get(p.y, oy, c, y[c]);
                get(gr, 0, c, r[c]);
                if (has_du) get(q.du, odu, c, dn[c]);
                if (has_dr) get(gdr, odr, c, D[c]);
                if (GATE == kByElement) get(p.gate, og, c, a[c]);
            }
        }
        float g1 = 1.0f, d1 = 1.0f;
        if (token) {
            g1 = gate1;
            gate1 = row + step < p.T ? bf16_bits_to_f32(p.gate[row + step]) : 0.0f;   // the next row's
            if (p.gate_sigmoid) {
                g1 = sigmoidf(g1);
                d1 = g1 * (1.0f - g1);
            }
        }
        float rho_y = 1.0f;
        if (has_y) {
            float sum[1] = {0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (RING) get(p.y, oy, c, y[c]);
#pragma unroll
                for (int j = 0; j < 8; ++j) sum[0] = fmaf(y[c][j], y[c][j], sum[0]);
                if (GATE == kByElement) {
                    if (RING) get(p.gate, og, c, a[c]);
                    if (p.gate_sigmoid) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) a[c][j] = sigmoidf(a[c][j]);
                    }
                }
            }
            if (w_post) {
                ring_sum<1>(sum, group, tpr, red + half * norm_red_floats(tpr));
                half ^= 1;
                rho_y = rsqrtf(sum[0] * inv_h + p.eps);
            }
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) y[c][j] *= rho_y;   // m
        }
        float rho = 0.0f, rk = 0.0f;
        if (has_du) {
            float sum[2] = {0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (RING) {
                    get(gr, 0, c, r[c]);
                    get(q.du, odu, c, dn[c]);
                }
                if (has_y) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const float f = GATE == kByElement ? cw[c][j] * a[c][j] : GATE == kByRow ? cw[c][j] * g1 : cw[c][j];
                        r[c][j] = fmaf(f, y[c][j], r[c][j]);   // r'
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    sum[0] = fmaf(r[c][j], r[c][j], sum[0]);
                    sum[1] = fmaf(dn[c][j] * wq[c][j], r[c][j], sum[1]);
                }
            }
            ring_sum<2>(sum, group, tpr, red + half * norm_red_floats(tpr));
            half ^= 1;
            rho = rsqrtf(sum[0] * inv_h + p.eps);
            rk = sum[1] * inv_h * rho * rho * rho;   // rho mean(dn n) rho
        }
        float sum[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            if (!has_dr) {
#pragma unroll
                for (int j = 0; j < 8; ++j) D[c][j] = 0.0f;
            } else if (RING) {
                get(gdr, odr, c, D[c]);
            }
            if (has_du) {
                if (RING) get(q.du, odu, c, dn[c]);   // read again: 16 registers less over the exchange
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    gw_pre[c][j] = fmaf(dn[c][j], r[c][j] * rho, gw_pre[c][j]);
                    D[c][j] = fmaf(rho * wq[c][j], dn[c][j], fmaf(-rk, r[c][j], D[c][j]));
                }
            }
            if (q.dr && !dead) norm_store<VEC>(static_cast<RT*>(q.dr) + at, c, t, tpr, H, D[c]);
            if (!has_y) continue;
            float dgf[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float e = D[c][j] * y[c][j];
                if (GATE == kByRow) {
                    E[c][j] = fmaf(g1, e, E[c][j]);
                    sum[1] = fmaf(cw[c][j], e, sum[1]);        // a token gate's gradient, and mean(dm m)
                    D[c][j] *= cw[c][j] * g1;                  // dm
                } else if (GATE == kByColumn) {
                    E[c][j] += e;
                    sum[0] = fmaf(cw[c][j], e, sum[0]);
                    D[c][j] *= cw[c][j];
                } else {
                    const float ca = cw[c][j] * a[c][j];
                    E[c][j] = fmaf(a[c][j], e, E[c][j]);
                    sum[0] = fmaf(ca, e, sum[0]);
                    dgf[j] = cw[c][j] * e * (p.gate_sigmoid ? a[c][j] * (1.0f - a[c][j]) : 1.0f);
                    D[c][j] *= ca;
                }
            }
            if (GATE == kByElement && q.dgate && !dead)
                norm_store<VEC>(static_cast<uint16_t*>(q.dgate) + at, c, t, tpr, H, dgf);
        }
        if (GATE == kByRow) sum[0] = sum[1];
        {
            float one[1] = {sum[0]};
            ring_sum<1>(one, group, tpr, red + half * norm_red_floats(tpr));   // also: everyone has read the stage
            half ^= 1;
            sum[0] = one[0];
        }
        if (RING) fill(row + stages * step, s);
        if (has_y) {
            if (token && q.dgate && t == 0 && !dead) static_cast<float*>(q.dgate)[row] = sum[0] * d1;
            if (q.dy && !dead) {
                const float k = w_post ? sum[0] * (GATE == kByRow ? g1 : 1.0f) * inv_h : 0.0f;
#pragma unroll
                for (int c = 0; c < C; ++c) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) D[c][j] = rho_y * fmaf(-k, y[c][j], D[c][j]);
                    norm_store<VEC>(q.dy + at, c, t, tpr, H, D[c]);
                }
            }
        }
        if (++s == stages) {
            s = 0;
            parity ^= 1;
        }
    }
    if (dead) atomicOr(&g_op_status, kDevLoadTimeout);
    if (!q.part) return;
    // the CTA's groups join in order, over the stages (every copy has landed and been read), then one
    // partial per CTA
    __syncthreads();
    float* cols = reinterpret_cast<float*>(norm_dyn);   // [3][H] when the CTA has more than one group
    float* out = q.part + (size_t)blockIdx.x * 3 * H;
    for (int g = 0; g < groups; ++g) {
        if (group == g) {
            float* to = g < groups - 1 ? cols : out;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float ga[8], wp[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) ga[j] = wp[j] = 1.0f;
                if (GATE == kByColumn) {
                    norm_load<VEC>(p.gate, c, t, tpr, H, true, ga);
                    if (w_post) norm_load<VEC>(p.w_post, c, t, tpr, H, true, wp);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int e = norm_elem<VEC>(c, j, t, tpr);
                    if (e >= H) continue;
                    float da = 1.0f;
                    if (GATE == kByColumn && p.gate_sigmoid) {
                        ga[j] = sigmoidf(ga[j]);
                        da = ga[j] * (1.0f - ga[j]);
                    }
                    const float v[3] = {p.scale * (GATE == kByColumn ? ga[j] : 1.0f) * E[c][j], gw_pre[c][j],
                                        p.scale * wp[j] * da * E[c][j]};
#pragma unroll
                    for (int i = 0; i < 3; ++i) to[i * H + e] = g > 0 ? cols[i * H + e] + v[i] : v[i];
                }
            }
        }
        if (groups > 1) __syncthreads();
    }
}

// out_i[c] = sum over g of part[g][i][c], i < 3, c < W: 32 columns per CTA, 32 threads per column
// each adding every 32nd partial, then the 32 sums in order.  A fixed order: no atomics.
__global__ void __launch_bounds__(1024) column_sum_kernel(const float* part, int G, int W, int segs, float* o0,
                                                          float* o1, float* o2)
{
    __shared__ float s[32][33];
    griddep_wait();
    const int x = threadIdx.x & 31, yy = threadIdx.x >> 5;
    const int seg = blockIdx.y, c = blockIdx.x * 32 + x;
    float* out = seg == 0 ? o0 : seg == 1 ? o1 : o2;
    if (!out) return;
    float v = 0.0f;
    if (c < W)
        for (int g = yy; g < G; g += 32) v += part[((size_t)g * segs + seg) * W + c];
    s[yy][x] = v;
    __syncthreads();
    v = warp_sum(s[x][yy]);   // lane x holds partial x of column yy
    const int col = blockIdx.x * 32 + yy;
    if (x == 0 && col < W) out[col] = v;
}

}  // namespace fe
