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

#include "cluster.cuh"
#include "common.cuh"

namespace fe {

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
    int64_t rows_per_cta;
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

// The gradients.  With n = r' rho and dn = du w_pre:
//   D  = dr' + rho (dn - n mean(dn n))            gradient at r', and at r
//   dv = s a D,  dg = s v D a'(g),  dm = dv w_post
//   dy = rho_y (dm - m mean(dm m))                (dy = dv without w_post)
//   dw_pre = sum_t du n,  dw_post = sum_t dv m,  dg summed over what the gate was broadcast to
// r' is rebuilt in fp32 from r and y, which the gradients need anyway, so the forward pass saves
// nothing.  Each group walks its CTA's rows; the sums over rows stay in the registers of the
// thread that owns the column, one partial per CTA, added in a fixed order by column_sum_kernel.
template <int VEC, int C, bool R32, int MAXT>
__global__ void __launch_bounds__(MAXT) block_norm_backward_kernel(NormBwdParams q, int tpr)
{
    using RT = typename std::conditional<R32, float, uint16_t>::type;
    __shared__ float red[2][32][2];
    griddep_wait();
    const NormParams& p = q.f;
    const int t = threadIdx.x & (tpr - 1), sub = threadIdx.x / tpr, groups = blockDim.x / tpr;
    const float inv_h = 1.0f / (float)p.H;
    float gw_post[C][8], gw_pre[C][8], gg[C][8];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) gw_post[c][j] = gw_pre[c][j] = gg[c][j] = 0.0f;
    int half = 0;
    const int64_t row0 = (int64_t)blockIdx.x * q.rows_per_cta;
    const int64_t row1 = min(p.T, row0 + q.rows_per_cta);
    for (int64_t rb = row0; rb < row1; rb += groups) {
        const int64_t row = rb + sub;
        const bool on = row < row1;
        const size_t base = (size_t)(on ? row : 0) * p.H;
        float r[C][8], y[C][8], a[C][8], D[C][8], dn[C][8];
        float g1 = 1.0f, rho_y = 1.0f, rho = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            norm_load<VEC>(static_cast<const RT*>(p.r) + base, c, t, tpr, p.H, on, r[c]);
            if (p.y) norm_load<VEC>(p.y + base, c, t, tpr, p.H, on, y[c]);
            if (q.dr_out) norm_load<VEC>(static_cast<const RT*>(q.dr_out) + base, c, t, tpr, p.H, on, D[c]);
            else
#pragma unroll
                for (int j = 0; j < 8; ++j) D[c][j] = 0.0f;
            if (q.du) norm_load<VEC>(q.du + base, c, t, tpr, p.H, on, dn[c]);
            if (p.gate_kind == kGateChannel || p.gate_kind == kGateFull)
                norm_load<VEC>(p.gate + (p.gate_kind == kGateFull ? base : 0), c, t, tpr, p.H, on, a[c]);
        }
        const bool gate_elem = p.gate_kind == kGateChannel || p.gate_kind == kGateFull;
        if (p.gate_kind == kGateToken && on) g1 = bf16_bits_to_f32(p.gate[row]);
        if (p.gate_sigmoid) {
            if (gate_elem) {
#pragma unroll
                for (int c = 0; c < C; ++c)
#pragma unroll
                    for (int j = 0; j < 8; ++j) a[c][j] = sigmoidf(a[c][j]);
            } else {
                g1 = sigmoidf(g1);
            }
        }
        if (p.w_post) {
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) s[0] += y[c][j] * y[c][j];
            group_sum<2>(s, tpr, &red[half]);
            half ^= 1;
            rho_y = rsqrtf(s[0] * inv_h + p.eps);
        }
        if (q.du) {
            float s[2] = {0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float w[8], wp[8];
                norm_load<VEC>(p.w_pre, c, t, tpr, p.H, true, w);
                if (p.w_post) norm_load<VEC>(p.w_post, c, t, tpr, p.H, true, wp);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    if (p.y) {
                        float v = p.scale * g1 * rho_y * y[c][j];
                        if (p.w_post) v *= wp[j];
                        if (gate_elem) v *= a[c][j];
                        r[c][j] += v;   // r'
                    }
                    s[0] += r[c][j] * r[c][j];
                    s[1] += dn[c][j] * w[j] * r[c][j];
                }
            }
            group_sum<2>(s, tpr, &red[half]);
            half ^= 1;
            rho = rsqrtf(s[0] * inv_h + p.eps);
            const float k = s[1] * inv_h * rho * rho;   // mean(dn n) rho
#pragma unroll
            for (int c = 0; c < C; ++c) {
                float w[8];
                norm_load<VEC>(p.w_pre, c, t, tpr, p.H, true, w);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    gw_pre[c][j] += on ? dn[c][j] * r[c][j] * rho : 0.0f;
                    D[c][j] += rho * (dn[c][j] * w[j] - k * r[c][j]);
                }
            }
        }
        if (q.dr && on) {
#pragma unroll
            for (int c = 0; c < C; ++c) norm_store<VEC>(static_cast<RT*>(q.dr) + base, c, t, tpr, p.H, D[c]);
        }
        if (!p.y) continue;
        // y -> m, D -> dv; the row sums of dm m and of the token gate's gradient
        const bool token = p.gate_kind == kGateToken;
        float s[2] = {0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float wp[8], dgf[8];
            if (p.w_post) norm_load<VEC>(p.w_post, c, t, tpr, p.H, true, wp);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float m = y[c][j] * rho_y;
                const float w = p.w_post ? wp[j] : 1.0f;
                const float act = gate_elem ? a[c][j] : g1;
                const float da = p.gate_sigmoid ? act * (1.0f - act) : 1.0f;
                const float dg = p.scale * w * m * D[c][j] * da;
                const float dv = p.scale * act * D[c][j];
                if (token) s[1] += dg;
                else if (p.gate_kind == kGateChannel) gg[c][j] += on ? dg : 0.0f;
                dgf[j] = dg;
                gw_post[c][j] += on ? dv * m : 0.0f;
                D[c][j] = dv * w;   // dm
                s[0] += D[c][j] * m;
                y[c][j] = m;
            }
            if (p.gate_kind == kGateFull && q.dgate && on)
                norm_store<VEC>(static_cast<uint16_t*>(q.dgate) + base, c, t, tpr, p.H, dgf);
        }
        if (p.w_post || token) {
            group_sum<2>(s, tpr, &red[half]);
            half ^= 1;
            if (token && q.dgate && on && t == 0) static_cast<float*>(q.dgate)[row] = s[1];
        }
        if (q.dy && on) {
            const float k = p.w_post ? s[0] * inv_h : 0.0f;
#pragma unroll
            for (int c = 0; c < C; ++c) {
#pragma unroll
                for (int j = 0; j < 8; ++j) D[c][j] = rho_y * (D[c][j] - k * y[c][j]);
                norm_store<VEC>(q.dy + base, c, t, tpr, p.H, D[c]);
            }
        }
    }
    if (!q.part) return;
    // the CTA's groups join in shared memory, in order, then one partial per CTA
    extern __shared__ float cols[];   // [3][H] when the CTA has more than one group
    float* out = q.part + (size_t)blockIdx.x * 3 * p.H;
    for (int g = 0; g < groups; ++g) {
        if (sub == g) {
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int e = norm_elem<VEC>(c, j, t, tpr);
                    if (e >= p.H) continue;
                    float v[3] = {gw_post[c][j], gw_pre[c][j], gg[c][j]};
#pragma unroll
                    for (int i = 0; i < 3; ++i) {
                        if (g > 0) v[i] += cols[i * p.H + e];
                        if (g < groups - 1) cols[i * p.H + e] = v[i];
                        else out[i * p.H + e] = v[i];
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
