// The router's balance loss over T tokens of E logits, n of them kept by the mask:
//
//   p_t = softmax(l_t),  c_e = #{(t, j): idx[t][j] = e},  f_e = c_e / (n k),  P_e = (1/n) sum_t p_te
//   balance = E sum_e f_e P_e,   z = (1/n) sum_t logsumexp(l_t)^2,   loss = a balance + b z
//   dloss/dl_te = (a E / n) p_te (f_e - sum_i f_i p_ti) + (2 b / n) lse_t p_te
//
// One warp per row, the row in its registers: the logits are read once in either direction and the
// gradient written once, which is all the memory traffic there is.  A row without a finite logit
// (all -inf) has p = 0 and adds nothing to P and z.
#pragma once

#include "common.cuh"
#include "norm.cuh"

namespace fe {

constexpr int kBalThreads = 256, kBalWarps = kBalThreads / 32;
constexpr int kBalMaxE = 1024;

struct BalanceParams {
    const float* logits;      // [T][E]
    const int32_t* idx;       // [T][k]; ids outside [0, E) are not counted
    const uint8_t* mask;      // [T] or null
    int64_t T;
    int E, k;
    float a, b;               // coefficients of balance and z
    float* loss;              // [3]: loss, balance, z
    int32_t* counts;          // [E]
    int32_t* n_tokens;        // [1]
    float* part;              // [G][E] sums of p, then [G] sums of lse^2
    int32_t* ipart;           // [G][E] counts, then [G] kept tokens
    int G;
    // backward
    const float* dloss;       // [1] or null (1)
    void* dlogits;            // [T][E] float or bf16
    int dl_bf16;
};

// Lane's values of a row: element (i * 32 + lane) * VEC + j for i < NPL / VEC.
template <int NPL, int VEC>
FE_DEV int bal_elem(int i, int lane) { return ((i / VEC) * 32 + lane) * VEC + i % VEC; }

template <int NPL, int VEC>
FE_DEV void bal_load(const float* row, int E, int lane, float (&l)[NPL])
{
    if (VEC == 4) {
#pragma unroll
        for (int i = 0; i < NPL; i += VEC) {
            const int e = bal_elem<NPL, VEC>(i, lane);
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (e < E) v = __ldg(reinterpret_cast<const float4*>(row + e));
            l[i] = v.x;
            l[(i + 1) % NPL] = v.y;
            l[(i + 2) % NPL] = v.z;
            l[(i + 3) % NPL] = v.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NPL; ++i) {
            const int e = bal_elem<NPL, VEC>(i, lane);
            l[i] = e < E ? __ldg(row + e) : -INFINITY;
        }
    }
}

// l -> softmax numerators exp(l - max), returns 1 / sum and the logsumexp; 0 and 0 for a row of
// -inf.  NaN or +inf anywhere makes both NaN, as the formula does.
template <int NPL>
FE_DEV void bal_softmax(float (&l)[NPL], float& inv, float& lse)
{
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < NPL; ++i) m = fmaxf(m, l[i]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float mm = m == -INFINITY ? 0.0f : m;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        l[i] = __expf(l[i] - mm);
        s += l[i];
    }
    s = warp_sum(s);
    inv = s == 0.0f ? 0.0f : 1.0f / s;
    lse = s == 0.0f ? 0.0f : mm + logf(s);
}

template <int NPL, int VEC>
__global__ void __launch_bounds__(kBalThreads) balance_kernel(BalanceParams p)
{
    __shared__ int cnt[kBalMaxE];
    __shared__ float ps[kBalMaxE];
    __shared__ float zs[kBalWarps];
    __shared__ int ns[kBalWarps];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < p.E; e += kBalThreads) cnt[e] = 0;
    __syncthreads();
    float acc[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) acc[i] = 0.0f;
    float z = 0.0f;
    int n = 0;
    for (int64_t t = (int64_t)blockIdx.x * kBalWarps + warp; t < p.T; t += (int64_t)p.G * kBalWarps) {
        if (p.mask && p.mask[t] == 0) continue;   // the warp's lanes agree
        float l[NPL], inv, lse;
        bal_load<NPL, VEC>(p.logits + (size_t)t * p.E, p.E, lane, l);
        for (int j = lane; j < p.k; j += 32) {
            const int e = p.idx[(size_t)t * p.k + j];
            if ((unsigned)e < (unsigned)p.E) atomicAdd(&cnt[e], 1);   // integers: any order, one result
        }
        bal_softmax<NPL>(l, inv, lse);
#pragma unroll
        for (int i = 0; i < NPL; ++i) acc[i] += l[i] * inv;
        z += lse * lse;
        ++n;
    }
    // the CTA's warps join in warp order
    for (int w = 0; w < kBalWarps; ++w) {
        if (warp == w) {
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const int e = bal_elem<NPL, VEC>(i, lane);
                if (e < p.E) ps[e] = (w ? ps[e] : 0.0f) + acc[i];
            }
        }
        __syncthreads();
    }
    if (lane == 0) {
        zs[warp] = z;
        ns[warp] = n;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < p.E; e += kBalThreads) {
        p.part[(size_t)blockIdx.x * p.E + e] = ps[e];
        p.ipart[(size_t)blockIdx.x * p.E + e] = cnt[e];
    }
    if (threadIdx.x == 0) {
        float zz = 0.0f;
        int nn = 0;
        for (int w = 0; w < kBalWarps; ++w) {
            zz += zs[w];
            nn += ns[w];
        }
        p.part[(size_t)p.G * p.E + blockIdx.x] = zz;
        p.ipart[(size_t)p.G * p.E + blockIdx.x] = nn;
    }
}

// Joins the CTAs' partials in a fixed order and writes the loss and the counts: one CTA, a warp per
// 32 experts at a time, 32 threads down the partials of a column.
__global__ void __launch_bounds__(1024) balance_final_kernel(BalanceParams p)
{
    __shared__ float sf[32][33];
    __shared__ int si[32][33];
    __shared__ float dot[32];
    griddep_wait();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    float fp = 0.0f;   // lane 0 of warp y: sum of counts * P over its experts
    for (int e0 = 0; e0 < p.E; e0 += 32) {
        const int e = e0 + x;
        float v = 0.0f;
        int c = 0;
        if (e < p.E)
            for (int g = y; g < p.G; g += 32) {
                v += p.part[(size_t)g * p.E + e];
                c += p.ipart[(size_t)g * p.E + e];
            }
        __syncthreads();
        sf[y][x] = v;
        si[y][x] = c;
        __syncthreads();
        const float P = warp_sum(sf[x][y]);
        const int cs = __reduce_add_sync(0xffffffffu, si[x][y]);
        if (x == 0 && e0 + y < p.E) {
            p.counts[e0 + y] = cs;
            fp += (float)cs * P;
        }
    }
    if (x == 0) dot[y] = fp;
    __syncthreads();
    if (y > 0) return;
    float z = 0.0f;
    int n = 0;
    for (int g = x; g < p.G; g += 32) {
        z += p.part[(size_t)p.G * p.E + g];
        n += p.ipart[(size_t)p.G * p.E + g];
    }
    z = warp_sum(z);
    n = __reduce_add_sync(0xffffffffu, n);
    const float d = warp_sum(dot[x]);
    if (x == 0) {
        const float fn = (float)max(n, 1);
        const float bal = (float)p.E * (d / (fn * (float)p.k)) / fn;
        const float zz = z / fn;
        // a part without a coefficient adds nothing, even where it overflowed
        p.loss[0] = (p.a != 0.0f ? p.a * bal : 0.0f) + (p.b != 0.0f ? p.b * zz : 0.0f);
        p.loss[1] = bal;
        p.loss[2] = zz;
        p.n_tokens[0] = n;
    }
}

template <int NPL, int VEC>
__global__ void __launch_bounds__(kBalThreads) balance_backward_kernel(BalanceParams p)
{
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = *p.n_tokens;
    const float up = (p.dloss ? *p.dloss : 1.0f) / (float)max(n, 1);
    const float fscale = 1.0f / ((float)max(n, 1) * (float)p.k);
    float f[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) {
        const int e = bal_elem<NPL, VEC>(i, lane);
        f[i] = e < p.E ? (float)p.counts[e] * fscale : 0.0f;
    }
    const float ca = up * p.a * (float)p.E, cb = 2.0f * up * p.b;
    for (int64_t t = (int64_t)blockIdx.x * kBalWarps + warp; t < p.T; t += (int64_t)gridDim.x * kBalWarps) {
        const bool keep = !p.mask || p.mask[t] != 0;
        float l[NPL];
        if (keep) {
            float inv, lse, d = 0.0f;
            bal_load<NPL, VEC>(p.logits + (size_t)t * p.E, p.E, lane, l);
            bal_softmax<NPL>(l, inv, lse);
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                l[i] *= inv;
                d += l[i] * f[i];
            }
            d = warp_sum(d);
#pragma unroll
            for (int i = 0; i < NPL; ++i) l[i] *= ca * (f[i] - d) + cb * lse;
        } else {
#pragma unroll
            for (int i = 0; i < NPL; ++i) l[i] = 0.0f;
        }
        if (VEC == 4) {
#pragma unroll
            for (int i = 0; i < NPL; i += VEC) {
                const int e = bal_elem<NPL, VEC>(i, lane);
                if (e >= p.E) continue;
                const float a = l[i], b = l[(i + 1) % NPL], c = l[(i + 2) % NPL], d = l[(i + 3) % NPL];
                if (p.dl_bf16)
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.dlogits) + (size_t)t * p.E + e) =
                        make_uint2(bf16x2_rn(a, b), bf16x2_rn(c, d));
                else
                    *reinterpret_cast<float4*>(static_cast<float*>(p.dlogits) + (size_t)t * p.E + e) =
                        make_float4(a, b, c, d);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NPL; ++i) {
                const int e = bal_elem<NPL, VEC>(i, lane);
                if (e >= p.E) continue;
                if (p.dl_bf16)
                    static_cast<uint16_t*>(p.dlogits)[(size_t)t * p.E + e] = (uint16_t)(bf16x2_rn(l[i], 0.0f) & 0xffffu);
                else
                    static_cast<float*>(p.dlogits)[(size_t)t * p.E + e] = l[i];
            }
        }
    }
}

}  // namespace fe
