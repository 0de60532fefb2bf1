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

constexpr int kBalMaxE = 1024;
constexpr int kBalThreads = 256, kBalWarps = kBalThreads / 32;   // backward
constexpr int kBalCluster = 8;                                   // CTAs that join partial sums
// Warps of a forward CTA by values per lane: their sums of p share 32 KB.
__host__ __device__ constexpr int bal_warps(int npl) { return npl <= 8 ? 32 : 256 / npl; }

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
    int G;                    // CTAs of the first pass; 0: one cluster does everything
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

// What is left once a cluster's CTAs each hold their share of sum_e c_e P_e: the loss, by rank 0.
// sums: {share of the dot product, sum of lse^2}, n: kept tokens, in every CTA's shared memory.
FE_DEV void bal_finish(const BalanceParams& p, float* sums, int* n, uint32_t rank, int ranks)
{
    cluster_sync();
    if (rank == 0 && threadIdx.x == 0) {
        float d = 0.0f, z = 0.0f;
        int nn = 0;
        const uint32_t fa = (uint32_t)__cvta_generic_to_shared(sums), na = (uint32_t)__cvta_generic_to_shared(n);
        for (int s = 0; s < ranks; ++s) {
            d += ld_cluster_f32(cluster_map(fa, s));
            z += ld_cluster_f32(cluster_map(fa + 4, s));
            nn += ld_cluster_s32(cluster_map(na, s));
        }
        const float fn = (float)max(nn, 1);
        const float bal = (float)p.E * (d / (fn * (float)p.k)) / fn;
        const float zz = z / fn;
        // a part without a coefficient adds nothing, even where it overflowed
        p.loss[0] = (p.a != 0.0f ? p.a * bal : 0.0f) + (p.b != 0.0f ? p.b * zz : 0.0f);
        p.loss[1] = bal;
        p.loss[2] = zz;
        p.n_tokens[0] = nn;
    }
    cluster_sync();   // the others' shared memory is read until here
}

// Sum of v over the CTA's warps, in warp order, in thread 0.
FE_DEV float bal_block_sum(float v, float* scratch)
{
    v = warp_sum(v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    if (threadIdx.x == 0)
        for (int w = 0; w < (int)blockDim.x / 32; ++w) s += scratch[w];
    return s;
}

// A warp takes every so many-th row, with the next one's loads under way; per lane the sums of its
// experts' p.  For a batch of a few rows per warp of one cluster (p.G = 0) the CTAs join their sums
// through distributed shared memory and the loss is one launch (T = 64, E = 128: 8.1 us as two
// launches); beyond, each CTA leaves a partial for balance_final_kernel.
template <int NPL, int VEC>
__global__ void __launch_bounds__(32 * bal_warps(NPL)) balance_kernel(BalanceParams p)
{
    constexpr int W = bal_warps(NPL);
    __shared__ float ps[W][32 * NPL];
    __shared__ int cnt[kBalMaxE];
    __shared__ float scratch[32];
    __shared__ float sums[2];
    __shared__ int ns[32], n_all;
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < p.E; e += 32 * W) cnt[e] = 0;
    __syncthreads();
    float acc[NPL], next[NPL];
#pragma unroll
    for (int i = 0; i < NPL; ++i) acc[i] = 0.0f;
    float z = 0.0f;
    int n = 0;
    const int64_t step = (int64_t)gridDim.x * W;
    auto kept = [&](int64_t t) { return !p.mask || p.mask[t] != 0; };
    int64_t t = (int64_t)blockIdx.x * W + warp;
    while (t < p.T && !kept(t)) t += step;   // the warp's lanes agree
    if (t < p.T) bal_load<NPL, VEC>(p.logits + (size_t)t * p.E, p.E, lane, next);
    while (t < p.T) {
        float l[NPL], inv, lse;
#pragma unroll
        for (int i = 0; i < NPL; ++i) l[i] = next[i];
        int e0 = -1;
        if (lane < p.k) e0 = p.idx[(size_t)t * p.k + lane];
        int64_t tn = t + step;
        while (tn < p.T && !kept(tn)) tn += step;
        if (tn < p.T) bal_load<NPL, VEC>(p.logits + (size_t)tn * p.E, p.E, lane, next);
        bal_softmax<NPL>(l, inv, lse);
#pragma unroll
        for (int i = 0; i < NPL; ++i) acc[i] += l[i] * inv;
        z += lse * lse;
        ++n;
        if ((unsigned)e0 < (unsigned)p.E) atomicAdd(&cnt[e0], 1);   // integers: any order, one result
        for (int j = lane + 32; j < p.k; j += 32) {
            const int e = p.idx[(size_t)t * p.k + j];
            if ((unsigned)e < (unsigned)p.E) atomicAdd(&cnt[e], 1);
        }
        t = tn;
    }
#pragma unroll
    for (int i = 0; i < NPL; ++i) ps[warp][bal_elem<NPL, VEC>(i, lane)] = acc[i];
    if (lane == 0) ns[warp] = n;
    const float zz = bal_block_sum(lane == 0 ? z : 0.0f, scratch);   // and every warp's sums are in place
    int nn = 0;
    if (threadIdx.x == 0)
        for (int w = 0; w < W; ++w) nn += ns[w];
    float* mine = &ps[0][0];   // the CTA's sums, over the first row
    for (int e = threadIdx.x; e < p.E; e += 32 * W) {
        float v = 0.0f;
#pragma unroll 8
        for (int w = 0; w < W; ++w) v += ps[w][e];
        if (p.G > 0) {
            p.part[(size_t)blockIdx.x * p.E + e] = v;
            p.ipart[(size_t)blockIdx.x * p.E + e] = cnt[e];
        } else {
            mine[e] = v;   // column e is this thread's alone
        }
    }
    if (p.G > 0) {
        if (threadIdx.x == 0) {
            p.part[(size_t)p.G * p.E + blockIdx.x] = zz;
            p.ipart[(size_t)p.G * p.E + blockIdx.x] = nn;
        }
        return;
    }
    cluster_sync();
    const uint32_t rank = cluster_rank();
    const int ranks = gridDim.x;
    float dot = 0.0f;
    for (int e = rank * (32 * W) + threadIdx.x; e < p.E; e += ranks * 32 * W) {
        const uint32_t fa = (uint32_t)__cvta_generic_to_shared(mine + e), ia = (uint32_t)__cvta_generic_to_shared(cnt + e);
        float v = 0.0f;
        int c = 0;
        for (int s = 0; s < ranks; ++s) {
            v += ld_cluster_f32(cluster_map(fa, s));
            c += ld_cluster_s32(cluster_map(ia, s));
        }
        p.counts[e] = c;
        dot += (float)c * v;
    }
    dot = bal_block_sum(dot, scratch);
    if (threadIdx.x == 0) {
        sums[0] = dot;
        sums[1] = zz;
        n_all = nn;
    }
    bal_finish(p, sums, &n_all, rank, ranks);
}

// Joins the CTAs' partials in a fixed order and writes the loss and the counts: one cluster, each CTA
// 32 experts at a time with 32 threads down the partials of a column.
__global__ void __cluster_dims__(kBalCluster, 1, 1) __launch_bounds__(1024) balance_final_kernel(BalanceParams p)
{
    __shared__ float sf[32][33];
    __shared__ int si[32][33];
    __shared__ float scratch[32];
    __shared__ float sums[2];
    __shared__ int n_all;
    griddep_wait();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank();
    float fp = 0.0f;   // lane 0 of warp y: sum of counts * P over its experts
    for (int e0 = 32 * rank; e0 < p.E; e0 += 32 * kBalCluster) {
        const int e = e0 + x;
        float v = 0.0f;
        int c = 0;
        if (e < p.E) {
#pragma unroll 4
            for (int g = y; g < p.G; g += 32) {
                v += p.part[(size_t)g * p.E + e];
                c += p.ipart[(size_t)g * p.E + e];
            }
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
    float z = 0.0f;
    int n = 0;
    if (rank == 0 && y == 0) {
        for (int g = x; g < p.G; g += 32) {
            z += p.part[(size_t)p.G * p.E + g];
            n += p.ipart[(size_t)p.G * p.E + g];
        }
        z = warp_sum(z);
        n = __reduce_add_sync(0xffffffffu, n);
    }
    const float d = bal_block_sum(x == 0 ? fp : 0.0f, scratch);
    if (threadIdx.x == 0) {
        sums[0] = d;
        sums[1] = z;
        n_all = n;
    }
    bal_finish(p, sums, &n_all, rank, kBalCluster);
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
