// The router's balance loss over T tokens of E logits, n of them kept by the mask:
//
//   p_t = softmax(l_t),  c_e = #{(t, j): idx[t][j] = e},  f_e = c_e / (n k),  P_e = (1/n) sum_t p_te
//   balance = E sum_e f_e P_e,   z = (1/n) sum_t logsumexp(l_t)^2,   loss = a balance + b z
//   dloss/dl_te = (a E / n) p_te (f_e - sum_i f_i p_ti) + (2 b / n) lse_t p_te
//
// 32 lanes or fewer per row, the row in their registers: the logits are read once in either direction and
// the gradient written once, which is all the memory traffic there is (T = 65536, E = 512: loss 35.8 us, 3.8
// TB/s, of which the second launch takes 5; gradient 43.1 us, 6.2 TB/s).  A row without a finite logit
// (all -inf) has p = 0 and adds nothing to P and z.
#pragma once

#include "bulk.cuh"
#include "cluster.cuh"
#include "common.cuh"
#include "norm.cuh"

namespace fe {

constexpr int kBalMaxE = 1024;
constexpr int kBalThreads = 256, kBalWarps = kBalThreads / 32;
constexpr int kBalCluster = 8;   // CTAs that join partial sums

// A row is held by L lanes (a power of two) with N values each: 16 values (E up to 512) keep four 16-byte
// loads per lane in flight whatever E is, and a warp takes 32 / L rows at once with log2 L shuffles
// per sum; rows of more than 512 have 32 values.
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

// Value i of lane r of a row's L lanes: consecutive VEC values per lane, L lanes side by side.
template <int L, int VEC>
FE_DEV int bal_elem(int i, int r) { return ((i / VEC) * L + r) * VEC + i % VEC; }

template <int L, int N, int VEC>
FE_DEV void bal_load(const float* row, int E, int r, bool on, float (&l)[N])
{
#pragma unroll
    for (int i = 0; i < N; i += VEC) {
        const int e = bal_elem<L, VEC>(i, r);
        if constexpr (VEC == 4) {
            float4 v = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
            if (on && e < E) v = *reinterpret_cast<const float4*>(row + e);
            l[i] = v.x;
            l[i + 1] = v.y;
            l[i + 2] = v.z;
            l[i + 3] = v.w;
        } else {
            l[i] = on && e < E ? row[e] : -INFINITY;
        }
    }
}

template <int L>
FE_DEV float bal_row_sum(float v)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// l -> softmax numerators exp(l - max), returns 1 / sum and the logsumexp; 0 and 0 for a row of
// -inf.  NaN or +inf anywhere makes both NaN, as the formula does.  A numerator far below the largest is off by up
// to |l - max| 2^-22 of itself (ex2_ftz's argument is rounded), one below 2^-126 is 0.
template <int L, int N>
FE_DEV void bal_softmax(float (&l)[N], float& inv, float& lse)
{
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < N; ++i) m = fmaxf(m, l[i]);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float mm = m == -INFINITY ? 0.0f : m;
    float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        l[i] = ex2_ftz((l[i] - mm) * kLog2e);
        l[i + 1] = ex2_ftz((l[i + 1] - mm) * kLog2e);
        s0 += l[i];
        s1 += l[i + 1];
    }
    float s = s0 + s1;
    s = bal_row_sum<L>(s);
    inv = s == 0.0f ? 0.0f : 1.0f / s;
    lse = s == 0.0f ? 0.0f : mm + logf(s);
}

// What is left once a cluster's CTAs each hold their share of sum_e c_e P_e: the loss, by rank 0.
// sums: {share of the dot product, sum of lse^2}, n: kept tokens, in every CTA's shared memory.
FE_DEV void bal_finish(const BalanceParams& p, float* sums, int* n, uint32_t rank, int ranks)
{
    cluster_sync();
    if (rank == 0 && threadIdx.x < 32) {
        const int lane = threadIdx.x;
        float ds = 0.0f, zs = 0.0f;
        int nn = 0;
        if (lane < ranks) {   // a rank per lane
            const uint32_t fa = cluster_map((uint32_t)__cvta_generic_to_shared(sums), lane);
            ds = ld_cluster_f32(fa);
            zs = ld_cluster_f32(fa + 4);
            nn = ld_cluster_s32(cluster_map((uint32_t)__cvta_generic_to_shared(n), lane));
        }
        const float d = warp_sum(ds), z = warp_sum(zs);
        nn = __reduce_add_sync(0xffffffffu, nn);
        if (lane == 0) {
            const float fn = (float)max(nn, 1);
            const float bal = (float)p.E * (d / (fn * (float)p.k)) / fn;
            const float zz = z / fn;
            // a part without a coefficient adds nothing, even where it overflowed
            p.loss[0] = (p.a != 0.0f ? p.a * bal : 0.0f) + (p.b != 0.0f ? p.b * zz : 0.0f);
            p.loss[1] = bal;
            p.loss[2] = zz;
            p.n_tokens[0] = nn;
        }
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

// One cluster is the grid: its CTAs' sums (mine: of p, cnt: counts, zz, nn: of lse^2 and kept tokens, in thread
// 0) join, each CTA finishing a share of the experts.
FE_DEV void bal_join(const BalanceParams& p, float* mine, int* cnt, float zz, int nn, float* scratch, float* sums, int* n_all)
{
    cluster_sync();
    const uint32_t rank = cluster_rank();
    const int ranks = gridDim.x;
    float dot = 0.0f;
    for (int e = rank * blockDim.x + threadIdx.x; e < p.E; e += ranks * blockDim.x) {
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
        *n_all = nn;
    }
    bal_finish(p, sums, n_all, rank, ranks);
}

// A warp takes every so many-th group of 32 / L rows, with the next group's loads under way; per lane the
// sums of its experts' p.  For a batch of a few groups per warp of one cluster (p.G = 0) the CTAs
// join their sums through distributed shared memory and the loss is one launch (T = 64, E = 128: 3.9 us,
// 8.1 as two launches); beyond, each CTA leaves a partial for balance_final_kernel.
template <int L, int N, int VEC>
__global__ void __launch_bounds__(kBalThreads, N == 16 ? 3 : 1) balance_kernel(BalanceParams p)
{
    constexpr int W = kBalWarps, R = 32 / L;
    __shared__ float ps[W][L * N];
    __shared__ int cnt[L * N];
    __shared__ float scratch[32];
    __shared__ float sums[2];
    __shared__ int ns[32], n_all;
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane % L, sub = lane / L;
    for (int e = threadIdx.x; e < p.E; e += 32 * W) cnt[e] = 0;
    __syncthreads();
    float acc[N], next[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    float z = 0.0f;
    int n = 0;
    const int64_t step = (int64_t)gridDim.x * W * R;
    int64_t t0 = ((int64_t)blockIdx.x * W + warp) * R;   // the warp's group of rows
    bool on = t0 + sub < p.T && (!p.mask || p.mask[t0 + sub] != 0);
    bal_load<L, N, VEC>(p.logits + (size_t)(on ? t0 + sub : 0) * p.E, p.E, r, on, next);
    for (; t0 < p.T; t0 += step) {
        float l[N], inv, lse;
        const bool now = on;
        const int64_t t = t0 + sub, tn = t + step;
#pragma unroll
        for (int i = 0; i < N; ++i) l[i] = next[i];
        on = tn < p.T && (!p.mask || p.mask[tn] != 0);
        bal_load<L, N, VEC>(p.logits + (size_t)(on ? tn : 0) * p.E, p.E, r, on, next);
        if (now)
            for (int j = r; j < p.k; j += L) {
                const int e = p.idx[(size_t)t * p.k + j];
                if ((unsigned)e < (unsigned)p.E) atomicAdd(&cnt[e], 1);   // integers: any order, one result
            }
        __syncwarp();
        bal_softmax<L, N>(l, inv, lse);   // a row that is off is all -inf: zeros
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += l[i] * inv;
        if (r == 0) {
            z += lse * lse;
            n += now;
        }
    }
    // the warp's row groups join
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int o = L; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
        if (sub == 0) ps[warp][bal_elem<L, VEC>(i, r)] = acc[i];
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) ns[warp] = n;
    const float zz = bal_block_sum(z, scratch);   // and every warp's sums are in place
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
    bal_join(p, mine, cnt, zz, nn, scratch, sums, &n_all);
}

// The first pass over many rows: as balance_kernel leaves its partials, but every warp's groups of rows stream
// through its own ring in shared memory (one cp.async.bulk per group: its rows are neighbours), so
// that the loads of several groups are under way per warp while its chain of shuffles and exponentials
// runs.  Padded rows travel too and are left out.  A CTA per SM, or one cluster for all of a batch of a few
// groups per warp (p.G = 0).
constexpr int kBalRingSmem = 224 * 1024;
constexpr int kBalRingStages = 8;   // at most

__host__ __device__ constexpr int bal_ring_warps(int N) { return N == 16 ? 24 : 12; }

template <int L, int N>
__global__ void __launch_bounds__(32 * bal_ring_warps(N)) balance_ring_kernel(BalanceParams p, int stages)
{
    constexpr int W = bal_ring_warps(N), R = 32 / L;
    extern __shared__ __align__(128) uint8_t bal_dyn[];
    __shared__ int cnt[L * N];
    __shared__ float scratch[32];
    __shared__ float sums[2];
    __shared__ int ns[32], n_all;
    __shared__ uint64_t bars[W * kBalRingStages];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane % L, sub = lane / L;
    const uint32_t stage = 4u * R * p.E;   // a group of rows
    const uint32_t ring = smem_addr(bal_dyn) + warp * stages * stage, bar = smem_addr(&bars[kBalRingStages * warp]);
    for (int e = threadIdx.x; e < p.E; e += 32 * W) cnt[e] = 0;
    if (lane < stages) mbar_init(bar + 8 * lane, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    __syncthreads();
    griddep_wait();
    griddep_launch();
    const int64_t step = (int64_t)gridDim.x * W * R;
    bool dead = false;   // a wait ran out: no more copies
    auto fill = [&](int64_t t0, int s) {
        if (lane != 0 || t0 >= p.T || dead) return;
        const uint32_t bytes = 4u * p.E * (uint32_t)min((int64_t)R, p.T - t0);
        mbar_expect_tx(bar + 8 * s, bytes);
        bulk_g2s(ring + s * stage, p.logits + (size_t)t0 * p.E, bytes, bar + 8 * s);
    };
    const int64_t first = ((int64_t)blockIdx.x * W + warp) * R;
    for (int s = 0; s < stages; ++s) fill(first + s * step, s);
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    float z = 0.0f;
    int n = 0, s = 0;
    uint32_t parity = 0;
    // the next group's mask byte and chosen id are fetched a group ahead
    uint32_t keep_next = 0;
    int id_next = -1;
    auto ahead = [&](int64_t t) {
        keep_next = t < p.T;
        id_next = -1;
        if (t < p.T) {
            if (p.mask) keep_next = p.mask[t];
            if (r < p.k) id_next = p.idx[(size_t)t * p.k + r];
        }
    };
    ahead(first + sub);
    for (int64_t t0 = first; t0 < p.T; t0 += step) {
        const int64_t t = t0 + sub;
        const bool on = keep_next != 0;
        const int id = on ? id_next : -1;
        ahead(t + step);
        if (!dead && !mbar_wait(bar + 8 * s, parity, kNormTimeoutNs)) {
            dead = true;
            if (lane == 0) ring_drain(bar, s, parity, stages, (p.T - t0 + step - 1) / step);
        }
        float l[N], inv, lse;
        const uint32_t row = ring + s * stage + 4u * sub * p.E;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const int e = bal_elem<L, 4>(i, r);
            l[i] = l[i + 1] = l[i + 2] = l[i + 3] = -INFINITY;
            if (on && e < p.E)
                asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(l[i]), "=f"(l[i + 1]), "=f"(l[i + 2]), "=f"(l[i + 3])
                             : "r"(row + 4u * e));
        }
        bal_softmax<L, N>(l, inv, lse);   // a row that is off is all -inf: zeros
        __syncwarp();                     // the warp has read the stage
        fill(t0 + stages * step, s);
#pragma unroll
        for (int i = 0; i < N; ++i) acc[i] += l[i] * inv;
        if (r == 0) {
            z += lse * lse;
            n += on;
        }
        if ((unsigned)id < (unsigned)p.E) atomicAdd(&cnt[id], 1);   // integers: any order, one result
        if (on && p.k > L)
            for (int j = r + L; j < p.k; j += L) {
                const int e = p.idx[(size_t)t * p.k + j];
                if ((unsigned)e < (unsigned)p.E) atomicAdd(&cnt[e], 1);
            }
        __syncwarp();
        if (++s == stages) {
            s = 0;
            parity ^= 1;
        }
    }
    if (dead) atomicOr(&g_op_status, kOpLoadTimeout);
    const float zz = bal_block_sum(z, scratch);   // and every warp is done with its ring
    float(*ps)[L * N] = reinterpret_cast<float(*)[L * N]>(bal_dyn);
#pragma unroll
    for (int i = 0; i < N; ++i) {
#pragma unroll
        for (int o = L; o < 32; o <<= 1) acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], o);
        if (sub == 0) ps[warp][bal_elem<L, 4>(i, r)] = acc[i];
    }
    n = __reduce_add_sync(0xffffffffu, n);
    if (lane == 0) ns[warp] = n;
    __syncthreads();
    int nn = 0;
    if (threadIdx.x == 0)
        for (int w = 0; w < W; ++w) nn += ns[w];
    for (int e = threadIdx.x; e < p.E; e += 32 * W) {
        float v = 0.0f;
#pragma unroll 8
        for (int w = 0; w < W; ++w) v += ps[w][e];
        if (p.G > 0) {
            p.part[(size_t)blockIdx.x * p.E + e] = v;
            p.ipart[(size_t)blockIdx.x * p.E + e] = cnt[e];
        } else {
            ps[0][e] = v;   // column e is this thread's alone
        }
    }
    if (p.G == 0) {
        bal_join(p, ps[0], cnt, zz, nn, scratch, sums, &n_all);
    } else if (threadIdx.x == 0) {
        p.part[(size_t)p.G * p.E + blockIdx.x] = zz;
        p.ipart[(size_t)p.G * p.E + blockIdx.x] = nn;
    }
}

// Joins the CTAs' partials in a fixed order and writes the loss and the counts: one cluster, each CTA an
// eighth of the experts, 32 threads down the partials of a column.
__global__ void __cluster_dims__(kBalCluster, 1, 1) __launch_bounds__(1024) balance_final_kernel(BalanceParams p)
{
    constexpr int B = kBalMaxE / 32 / kBalCluster;   // blocks of 32 experts per CTA, at most
    __shared__ float sf[B][32][33];
    __shared__ int si[B][32][33];
    __shared__ float scratch[32];
    __shared__ float sums[2];
    __shared__ int n_all;
    griddep_wait();
    griddep_launch();
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const uint32_t rank = cluster_rank();
    // rank 0's first warp also joins the other sums: its loads go out before the columns'
    float z = 0.0f;
    int n = 0;
    if (rank == 0 && y == 0)
        for (int g = x; g < p.G; g += 32) {
            z += p.part[(size_t)p.G * p.E + g];
            n += p.ipart[(size_t)p.G * p.E + g];
        }
#pragma unroll
    for (int b = 0; b < B; ++b) {
        const int e = 32 * (rank + kBalCluster * b) + x;
        if (32 * (rank + kBalCluster * b) >= p.E) break;
        float v = 0.0f;
        int c = 0;
        // 160 partials are asked for at once: one latency for a CTA an SM
        for (int g0 = y; g0 < p.G; g0 += 32 * 5) {
            float w[5];
            int i[5];
#pragma unroll
            for (int j = 0; j < 5; ++j) {
                const bool on = g0 + 32 * j < p.G && e < p.E;
                w[j] = on ? p.part[(size_t)(g0 + 32 * j) * p.E + e] : 0.0f;
                i[j] = on ? p.ipart[(size_t)(g0 + 32 * j) * p.E + e] : 0;
            }
#pragma unroll
            for (int j = 0; j < 5; ++j) {
                v += w[j];
                c += i[j];
            }
        }
        sf[b][y][x] = v;
        si[b][y][x] = c;
    }
    __syncthreads();
    float fp = 0.0f;   // lane 0 of warp y: sum of counts * P over its experts
#pragma unroll
    for (int b = 0; b < B; ++b) {
        if (32 * (rank + kBalCluster * b) >= p.E) break;
        const int e = 32 * (rank + kBalCluster * b) + y;
        const float P = warp_sum(sf[b][x][y]);
        const int cs = __reduce_add_sync(0xffffffffu, si[b][x][y]);
        if (x == 0 && e < p.E) {
            p.counts[e] = cs;
            fp += (float)cs * P;
        }
    }
    if (rank == 0 && y == 0) {
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

template <int L, int N, int VEC>
__global__ void __launch_bounds__(kBalThreads) balance_backward_kernel(BalanceParams p)
{
    constexpr int W = kBalWarps, R = 32 / L;
    griddep_wait();
    griddep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int r = lane % L, sub = lane / L;
    const int n = *p.n_tokens;
    const float up = (p.dloss ? *p.dloss : 1.0f) / (float)max(n, 1);
    const float fscale = 1.0f / ((float)max(n, 1) * (float)p.k);
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int e = bal_elem<L, VEC>(i, r);
        f[i] = e < p.E ? (float)p.counts[e] * fscale : 0.0f;
    }
    const float ca = up * p.a * (float)p.E, cb = 2.0f * up * p.b;
    for (int64_t t0 = ((int64_t)blockIdx.x * W + warp) * R; t0 < p.T; t0 += (int64_t)gridDim.x * W * R) {
        const int64_t t = t0 + sub;
        const bool on = t < p.T && (!p.mask || p.mask[t] != 0);
        float l[N], inv, lse, d = 0.0f;
        bal_load<L, N, VEC>(p.logits + (size_t)(on ? t : 0) * p.E, p.E, r, on, l);
        bal_softmax<L, N>(l, inv, lse);   // a row that is off is all -inf: zeros
#pragma unroll
        for (int i = 0; i < N; ++i) {
            l[i] *= inv;
            d += l[i] * f[i];
        }
        d = bal_row_sum<L>(d);
#pragma unroll
        for (int i = 0; i < N; ++i) l[i] = on ? l[i] * (ca * (f[i] - d) + cb * lse) : 0.0f;
        if (t >= p.T) continue;
#pragma unroll
        for (int i = 0; i < N; i += VEC) {
            const int e = bal_elem<L, VEC>(i, r);
            if (e >= p.E) continue;
            const size_t at = (size_t)t * p.E + e;
            if constexpr (VEC == 4) {
                if (p.dl_bf16)
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.dlogits) + at) =
                        make_uint2(bf16x2_rn(l[i], l[i + 1]), bf16x2_rn(l[i + 2], l[i + 3]));
                else
                    *reinterpret_cast<float4*>(static_cast<float*>(p.dlogits) + at) =
                        make_float4(l[i], l[i + 1], l[i + 2], l[i + 3]);
            } else {
                if (p.dl_bf16) static_cast<uint16_t*>(p.dlogits)[at] = (uint16_t)(bf16x2_rn(l[i], 0.0f) & 0xffffu);
                else static_cast<float*>(p.dlogits)[at] = l[i];
            }
        }
    }
}

}  // namespace fe
