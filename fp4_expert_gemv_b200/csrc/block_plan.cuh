// Host-side plans of the operators around the experts: launch shapes, shared memory, workspaces and shares of
// tiles.  Plain arithmetic on sizes, no CUDA call, so that it is checked on the CPU as it is.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "balance.cuh"
#include "linear.cuh"
#include "norm.cuh"

namespace fe_plan {

inline size_t align256(size_t n) { return (n + 255) & ~(size_t)255; }

// CTAs that leave partial sums over rows, at most: two on each of 148 SMs.  The workspace sizes must not depend
// on the device that is current when they are asked for, so a grid keeps to this number instead.
constexpr int kMaxPartials = 296;

// ---- norms ------------------------------------------------------------------------------

// Threads of a row: 8 elements each, as many as cover the row, from one warp to 1024.
inline int norm_threads(int H, int chunk)
{
    int tpr = 32;
    while (tpr < 1024 && tpr * 8 * chunk < H) tpr *= 2;
    return tpr;
}

// The streamed kernels' launch: groups of tpr threads with 16 columns each, a CTA of 512 threads per SM, as
// many stages (to four) as fit.
struct NormRingPlan {
    int tpr, threads, stages, grid;
    size_t smem;
};

constexpr size_t kNormRingSmem = 220 * 1024;

inline bool norm_ring_plan(int64_t T, int H, uint32_t stage, int sms, NormRingPlan* b)
{
    b->tpr = norm_threads(H, fe::kRingC);
    if (b->tpr > 512) return false;
    b->threads = 512;
    const int groups = b->threads / b->tpr;
    for (b->stages = 4; b->stages >= 2; --b->stages) {
        b->smem = (size_t)groups * (b->stages * stage + fe::norm_group_extra(b->tpr, b->stages));
        if (b->smem <= kNormRingSmem) break;
    }
    b->grid = (int)std::min<int64_t>(std::min(sms, kMaxPartials), (T + groups - 1) / groups);
    return b->stages >= 2;
}

// Shared memory of the streamed backward pass's end: three sums of each of the groups.
inline size_t norm_ring_sums(const NormRingPlan& b, int H) { return sizeof(float) * 3 * (size_t)H * (b.threads / b.tpr); }

// The column-by-column backward pass: groups of up to 512 threads a row, two CTAs an SM, a group's two sums
// over rows and its exchange in shared memory.
struct NormColumnsPlan {
    int tpr, threads, grid;
    size_t smem;
};

inline NormColumnsPlan norm_columns_plan(int64_t T, int H, int sms)
{
    NormColumnsPlan b;
    b.threads = 512;
    b.tpr = std::min(b.threads, norm_threads(H, 1));
    const int groups = b.threads / b.tpr;
    b.smem = sizeof(float) * groups * (2 * (size_t)fe::norm_red_floats(b.tpr) + 2 * (size_t)H);
    b.grid = (int)std::min<int64_t>(std::min(2 * sms, kMaxPartials), (T + groups - 1) / groups);
    return b;
}

// Three sums of H from every CTA that leaves some.
inline size_t norm_workspace(int64_t T, int H)
{
    return sizeof(float) * 3 * (size_t)H * (size_t)std::min<int64_t>(kMaxPartials, std::max<int64_t>(T, 1));
}

// ---- balance loss -------------------------------------------------------------------------

// Lanes that hold a row of E logits, 16 values each (32 beyond 512).
inline int balance_lanes(int E)
{
    int l = 1;
    while (l < 32 && 16 * l < E) l *= 2;
    return l;
}

// CTAs of the forward pass: a group of rows per warp, up to kMaxBalanceCtas of them.
constexpr int kMaxBalanceCtas = 444;
inline int balance_ctas(int64_t T, int E)
{
    const int rows = fe::kBalWarps * (32 / balance_lanes(E));
    return (int)std::max<int64_t>(1, std::min<int64_t>(kMaxBalanceCtas, (T + rows - 1) / rows));
}

// Rows that one cluster takes by itself, two groups per warp: with the rows in registers (64 x 128: 3.9 us),
// then through the rings, which have more warps but want whole 16-byte pieces (1024 x 128: 7.4 us, 8.1 from
// registers).  Beyond, two launches are faster: 2048 x 128 takes 8.2 us, 9.2 in one; 4096 8.9, 13.3 in one,
// as eight SMs take in too little.
inline int64_t balance_small(int E) { return (int64_t)2 * fe::kBalCluster * fe::kBalWarps * (32 / balance_lanes(E)); }

inline bool balance_fused(int64_t T, int E)
{
    if (E % 4 != 0) return T <= 2 * balance_small(E);
    return T <= (int64_t)2 * fe::kBalCluster * fe::bal_ring_warps(E > 512 ? 32 : 16) * (32 / balance_lanes(E));
}

// CTAs of the streamed pass over many rows: enough for a group of rows per two warps, a CTA an SM at most, and no
// more than the workspace has partials for: the second pass has the fewer to join.
inline int balance_ring_ctas(int64_t T, int E, int sms)
{
    const int rows = 32 / balance_lanes(E), W = fe::bal_ring_warps(E > 512 ? 32 : 16);
    const int64_t groups = (T + rows - 1) / rows;
    return (int)std::min<int64_t>(std::min(sms, balance_ctas(T, E)), (2 * groups + W - 1) / W);
}

// A partial is E + 1 sums and as many counts.
inline size_t balance_workspace(int64_t T, int E) { return balance_fused(T, E) ? 0 : 8 * (size_t)balance_ctas(T, E) * ((size_t)E + 1); }

// Dynamic shared memory of the streamed pass, and the stages of a warp's ring (to eight) that fit, each a
// group of 32 / L rows.
constexpr int balance_ring_room(int L, int N)
{
    return fe::kBalRingSmem - 4 * L * N - 1024 - 8 * fe::kBalRingStages * fe::bal_ring_warps(N);
}

inline int balance_stages(int E, int L, int N)
{
    return std::min(fe::kBalRingStages, balance_ring_room(L, N) / (4 * (32 / L) * E * fe::bal_ring_warps(N)));
}

// The rings, and over them at the end a row of sums per warp.
inline size_t balance_ring_smem(int E, int L, int N)
{
    const int W = fe::bal_ring_warps(N);
    return std::max((size_t)balance_stages(E, L, N) * W * 4 * (32 / L) * E, sizeof(float) * W * L * N);
}

// ---- dense product --------------------------------------------------------------------------

inline int lin_tile_cols(const fe::LinProblem& p, int BN) { return p.act == fe::kActSwiglu ? BN / 2 : BN; }

// The tile width (0: 256, 1: 192, 2: 128) whose busiest pair has least to do.  A k step of 256 columns takes 512
// cycles of products; narrower ones less, but a little more per column (A is read as often).
inline int lin_width(const fe::LinParams& P, int n, int pairs)
{
    const int widths[3] = {256, 192, 128};
    const int64_t cost[3] = {512, 392, 272};
    int best = 0;
    int64_t least = INT64_MAX;
    for (int w = 0; w < 3; ++w) {
        int64_t total = 0, longest = 0;
        for (int i = 0; i < n; ++i) {
            const int tc = lin_tile_cols(P.p[i], widths[w]);
            const int64_t tiles = (int64_t)((P.p[i].cols + tc - 1) / tc) * ((P.p[i].M + fe::kLinM - 1) / fe::kLinM);
            const int64_t steps = (P.p[i].K + 63) / 64 + 2;
            if (n == 1) total = (tiles + pairs - 1) / pairs * steps * pairs;
            else total += tiles * steps;
            longest = std::max(longest, steps);
        }
        const int64_t c = std::max((total + pairs - 1) / pairs, longest) * cost[w];
        if (c < least) {
            least = c;
            best = w;
        }
    }
    return best;
}

// Shares out two problems' tiles, the first's (fewer and longer) evenly, the second's so that the pairs
// end together: the smallest finish time, found by bisection, that has room for all of them.
inline void lin_share(fe::LinParams& P, int pairs)
{
    const int64_t ca = (P.p[0].K + 63) / 64 + 2, cb = (P.p[1].K + 63) / 64 + 2;   // k steps, and a tile's ends
    const int na = P.p[0].tiles, nb = P.p[1].tiles;
    auto load = [&](int c) { return (int64_t)(na / pairs + (c < na % pairs ? 1 : 0)) * ca; };
    const int64_t la = load(0), lb = load(pairs - 1);
    const int xa = na % pairs;
    auto room = [&](int64_t L) {
        return (L > la ? (L - la) / cb : 0) * xa + (L > lb ? (L - lb) / cb : 0) * (pairs - xa);
    };
    int64_t lo = 0, hi = la + cb * ((int64_t)nb + 1);
    while (lo < hi) {
        const int64_t mid = (lo + hi) / 2;
        if (room(mid) >= nb) hi = mid;
        else lo = mid + 1;
    }
    int ta = 0, tb = 0;
    for (int c = 0; c < pairs; ++c) {
        P.start[0][c] = ta;
        P.start[1][c] = tb;
        ta += na / pairs + (c < xa ? 1 : 0);
        const int64_t l = load(c);
        tb += (int)std::min<int64_t>(nb - tb, lo > l ? (lo - l) / cb : 0);
    }
    P.start[0][pairs] = na;
    P.start[1][pairs] = nb;
}

constexpr int kSplSmem = 227 * 1024;   // all that a CTA can have

// CTAs that share a tile's contraction (a power of two, to 8) and the tile's columns: of those whose
// clusters all run at once (room[lg]: clusters of 2^lg), with two k steps or more a CTA, the least that an SM has
// to take in, which is what bounds these products: its k steps' operands at 72 bytes a clock (measured), and its
// share of the other CTAs' partial sums, which cross between SMs at a fifth of that.  1024 x 1000, K = 2048: 9.0 us
// with 128 columns and two CTAs (9.5 when both were measured), 10.6 us with 64 and no split; 256 x 2048, K = 768: 5.6 us with 64 columns and
// two, 7.6 us with 128 and four.  ways 0 if the tiles alone fill the SMs.
inline void split_choice(bool glu, int cols, int M, int K, const int (&room)[4], int* ways, int* BN)
{
    *ways = 0;
    int64_t least = INT64_MAX;
    const int steps = (K + 63) / 64;
    for (const int bn : {64, 128}) {
        const int w = glu ? bn / 2 : bn;
        const int64_t tiles = (int64_t)((cols + w - 1) / w) * ((M + 127) / 128);
        for (int lg = bn == 64 ? 0 : 1; lg <= 3; ++lg) {   // 128 columns' sums and stages fit with a split only
            const int n = 1 << lg;
            if (tiles > room[lg] || (lg > 0 && steps < 2 * n)) break;
            const int rows = std::min(M, 128);
            const int64_t cost = (int64_t)((steps + n - 1) / n) * 128 * (rows + bn) + 5 * 4 * bn * rows / n * (n - 1);
            if (cost < least) {
                least = cost;
                *ways = n;
                *BN = bn;
            }
        }
    }
}

// Stages of a CTA's ring: its k steps, as many as fit beside the sums and the residual.
inline int split_stages(int K, int BN, int splits, uint32_t res_bytes)
{
    int stages = std::min(fe::kSplMaxStages, ((K + 63) / 64 + splits - 1) / splits);
    while (fe::spl_smem(BN, stages, res_bytes) > kSplSmem) --stages;
    return stages;
}

// Backward workspace: dz [M][roundup8(N)] bf16 where it is written, then the column partials behind db.
inline int dz_chunks(int64_t M) { return (int)std::max<int64_t>(1, std::min<int64_t>(256, (M + 31) / 32)); }
inline int64_t dz_rows(int64_t M) { return (M + dz_chunks(M) - 1) / dz_chunks(M); }   // of a chunk, the last may have fewer
inline size_t dz_bytes(int64_t M, int N, bool written) { return written ? align256(2 * (size_t)M * (((size_t)N + 7) / 8 * 8)) : 0; }
inline size_t db_bytes(int64_t M, int N, bool db) { return db ? sizeof(float) * (size_t)dz_chunks(M) * N : 0; }
// dz is dy itself without an activation, when its rows suit TMA; db alone needs none.
inline bool dz_written(int act, bool dy_rows16, bool dx, bool dw) { return (dx || dw) && !(act == fe::kActNone && dy_rows16); }

}  // namespace fe_plan
