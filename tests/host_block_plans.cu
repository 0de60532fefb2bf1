// Host-side checks of the plans of the operators around the experts, compiled from the library's own header and run
// on the CPU (tests/test_host_plans.py): every workspace holds what the grids write, every layout fits its shared
// memory, every tile and k step belongs to exactly one CTA, rows and sums are covered.  Prints "ok" or the first
// failed checks, and exits nonzero on a failure.
#include <cstdio>
#include <cstdlib>
#include <vector>

#include "../fp4_expert_gemv_b200/csrc/block_plan.cuh"

using namespace fe_plan;

static int failures = 0;
#define CHECK(cond, ...)                                        \
    do {                                                        \
        if (!(cond)) {                                          \
            if (failures++ < 10) {                              \
                std::printf("FAILED %s: ", #cond);              \
                std::printf(__VA_ARGS__);                       \
                std::printf("\n");                              \
            }                                                   \
        }                                                       \
    } while (0)

constexpr size_t kMaxSmem = 227 * 1024;   // dynamic shared memory a block may opt into

static void norms()
{
    for (int sms : {1, 132, 148, 160})
        for (int H = 1; H <= fe::kNormMaxH; H += H < 600 ? 1 : H < 4000 ? 37 : 411)
            for (int64_t T : {1ll, 2ll, 5ll, 147ll, 148ll, 149ll, 295ll, 296ll, 297ll, 600ll, 4096ll, 100000ll, (1ll << 31) - 1}) {
                const size_t room = norm_workspace(T, H) / (sizeof(float) * 3 * H);
                const NormColumnsPlan c = norm_columns_plan(T, H, sms);
                CHECK(c.grid >= 1 && (size_t)c.grid <= room && c.grid <= 2 * sms, "columns T=%lld H=%d sms=%d", (long long)T, H, sms);
                CHECK(c.smem <= kNormRingSmem && c.tpr >= 32 && c.tpr <= 512 && (c.tpr & (c.tpr - 1)) == 0, "columns H=%d", H);
                // whole warps of a row's threads in groups: a barrier per group, sixteen at most
                CHECK(c.threads / c.tpr <= 16, "columns H=%d", H);
                if (H % 8) continue;
                for (int f32 = 0; f32 < 2; ++f32)
                    for (int full = 0; full < 2; ++full) {
                        const uint32_t stages[3] = {fe::norm_fwd_stage(H, f32, true, full), fe::norm_fwd_stage(H, f32, false, false),
                                                    fe::norm_bwd_stage(H, f32, full)};
                        for (uint32_t stage : stages) {
                            NormRingPlan b;
                            CHECK(stage % 16 == 0, "H=%d stage=%u", H, stage);
                            if (!norm_ring_plan(T, H, stage, sms, &b)) continue;
                            const int groups = b.threads / b.tpr;
                            CHECK(b.stages >= 2 && b.stages <= 4 && b.smem <= kNormRingSmem, "ring H=%d", H);
                            CHECK(b.smem >= (size_t)groups * (b.stages * stage + 4 * 2 * fe::norm_red_floats(b.tpr) + 8 * b.stages), "ring H=%d", H);
                            CHECK(b.tpr * 8 * fe::kRingC >= H && groups <= 16, "ring H=%d", H);   // 15 named barriers and one of a single warp
                            CHECK(groups <= 15 || b.tpr == 32, "ring H=%d", H);
                            CHECK(b.grid >= 1 && b.grid <= sms && (size_t)b.grid <= room, "ring T=%lld H=%d sms=%d", (long long)T, H, sms);
                            CHECK(norm_ring_sums(b, H) <= kNormRingSmem, "ring sums H=%d", H);
                        }
                    }
            }
    for (int H = 1; H <= fe::kNormMaxH; ++H) {   // the plain kernel's threads cover the row
        const int chunk = H <= 8192 ? 1 : 2;
        CHECK(norm_threads(H, chunk) * 8 * chunk >= H && norm_threads(H, chunk) <= 1024, "H=%d", H);
    }
}

static void balance()
{
    for (int E = 1; E <= fe::kBalMaxE; E += E < 70 || E > 500 ? 1 : 7) {
        const int L = balance_lanes(E), N = E > 512 ? 32 : 16, R = 32 / L;
        CHECK(L * N >= E && L <= 32, "E=%d", E);
        if (E % 4 == 0) {
            const int W = fe::bal_ring_warps(N), stages = balance_stages(E, L, N);
            CHECK(stages >= 2 && stages <= fe::kBalRingStages, "E=%d stages=%d", E, stages);
            const size_t fixed = 4 * L * N + 4 * 32 + 8 + 4 * 32 + 4 + 8 * fe::kBalRingStages * W;   // static arrays
            CHECK(balance_ring_smem(E, L, N) <= (size_t)balance_ring_room(L, N), "E=%d", E);
            CHECK(balance_ring_smem(E, L, N) + fixed <= kMaxSmem, "E=%d", E);
            CHECK(balance_ring_smem(E, L, N) >= (size_t)W * stages * 4 * R * E && balance_ring_smem(E, L, N) >= sizeof(float) * W * L * N, "E=%d", E);
        }
        for (int64_t T = 0; T < 6000; T += T < 700 ? 1 : 53)
            for (int sms : {1, 132, 148, 160}) {
                const size_t ws = balance_workspace(T, E);
                if (balance_fused(T, E)) {
                    CHECK(ws == 0, "E=%d T=%lld", E, (long long)T);
                    continue;
                }
                // partials of both forms of the first pass: [G][E] and [G] floats, the same of ints
                CHECK((size_t)balance_ctas(T, E) * (E + 1) * 8 <= ws, "E=%d T=%lld", E, (long long)T);
                const int G = balance_ring_ctas(T, E, sms);
                CHECK(G >= 1 && G <= sms && (size_t)G * (E + 1) * 8 <= ws, "E=%d T=%lld sms=%d G=%d", E, (long long)T, sms, G);
            }
    }
}

static fe::LinProblem problem(int M, int N, int K, int act, int BN)
{
    fe::LinProblem p{};
    p.M = M;
    p.N = N;
    p.K = K;
    p.act = act;
    p.cols = act == fe::kActSwiglu ? N / 2 : N;
    const int w = lin_tile_cols(p, BN);
    p.tiles_n = (p.cols + w - 1) / w;
    p.tiles = p.tiles_n * ((M + fe::kLinM - 1) / fe::kLinM);
    return p;
}

static void products()
{
    const int sizes[] = {8, 64, 72, 96, 264, 768, 1000, 1536, 2048, 4096, 5000, 16384, 100000};
    static fe::LinParams P;
    for (int M : sizes)
        for (int N : sizes)
            for (int K : sizes) {
                if ((int64_t)M * N * K > (int64_t)1 << 41) continue;
                for (int room : {1, 60, 74, 80, fe::kLinMaxPairs}) {
                    // dW [N][K] over M, dX [M][K] over N
                    P.n = 2;
                    P.p[0] = problem(N, K, M, fe::kActNone, 256);
                    P.p[1] = problem(M, K, N, fe::kActNone, 256);
                    const int width = lin_width(P, 2, room), BN = width == 0 ? 256 : width == 1 ? 192 : 128;
                    P.p[0] = problem(N, K, M, fe::kActNone, BN);
                    P.p[1] = problem(M, K, N, fe::kActNone, BN);
                    const int pairs = std::min(room, P.p[0].tiles + P.p[1].tiles);
                    lin_share(P, pairs);
                    // each problem's tiles in order, every one given once
                    int64_t longest = 0, total = 0;
                    const int64_t c0 = (P.p[0].K + 63) / 64 + 2, c1 = (P.p[1].K + 63) / 64 + 2;
                    for (int i = 0; i < 2; ++i) {
                        CHECK(P.start[i][0] == 0 && P.start[i][pairs] == P.p[i].tiles, "M=%d N=%d K=%d pairs=%d", M, N, K, pairs);
                        for (int c = 0; c < pairs; ++c) CHECK(P.start[i][c] <= P.start[i][c + 1], "M=%d N=%d K=%d pairs=%d c=%d", M, N, K, pairs, c);
                    }
                    for (int c = 0; c < pairs; ++c) {
                        const int64_t l = (P.start[0][c + 1] - P.start[0][c]) * c0 + (P.start[1][c + 1] - P.start[1][c]) * c1;
                        longest = std::max(longest, l);
                        total += l;
                    }
                    // no pair ends more than a tile of each problem after the mean
                    CHECK(longest <= (total + pairs - 1) / pairs + c0 + c1, "M=%d N=%d K=%d pairs=%d longest=%lld total=%lld", M, N, K, pairs, (long long)longest, (long long)total);
                }
            }
    // the contraction's split
    const int rooms[3][4] = {{148, 74, 36, 16}, {148, 74, 33, 14}, {1, 1, 1, 1}};
    for (const auto& room : rooms)
        for (int M = 17; M <= 3000; M += M < 300 ? 1 : 61)
            for (int N : {2, 8, 64, 66, 500, 1000, 1536, 2048, 4096})
                for (int K : {8, 64, 72, 136, 768, 1992, 2048, 16384})
                    for (int glu = 0; glu < 2; ++glu) {
                        const int cols = glu ? N / 2 : N;
                        int ways = 0, BN = 0;
                        split_choice(glu, cols, M, K, room, &ways, &BN);
                        if (ways == 0) continue;
                        const int steps = (K + 63) / 64, w = glu ? BN / 2 : BN;
                        CHECK(BN == 64 || BN == 128, "M=%d N=%d K=%d", M, N, K);
                        CHECK(ways == 1 || ways == 2 || ways == 4 || ways == 8, "M=%d N=%d K=%d", M, N, K);
                        const int lg = ways == 1 ? 0 : ways == 2 ? 1 : ways == 4 ? 2 : 3;
                        CHECK((int64_t)((cols + w - 1) / w) * ((M + 127) / 128) <= room[lg], "M=%d N=%d K=%d", M, N, K);
                        int k = 0;   // every CTA has k steps, together all of them
                        for (int r = 0; r < ways; ++r) {
                            const int k0 = (int)((int64_t)steps * r / ways), k1 = (int)((int64_t)steps * (r + 1) / ways);
                            CHECK(k0 == k && k1 > k0, "M=%d N=%d K=%d r=%d", M, N, K, r);
                            k = k1;
                        }
                        CHECK(k == steps, "K=%d", K);
                        for (uint32_t res : {0u, (uint32_t)(128 / ways * w * 2)}) {
                            const int stages = split_stages(K, BN, ways, res);
                            CHECK(stages >= 1 && stages <= fe::kSplMaxStages && fe::spl_smem(BN, stages, res) <= kMaxSmem, "BN=%d ways=%d stages=%d", BN, ways, stages);
                            CHECK(2 * stages + 1 <= fe::kSplThreads && res % 16 == 0, "BN=%d ways=%d", BN, ways);
                        }
                    }
    // dz: the chunks cover the rows, and the partials fit
    for (int64_t M : {1ll, 31ll, 32ll, 33ll, 8191ll, 8192ll, 8193ll, 100000ll, 2200000ll, (1ll << 31) - 257})
        for (int N : {1, 7, 8, 264}) {
            const int64_t rows = dz_rows(M), used = (M + rows - 1) / rows;
            CHECK(used <= dz_chunks(M) && used >= 1 && used * rows >= M, "M=%lld", (long long)M);
            CHECK(db_bytes(M, N, true) >= sizeof(float) * (size_t)used * N && db_bytes(M, N, false) == 0, "M=%lld N=%d", (long long)M, N);
            CHECK(dz_bytes(M, N, true) >= 2 * (size_t)M * N && dz_bytes(M, N, true) % 256 == 0 && dz_bytes(M, N, false) == 0, "M=%lld N=%d", (long long)M, N);
        }
}

int main()
{
    norms();
    balance();
    products();
    if (failures) std::printf("%d failed\n", failures);
    else std::printf("ok\n");
    return failures != 0;
}
