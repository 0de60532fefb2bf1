// Entry points of the operators around the expert layer: the block's norms with gate and residual,
// the router's balance loss, and the dense product with its epilogue.  They need no handle: the
// caller passes every buffer, workspace included, and they run on the current device.  The
// declarations and the contract of every entry point are in include/fe_moe.h.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "../../include/fe_moe.h"
#include "balance.cuh"
#include "block_plan.cuh"
#include "common.cuh"
#include "host.h"
#include "linear.cuh"
#include "norm.cuh"

using fe_host::record_cuda;

using namespace fe_plan;

namespace {

#define FE_CUDA_TRY(expr)                                 \
    do {                                                  \
        cudaError_t err__ = (expr);                       \
        if (err__ != cudaSuccess) return record_cuda(err__, #expr); \
    } while (0)

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

using fe_host::overlap;
using fe_host::overlap_rows;

// SMs of the current device (looked up once per device).
int sm_count()
{
    static std::atomic<int> known[64];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = known[dev].load(std::memory_order_relaxed);
    if (n == 0) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
        known[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

// Every kernel here begins with griddepcontrol.wait, so its launch may overlap the tail of the
// kernel before it on the stream.
template <typename... KArgs, typename... Args>
cudaError_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t s, const Args&... args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// ---- norms ------------------------------------------------------------------------------

size_t dtype_bytes(int dt) { return dt == FE_DTYPE_F32 ? 4 : 2; }

bool gate_ok(int kind)
{
    const int k = kind & ~FE_GATE_SIGMOID;
    return (k == FE_GATE_NONE && kind == FE_GATE_NONE) || k == FE_GATE_CHANNEL || k == FE_GATE_TOKEN || k == FE_GATE_FULL;
}

size_t gate_elems(int kind, int64_t T, int H)
{
    switch (kind & ~FE_GATE_SIGMOID) {
        case FE_GATE_CHANNEL: return (size_t)H;
        case FE_GATE_TOKEN: return (size_t)T;
        case FE_GATE_FULL: return (size_t)T * H;
    }
    return 0;
}

// What both directions need of the forward's operands.
fe_status check_norm_operands(const void* r, int r_dtype, const void* y, const void* w_post, const void* gate,
                              int gate_kind, const void* w_pre, float eps, int64_t T, int H)
{
    if (T < 0 || H < 1 || (r_dtype != FE_DTYPE_BF16 && r_dtype != FE_DTYPE_F32) || !gate_ok(gate_kind) ||
        !(eps > 0.0f) || std::isinf(eps))
        return FE_ERR_INVALID_ARG;
    if (T > 0 && (gate_kind == FE_GATE_NONE) != (gate == nullptr)) return FE_ERR_INVALID_ARG;
    if (T > 0 && !y && (w_post || gate)) return FE_ERR_INVALID_ARG;
    if (!aligned(r, r_dtype == FE_DTYPE_F32 ? 4 : 2) || !aligned(y, 2) || !aligned(w_post, 2) || !aligned(gate, 2) ||
        !aligned(w_pre, 2))
        return FE_ERR_INVALID_ARG;
    if (H > fe::kNormMaxH || T > INT32_MAX) return FE_ERR_UNSUPPORTED;
    return FE_OK;
}

fe::NormParams norm_params(const void* r, const void* y, const void* w_post, const void* gate, int gate_kind, float scale,
                           const void* w_pre, float eps, int64_t T, int H)
{
    fe::NormParams p{};
    p.r = r;
    p.y = static_cast<const uint16_t*>(y);
    p.w_post = static_cast<const uint16_t*>(w_post);
    p.gate = static_cast<const uint16_t*>(gate);
    p.gate_kind = gate_kind & ~FE_GATE_SIGMOID;
    p.gate_sigmoid = (gate_kind & FE_GATE_SIGMOID) != 0;
    p.scale = scale;
    p.w_pre = static_cast<const uint16_t*>(w_pre);
    p.eps = eps;
    p.T = T;
    p.H = H;
    return p;
}

// 16-byte accesses need a row length of whole chunks and every row pointer aligned.
bool norm_vec(const fe::NormParams& p)
{
    return p.H % 8 == 0 && aligned(p.r, 16) && aligned(p.y, 16) && aligned(p.w_post, 16) && aligned(p.w_pre, 16) &&
           (p.gate_kind == FE_GATE_TOKEN || aligned(p.gate, 16)) && aligned(p.r_out, 16) && aligned(p.u, 16);
}

template <int C>
cudaError_t norm_launch(const fe::NormParams& p, bool r32, int tpr, cudaStream_t s)
{
    const int threads = std::max(tpr, 128);
    const dim3 grid((unsigned)((p.T + threads / tpr - 1) / (threads / tpr)));
    if (norm_vec(p))
        return r32 ? launch(fe::block_norm_kernel<8, C, true>, grid, threads, 0, s, p, tpr)
                   : launch(fe::block_norm_kernel<8, C, false>, grid, threads, 0, s, p, tpr);
    return r32 ? launch(fe::block_norm_kernel<1, C, true>, grid, threads, 0, s, p, tpr)
               : launch(fe::block_norm_kernel<1, C, false>, grid, threads, 0, s, p, tpr);
}

// Opts a kernel into kNormRingSmem of shared memory, once per device.
template <typename K>
cudaError_t norm_ring_ready(K kernel, std::atomic<bool>* ready)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kNormRingSmem);
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
    return cudaSuccess;
}

template <bool R32, int GATE, bool Y>
cudaError_t norm_ring_launch(const fe::NormParams& p, const NormRingPlan& b, cudaStream_t s)
{
    static std::atomic<bool> ready[64];
    const auto kernel = fe::block_norm_ring_kernel<R32, GATE, Y>;
    const cudaError_t e = norm_ring_ready(kernel, ready);
    if (e != cudaSuccess) return e;
    return launch(kernel, b.grid, b.threads, b.smem, s, p, b.tpr, b.stages);
}

template <bool R32>
cudaError_t norm_ring(const fe::NormParams& p, const NormRingPlan& b, cudaStream_t s)
{
    if (!p.y) return norm_ring_launch<R32, fe::kByRow, false>(p, b, s);
    if (p.gate_kind == FE_GATE_CHANNEL) return norm_ring_launch<R32, fe::kByColumn, true>(p, b, s);
    if (p.gate_kind == FE_GATE_FULL) return norm_ring_launch<R32, fe::kByElement, true>(p, b, s);
    return norm_ring_launch<R32, fe::kByRow, true>(p, b, s);
}

template <bool R32, int GATE, bool ALL>
cudaError_t norm_bwd_columns(const fe::NormBwdParams& q, int sms, int* partials, cudaStream_t s)
{
    static std::atomic<bool> ready[64];
    const NormColumnsPlan b = norm_columns_plan(q.f.T, q.f.H, sms);
    *partials = b.grid;
    const auto kernel = fe::block_norm_backward_any_kernel<R32, GATE, ALL>;
    const cudaError_t e = norm_ring_ready(kernel, ready);
    if (e != cudaSuccess) return e;
    return launch(kernel, b.grid, b.threads, b.smem, s, q, b.tpr);
}

// Through the ring when rows are whole aligned chunks and every operand is there, else column by column.
template <bool R32, int GATE>
cudaError_t norm_bwd_any(const fe::NormBwdParams& q, bool vec, int sms, int* partials, cudaStream_t s)
{
    static std::atomic<bool> ring_ready[64];
    const int H = q.f.H;
    NormRingPlan b;
    if (vec && q.f.y && q.du && q.dr_out &&
        norm_ring_plan(q.f.T, H, fe::norm_bwd_stage(H, R32, GATE == fe::kByElement), sms, &b)) {
        b.smem = std::max(b.smem, norm_ring_sums(b, H));
        *partials = b.grid;
        const auto kernel = fe::block_norm_backward_ring_kernel<R32, GATE>;
        const cudaError_t e = norm_ring_ready(kernel, ring_ready);
        if (e != cudaSuccess) return e;
        return launch(kernel, b.grid, b.threads, b.smem, s, q, b.tpr, b.stages);
    }
    const bool all = q.f.y && q.f.w_post && q.du && q.dr_out && q.dr && q.dy && (GATE != fe::kByElement || q.dgate);
    return all ? norm_bwd_columns<R32, GATE, true>(q, sms, partials, s) : norm_bwd_columns<R32, GATE, false>(q, sms, partials, s);
}

template <bool R32>
cudaError_t norm_bwd(const fe::NormBwdParams& q, bool vec, int sms, int* partials, cudaStream_t s)
{
    if (q.f.gate_kind == FE_GATE_CHANNEL) return norm_bwd_any<R32, fe::kByColumn>(q, vec, sms, partials, s);
    if (q.f.gate_kind == FE_GATE_FULL) return norm_bwd_any<R32, fe::kByElement>(q, vec, sms, partials, s);
    return norm_bwd_any<R32, fe::kByRow>(q, vec, sms, partials, s);
}

// ---- balance loss -------------------------------------------------------------------------

fe_status check_balance(const float* logits, int64_t T, int E, int top_k)
{
    if (T < 0 || E < 1 || top_k < 1 || top_k > E || (T > 0 && !logits) || !aligned(logits, 4)) return FE_ERR_INVALID_ARG;
    if (E > fe::kBalMaxE || T > INT32_MAX / top_k) return FE_ERR_UNSUPPORTED;
    return FE_OK;
}

template <int L, int N, int VEC>
cudaError_t balance_run(const fe::BalanceParams& p, bool backward, int grid, cudaStream_t s)
{
    if (backward) return launch(fe::balance_backward_kernel<L, N, VEC>, grid, fe::kBalThreads, 0, s, p);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(fe::kBalThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.G > 0 ? 1 : grid;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fe::balance_kernel<L, N, VEC>, p);
}

template <int L, int N>
cudaError_t balance_ring_run(const fe::BalanceParams& p, cudaStream_t s)
{
    static std::atomic<bool> ready[64];
    const int W = fe::bal_ring_warps(N), stages = balance_stages(p.E, L, N);
    const size_t smem = balance_ring_smem(p.E, L, N);
    const auto kernel = fe::balance_ring_kernel<L, N>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, balance_ring_room(L, N));
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.G > 0 ? p.G : fe::kBalCluster);
    cfg.blockDim = dim3(32 * W);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = p.G > 0 ? 1 : fe::kBalCluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p, stages);
}

cudaError_t balance_ring_dispatch(const fe::BalanceParams& p, cudaStream_t s)
{
    if (p.E > 512) return balance_ring_run<32, 32>(p, s);
    switch (balance_lanes(p.E)) {
        case 1: return balance_ring_run<1, 16>(p, s);
        case 2: return balance_ring_run<2, 16>(p, s);
        case 4: return balance_ring_run<4, 16>(p, s);
        case 8: return balance_ring_run<8, 16>(p, s);
        case 16: return balance_ring_run<16, 16>(p, s);
    }
    return balance_ring_run<32, 16>(p, s);
}

template <int L, int N>
cudaError_t balance_vec(const fe::BalanceParams& p, bool backward, int grid, bool vec, cudaStream_t s)
{
    return vec ? balance_run<L, N, 4>(p, backward, grid, s) : balance_run<L, N, 1>(p, backward, grid, s);
}

cudaError_t balance_dispatch(const fe::BalanceParams& p, bool backward, int grid, bool vec, cudaStream_t s)
{
    if (p.E > 512) return balance_vec<32, 32>(p, backward, grid, vec, s);
    switch (balance_lanes(p.E)) {
        case 1: return balance_vec<1, 16>(p, backward, grid, vec, s);
        case 2: return balance_vec<2, 16>(p, backward, grid, vec, s);
        case 4: return balance_vec<4, 16>(p, backward, grid, vec, s);
        case 8: return balance_vec<8, 16>(p, backward, grid, vec, s);
        case 16: return balance_vec<16, 16>(p, backward, grid, vec, s);
    }
    return balance_vec<32, 16>(p, backward, grid, vec, s);
}

// ---- dense product --------------------------------------------------------------------------


bool act_ok(int act, int N) { return act >= FE_ACT_NONE && act <= FE_ACT_SWIGLU && (act != FE_ACT_SWIGLU || N % 2 == 0); }
int out_cols(int act, int N) { return act == FE_ACT_SWIGLU ? N / 2 : N; }

// Bytes that M rows of `cols` bf16 with stride ld span.
size_t span(int64_t M, int64_t ld, int64_t cols) { return M > 0 ? 2 * ((size_t)(M - 1) * ld + cols) : 0; }

fe_status check_linear_shape(int64_t M, int N, int K, int act)
{
    if (M < 0 || N < 1 || K < 1 || !act_ok(act, N)) return FE_ERR_INVALID_ARG;
    // TMA rows are multiples of 16 bytes; tile counts and coordinates are 32-bit
    if (K % 8 != 0 || M > INT32_MAX - 256 || N > INT32_MAX - 256 || K > INT32_MAX - 256 ||
        (M / 128 + 1) * (int64_t)(std::max(N, K) / 64 + 1) > INT32_MAX / 4 ||
        (int64_t)(N / 128 + 1) * (K / 64 + 1) > INT32_MAX / 4)
        return FE_ERR_UNSUPPORTED;
    return FE_OK;
}

typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                             const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn()
{
    static EncodeFn fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// Map over a bf16 matrix [rows][cols] with row stride ld (elements), boxes of bc columns x br rows in
// the swizzle of their row's bytes; zeros outside, nothing stored there.
cudaError_t tensor_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int bc, int br)
{
    EncodeFn fn = encode_fn();
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(rows > 1 ? ld : (cols + 7) / 8 * 8) * 2};
    const cuuint32_t box[2] = {(cuuint32_t)bc, (cuuint32_t)br}, es[2] = {1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box, es,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, bc == 64 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

struct Matrix {
    const void* p;
    int64_t rows, cols, ld;
};

// D [M][N] = A B^T with its operands as stored: a_mn: A is [K][M]; b_mn: B is [K][N].
struct Product {
    Matrix a, b;
    bool a_mn, b_mn;
    int M, N, K;
};

// Rows of 16 bytes: what a TMA box needs of its matrix.
bool tma_rows(const void* p, int64_t rows, int64_t ld) { return aligned(p, 16) && (rows <= 1 || ld % 8 == 0); }

// CTA pairs that run at once (looked up once per device and kernel).
template <int BN, bool PLAIN>
cudaError_t lin_pairs(int* pairs)
{
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int n = known[dev].load(std::memory_order_acquire);
    if (n == 0) {
        e = cudaFuncSetAttribute(fe::linear_gemm_kernel<BN, PLAIN>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)fe::lin_smem(BN, PLAIN));
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(2);
        cfg.blockDim = dim3(fe::kLinThreads);
        cfg.dynamicSmemBytes = fe::lin_smem(BN, PLAIN);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 2;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, fe::linear_gemm_kernel<BN, PLAIN>, &cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorLaunchOutOfResources;
        n = std::min(n, fe::kLinMaxPairs);
        known[dev].store(n, std::memory_order_release);
    }
    *pairs = n;
    return cudaSuccess;
}

template <int BN, bool PLAIN>
cudaError_t lin_launch(fe::LinParams& P, const Product* f, int n, cudaStream_t s)
{
    int pairs = 0;
    cudaError_t e = lin_pairs<BN, PLAIN>(&pairs);
    P.n = n;
    int tiles = 0;
    for (int i = 0; i < n && e == cudaSuccess; ++i) {
        fe::LinProblem& p = P.p[i];
        const int w = lin_tile_cols(p, BN);
        p.tiles_n = (p.cols + w - 1) / w;
        p.tiles = p.tiles_n * ((p.M + fe::kLinM - 1) / fe::kLinM);
        tiles += p.tiles;
        e = tensor_map(&p.ta, f[i].a.p, f[i].a.rows, f[i].a.cols, f[i].a.ld, 64, p.a_mn ? 64 : 128);
        if (e == cudaSuccess)
            e = tensor_map(&p.tb, f[i].b.p, f[i].b.rows, f[i].b.cols, f[i].b.ld, 64, p.b_mn ? 64 : BN / 2);
        if (e == cudaSuccess && p.vec_out) e = tensor_map(&p.to, p.out, p.M, p.cols, p.ldo, 32, 32);
        if (e == cudaSuccess && p.vec_res) e = tensor_map(&p.tr, p.res, p.M, p.cols, p.ldr, 32, 32);
        if (e == cudaSuccess && p.vec_z) e = tensor_map(&p.tz, p.z, p.M, p.N, p.N, 32, 32);
    }
    if (e != cudaSuccess) return e;
    pairs = std::min(pairs, tiles);
    if (n == 2) lin_share(P, pairs);
    return launch(fe::linear_gemm_kernel<BN, PLAIN>, dim3(2 * pairs), dim3(fe::kLinThreads), fe::lin_smem(BN, PLAIN), s, P);
}

// Runs one product, or two in one launch, with the epilogues already in P.p.
cudaError_t lin_run(fe::LinParams& P, const Product* f, int n, cudaStream_t s)
{
    for (int i = 0; i < n; ++i) {
        fe::LinProblem& p = P.p[i];
        p.M = f[i].M;
        p.N = f[i].N;
        p.K = f[i].K;
        p.a_mn = f[i].a_mn;
        p.b_mn = f[i].b_mn;
        p.vec_out = tma_rows(p.out, p.M, p.ldo);
        p.vec_res = p.res && tma_rows(p.res, p.M, p.ldr);
        p.vec_z = p.z && tma_rows(p.z, p.M, p.N) && (p.act != FE_ACT_SWIGLU || p.cols % 8 == 0);
    }
    int pairs = 0;
    const cudaError_t e = lin_pairs<256, true>(&pairs);
    if (e != cudaSuccess) return e;
    const int best = lin_width(P, n, pairs);
    bool plain = true;   // nothing but the product: the lean epilogue
    for (int i = 0; i < n; ++i) plain &= P.p[i].act == FE_ACT_NONE && !P.p[i].bias && !P.p[i].res && !P.p[i].z;
    if (plain)
        return best == 0   ? lin_launch<256, true>(P, f, n, s)
               : best == 1 ? lin_launch<192, true>(P, f, n, s)
                           : lin_launch<128, true>(P, f, n, s);
    return best == 0   ? lin_launch<256, false>(P, f, n, s)
           : best == 1 ? lin_launch<192, false>(P, f, n, s)
                       : lin_launch<128, false>(P, f, n, s);
}

// Products of few tiles, the contraction split over clusters.
template <bool GLU, int BN, bool VEC>
cudaError_t split_launch(const fe::LinProblem& q, const Product& f, int splits, cudaStream_t s)
{
    static std::atomic<bool> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(fe::linear_split_kernel<GLU, BN, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSplSmem);
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
    fe::LinSplitParams p{};
    e = tensor_map(&p.ta, f.a.p, f.a.rows, f.a.cols, f.a.ld, 64, 128);
    if (e == cudaSuccess) e = tensor_map(&p.tb, f.b.p, f.b.rows, f.b.cols, f.b.ld, 64, BN / 2);
    if (e != cudaSuccess) return e;
    const int w = lin_tile_cols(q, BN);
    p.M = f.M;
    p.N = f.N;
    p.K = f.K;
    p.splits = splits;
    p.act = q.act;
    p.cols = q.cols;
    p.bias = q.bias;
    p.res = q.res;
    p.ldr = q.ldr;
    p.vec_res = q.cols % 8 == 0 && q.ldr % 8 == 0 && aligned(q.res, 16);
    p.res_bytes = q.res ? 128 / splits * w * 2 : 0;
    p.stages = split_stages(f.K, BN, splits, p.res_bytes);
    p.out = q.out;
    p.ldo = q.ldo;
    p.z = q.z;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((q.cols + w - 1) / w, (f.M + 127) / 128, splits);
    cfg.blockDim = dim3(fe::kSplThreads);
    cfg.dynamicSmemBytes = fe::spl_smem(BN, p.stages, p.res_bytes);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = splits;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, fe::linear_split_kernel<GLU, BN, VEC>, p);
}

template <bool GLU>
cudaError_t split_run(const fe::LinProblem& q, const Product& f, int BN, int splits, cudaStream_t s)
{
    const bool vec = q.cols % 4 == 0 && q.ldo % 4 == 0 && aligned(q.out, 8) && aligned(q.z, 8);
    if (BN == 64)
        return vec ? split_launch<GLU, 64, true>(q, f, splits, s) : split_launch<GLU, 64, false>(q, f, splits, s);
    return vec ? split_launch<GLU, 128, true>(q, f, splits, s) : split_launch<GLU, 128, false>(q, f, splits, s);
}

// Clusters of 2^lg CTAs, one to an SM, that run at once, lg to 3 (looked up once per device): a cluster lies
// within one of the GPU's groups of SMs, so those of 8 leave some of them over.
cudaError_t split_room(int (&room)[4])
{
    static std::atomic<int> known[64][4];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    for (int lg = 0; lg <= 3; ++lg) {
        int& n = room[lg];
        n = known[dev][lg].load(std::memory_order_acquire);
        if (n != 0) continue;
        e = cudaFuncSetAttribute(fe::linear_split_kernel<false, 128, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSplSmem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(1, 1, 1 << lg);
        cfg.blockDim = dim3(fe::kSplThreads);
        cfg.dynamicSmemBytes = kSplSmem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1 << lg;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, fe::linear_split_kernel<false, 128, true>, &cfg);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorLaunchOutOfResources;
        known[dev][lg].store(n, std::memory_order_release);
    }
    return cudaSuccess;
}

// split_choice for the current device; ways 0 if the tiles alone fill the SMs.
cudaError_t split_ways(const fe::LinProblem& q, const Product& f, int* ways, int* BN)
{
    int room[4];
    const cudaError_t e = split_room(room);
    if (e != cudaSuccess) return e;
    split_choice(q.act == FE_ACT_SWIGLU, q.cols, f.M, f.K, room, ways, BN);
    return cudaSuccess;
}

template <bool GLU>
cudaError_t rows_launch(const fe::LinRowsParams& p, cudaStream_t s)
{
    if (p.M == 1) {
        const int grid = (p.cols + fe::kLinRowsWarps - 1) / fe::kLinRowsWarps;
        return launch(fe::linear_rows_kernel<GLU>, grid, 32 * fe::kLinRowsWarps, 0, s, p);
    }
    const int grid = (p.cols + (GLU ? 7 : 15)) / (GLU ? 8 : 16);
    if (p.M <= 8) return launch(fe::linear_skinny_kernel<1, GLU>, grid, 256, 0, s, p);
    return launch(fe::linear_skinny_kernel<2, GLU>, grid, 256, 0, s, p);
}

template <int VEC>
cudaError_t dz_launch(int act, dim3 grid, const fe::LinDzParams& p, cudaStream_t s)
{
    switch (act) {
        case FE_ACT_RELU: return launch(fe::linear_dz_kernel<VEC, fe::kActRelu>, grid, 256, 0, s, p);
        case FE_ACT_GELU: return launch(fe::linear_dz_kernel<VEC, fe::kActGelu>, grid, 256, 0, s, p);
        case FE_ACT_SILU: return launch(fe::linear_dz_kernel<VEC, fe::kActSilu>, grid, 256, 0, s, p);
        case FE_ACT_SWIGLU: return launch(fe::linear_dz_kernel<VEC, fe::kActSwiglu>, grid, 256, 0, s, p);
    }
    return launch(fe::linear_dz_kernel<VEC, fe::kActNone>, grid, 256, 0, s, p);
}

}  // namespace

namespace fe_host {

fe_status check_block_norm(const void* r, int r_dtype, const void* y, const void* w_post, const void* gate,
                           int gate_kind, const void* w_pre, float eps, int64_t T, int H, const void* r_out,
                           const void* u)
{
    const fe_status st = check_norm_operands(r, r_dtype, y, w_post, gate, gate_kind, w_pre, eps, T, H);
    if (st != FE_OK) return st;
    if (T == 0) return FE_OK;
    if ((u != nullptr) != (w_pre != nullptr) || (r_out && !y) || (!r_out && !u)) return FE_ERR_INVALID_ARG;
    if (!r || !aligned(r_out, r_dtype == FE_DTYPE_F32 ? 4 : 2) || !aligned(u, 2)) return FE_ERR_INVALID_ARG;
    // r_out may be r itself; no other output may touch an operand or the other output
    const size_t nr = (size_t)T * H * dtype_bytes(r_dtype), nb = (size_t)T * H * 2, nw = (size_t)H * 2;
    const size_t ng = 2 * gate_elems(gate_kind, T, H);
    const void* outs[2] = {r_out, u};
    const size_t ns[2] = {nr, nb};
    for (int i = 0; i < 2; ++i) {
        if (outs[i] != r && overlap(outs[i], ns[i], r, nr)) return FE_ERR_INVALID_ARG;
        if (i == 1 && outs[i] && outs[i] == r) return FE_ERR_INVALID_ARG;
        if (overlap(outs[i], ns[i], y, nb) || overlap(outs[i], ns[i], gate, ng) || overlap(outs[i], ns[i], w_post, nw) ||
            overlap(outs[i], ns[i], w_pre, nw))
            return FE_ERR_INVALID_ARG;
    }
    if (overlap(r_out, nr, u, nb)) return FE_ERR_INVALID_ARG;
    return FE_OK;
}

fe_status check_linear(const void* x, int64_t ldx, const void* w, const void* bias, const void* residual, int64_t ldr,
                       int64_t M, int N, int K, int act, const void* y, int64_t ldy, const void* z)
{
    const fe_status st = check_linear_shape(M, N, K, act);
    if (st != FE_OK) return st;
    const int cols = out_cols(act, N);
    if (M == 0) return FE_OK;
    if (!x || !w || !y || ldx < K || ldy < cols || (residual && ldr < cols)) return FE_ERR_INVALID_ARG;
    if (ldx % 8 != 0) return FE_ERR_UNSUPPORTED;
    if (!aligned(x, 16) || !aligned(w, 16) || !aligned(bias, 2) || !aligned(residual, 2) || !aligned(y, 2) ||
        !aligned(z, 2))
        return FE_ERR_INVALID_ARG;
    const size_t ny = span(M, ldy, cols), nz = 2 * (size_t)M * N, nx = span(M, ldx, K), nw = 2 * (size_t)N * K;
    const size_t nres = span(M, ldr, cols), nbias = 2 * (size_t)N;
    if (overlap_rows(y, ny, 2 * (size_t)ldy, 2 * (size_t)cols, x, nx, 2 * (size_t)ldx, 2 * (size_t)K) || overlap(y, ny, w, nw) || overlap(y, ny, bias, nbias) || overlap(y, ny, z, nz) ||
        overlap(z, nz, x, nx) || overlap(z, nz, w, nw) || overlap(z, nz, bias, nbias) || overlap(z, nz, residual, nres))
        return FE_ERR_INVALID_ARG;
    // y may be the residual itself (the sum in place) or lie beside it, not be a shifted view of it
    if (overlap_rows(y, ny, 2 * (size_t)ldy, 2 * (size_t)cols, residual, nres, 2 * (size_t)ldr, 2 * (size_t)cols) &&
        (y != residual || ldy != ldr))
        return FE_ERR_INVALID_ARG;
    return FE_OK;
}

}  // namespace fe_host

extern "C" {

fe_status fe_moe_block_norm(const void* r, int r_dtype, const void* y, const void* w_post, const void* gate,
                            int gate_kind, float scale, const void* w_pre, float eps, int64_t T, int H, void* r_out,
                            void* u, fe_stream_t stream)
{
    const fe_status st =
        fe_host::check_block_norm(r, r_dtype, y, w_post, gate, gate_kind, w_pre, eps, T, H, r_out, u);
    if (st != FE_OK) return st;
    if (T == 0) return FE_OK;
    fe::NormParams p = norm_params(r, y, w_post, gate, gate_kind, scale, w_pre, eps, T, H);
    p.r_out = r_out;
    p.u = static_cast<uint16_t*>(u);
    const bool r32 = r_dtype == FE_DTYPE_F32;
    const cudaStream_t s = (cudaStream_t)stream;
    // The streamed kernel pays from a few rows per group.  With it and without, us:
    //   H = 2048 (four groups on each of 148 SMs), bf16 rows: 3.5, 3.6 at one row per group, 5.0, 5.5 at two, 10.4, 13.5 at
    //   four, 38.8, 64.0 at 24; fp32 rows: 15.3, 13.3 at four, 18.7, 18.5 at six, 30.7, 33.5 at twelve, 60, 63 at 24;
    //   H = 512 (16 groups), bf16: 3.4, 3.6 at one, 4.6, 5.2 at two, 19.6, 30.9 at twelve; fp32: 13.7, 12.0 at four, 17.2,
    //   16.8 at six, 30.4, 30.4 at twelve, 63.8, 57.5 at 24;  H = 4096 (two groups), bf16: 4.0, 3.4 at one, 6.0, 6.0 at two,
    //   27, 42 at twelve; fp32: 21.8, 22.9 at six, 37, 42 at twelve.
    // The rule does not look at H: narrow fp32 rows in large batches lose up to a tenth by it.
    NormRingPlan ring;
    const int sms = sm_count();
    if (sms < 1) return record_cuda(cudaErrorInvalidDevice, "device");
    if (norm_vec(p) &&
        norm_ring_plan(T, H, fe::norm_fwd_stage(H, r32, y != nullptr, p.gate_kind == FE_GATE_FULL), sms, &ring) &&
        T >= (int64_t)(r32 ? 6 : 2) * sms * (512 / ring.tpr)) {
        FE_CUDA_TRY(r32 ? norm_ring<true>(p, ring, s) : norm_ring<false>(p, ring, s));
        return FE_OK;
    }
    FE_CUDA_TRY(H <= 8192 ? norm_launch<1>(p, r32, norm_threads(H, 1), s) : norm_launch<2>(p, r32, norm_threads(H, 2), s));
    return FE_OK;
}

size_t fe_moe_block_norm_workspace(int64_t T, int H)
{
    if (T < 0 || H < 1 || H > fe::kNormMaxH) return 0;
    return norm_workspace(T, H);
}

fe_status fe_moe_block_norm_backward(const void* dr_out, const void* du, const void* r, int r_dtype, const void* y,
                                     const void* w_post, const void* gate, int gate_kind, float scale,
                                     const void* w_pre, float eps, int64_t T, int H, void* dr, void* dy, void* dgate,
                                     float* dw_post, float* dw_pre, void* workspace, size_t workspace_bytes,
                                     fe_stream_t stream)
{
    fe_status st = check_norm_operands(r, r_dtype, y, w_post, gate, gate_kind, w_pre, eps, T, H);
    if (st != FE_OK) return st;
    const int kind = gate_kind & ~FE_GATE_SIGMOID;
    const int rb = r_dtype == FE_DTYPE_F32 ? 4 : 2;
    if ((dgate && kind == FE_GATE_NONE) || (dw_post && !w_post) || (dw_pre && !w_pre)) return FE_ERR_INVALID_ARG;
    if (T > 0 && ((du != nullptr) != (w_pre != nullptr) || (!dr_out && !du) || (dy && !y) ||
                  (!dr && !dy && !dgate && !dw_post && !dw_pre)))
        return FE_ERR_INVALID_ARG;
    if (!aligned(dr_out, rb) || !aligned(du, 2) || !aligned(dr, rb) || !aligned(dy, 2) ||
        !aligned(dgate, kind == FE_GATE_FULL ? 2 : 4) || !aligned(dw_post, 4) || !aligned(dw_pre, 4) ||
        !aligned(workspace, 4))
        return FE_ERR_INVALID_ARG;
    if (T > 0 && !r) return FE_ERR_INVALID_ARG;
    const bool sums = dw_post || dw_pre || (dgate && kind == FE_GATE_CHANNEL);
    const size_t need = sums ? fe_moe_block_norm_workspace(T, H) : 0;
    if (sums && !workspace) return FE_ERR_INVALID_ARG;
    if (workspace_bytes < need) return FE_ERR_CAPACITY;
    const size_t nr = (size_t)T * H * rb, nb = (size_t)T * H * 2, nw = (size_t)H * 2, ng = gate_elems(gate_kind, T, H);
    const void* ins[7] = {dr_out, du, r, y, w_post, gate, w_pre};
    const size_t in_n[7] = {nr, nb, nr, nb, nw, 2 * ng, nw};
    const void* outs[6] = {dr, dy, dgate, dw_post, dw_pre, sums ? workspace : nullptr};
    const size_t out_n[6] = {nr, nb, (kind == FE_GATE_FULL ? 2 : 4) * ng, 4 * (size_t)H, 4 * (size_t)H, need};
    for (int i = 0; i < 6; ++i) {
        for (int j = 0; j < 7; ++j)   // dr may be dr_out itself
            if (overlap(outs[i], out_n[i], ins[j], in_n[j]) && !(i == 0 && j == 0 && dr == dr_out)) return FE_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], out_n[i], outs[j], out_n[j])) return FE_ERR_INVALID_ARG;
    }
    const cudaStream_t s = (cudaStream_t)stream;
    if (T == 0) {   // sums over no rows
        if (dw_post) FE_CUDA_TRY(cudaMemsetAsync(dw_post, 0, 4 * (size_t)H, s));
        if (dw_pre) FE_CUDA_TRY(cudaMemsetAsync(dw_pre, 0, 4 * (size_t)H, s));
        if (dgate && kind == FE_GATE_CHANNEL) FE_CUDA_TRY(cudaMemsetAsync(dgate, 0, 4 * (size_t)H, s));
        return FE_OK;
    }
    const int sms = sm_count();
    if (sms < 1) return record_cuda(cudaErrorInvalidDevice, "device");
    fe::NormBwdParams q{};
    q.f = norm_params(r, y, w_post, gate, gate_kind, scale, w_pre, eps, T, H);
    q.dr_out = dr_out;
    q.du = static_cast<const uint16_t*>(du);
    q.dr = dr;
    q.dy = static_cast<uint16_t*>(dy);
    q.dgate = kind == FE_GATE_CHANNEL ? nullptr : dgate;
    q.part = sums ? static_cast<float*>(workspace) : nullptr;
    const bool vec = norm_vec(q.f) && aligned(dr_out, 16) && aligned(du, 16) && aligned(dr, 16) && aligned(dy, 16) &&
                     (kind != FE_GATE_FULL || aligned(dgate, 16));
    const bool r32 = r_dtype == FE_DTYPE_F32;
    int partials = 0;
    FE_CUDA_TRY(r32 ? norm_bwd<true>(q, vec, sms, &partials, s) : norm_bwd<false>(q, vec, sms, &partials, s));
    if (sums)
        FE_CUDA_TRY(launch(fe::column_sum_kernel, dim3((H + 31) / 32, 3), dim3(1024), 0, s,
                           static_cast<const float*>(workspace), partials, H, 3, dw_post, dw_pre,
                           kind == FE_GATE_CHANNEL ? static_cast<float*>(dgate) : static_cast<float*>(nullptr)));
    return FE_OK;
}

size_t fe_moe_balance_workspace(int64_t T, int E)
{
    if (T < 0 || E < 1 || E > fe::kBalMaxE) return 0;
    return balance_workspace(T, E);
}

fe_status fe_moe_balance_loss(const float* logits, const int32_t* idx, const uint8_t* mask, int64_t T, int E, int top_k,
                              float balance_coef, float z_coef, float* loss, int32_t* counts, int32_t* n_tokens,
                              void* workspace, size_t workspace_bytes, fe_stream_t stream)
{
    const fe_status st = check_balance(logits, T, E, top_k);
    if (st != FE_OK) return st;
    if ((T > 0 && !idx) || !loss || !counts || !n_tokens || !aligned(idx, 4) || !aligned(loss, 4) ||
        !aligned(counts, 4) || !aligned(n_tokens, 4) || !aligned(workspace, 4))
        return FE_ERR_INVALID_ARG;
    const size_t need = fe_moe_balance_workspace(T, E);
    if (need > 0 && !workspace) return FE_ERR_INVALID_ARG;
    if (workspace_bytes < need) return FE_ERR_CAPACITY;
    const void* ins[3] = {logits, idx, mask};
    const size_t in_n[3] = {4 * (size_t)T * E, 4 * (size_t)T * top_k, (size_t)T};
    const void* outs[4] = {loss, counts, n_tokens, workspace};
    const size_t out_n[4] = {12, 4 * (size_t)E, 4, need};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 3; ++j)
            if (overlap(outs[i], out_n[i], ins[j], in_n[j])) return FE_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], out_n[i], outs[j], out_n[j])) return FE_ERR_INVALID_ARG;
    }
    fe::BalanceParams p{};
    p.logits = logits;
    p.idx = idx;
    p.mask = mask;
    p.T = T;
    p.E = E;
    p.k = top_k;
    p.a = balance_coef;
    p.b = z_coef;
    p.loss = loss;
    p.counts = counts;
    p.n_tokens = n_tokens;
    const int ctas = balance_ctas(T, E);
    const bool vec = E % 4 == 0 && aligned(logits, 16);
    const cudaStream_t s = (cudaStream_t)stream;
    if (balance_fused(T, E)) {
        int n = 1;   // CTAs of the cluster: a group per warp, to eight
        while (n < fe::kBalCluster && n < ctas) n *= 2;
        p.G = 0;
        if (vec && T > balance_small(E)) FE_CUDA_TRY(balance_ring_dispatch(p, s));
        else FE_CUDA_TRY(balance_dispatch(p, false, n, vec, s));
        return FE_OK;
    }
    p.G = ctas;
    p.part = static_cast<float*>(workspace);
    p.ipart = reinterpret_cast<int32_t*>(p.part + (size_t)p.G * (E + 1));
    const int sms = sm_count();
    if (sms < 1) return record_cuda(cudaErrorInvalidDevice, "device");
    if (vec) {
        p.G = balance_ring_ctas(T, E, sms);
        p.ipart = reinterpret_cast<int32_t*>(p.part + (size_t)p.G * (E + 1));
        FE_CUDA_TRY(balance_ring_dispatch(p, s));
    } else {
        FE_CUDA_TRY(balance_dispatch(p, false, p.G, vec, s));
    }
    FE_CUDA_TRY(launch(fe::balance_final_kernel, dim3(fe::kBalCluster), dim3(1024), 0, s, p));
    return FE_OK;
}

fe_status fe_moe_balance_loss_backward(const float* logits, const int32_t* counts, const int32_t* n_tokens,
                                       const uint8_t* mask, const float* dloss, int64_t T, int E, int top_k,
                                       float balance_coef, float z_coef, void* dlogits, int dlogits_dtype,
                                       fe_stream_t stream)
{
    const fe_status st = check_balance(logits, T, E, top_k);
    if (st != FE_OK) return st;
    if (dlogits_dtype != FE_DTYPE_F32 && dlogits_dtype != FE_DTYPE_BF16) return FE_ERR_INVALID_ARG;
    if (T == 0) return FE_OK;
    const size_t eb = dtype_bytes(dlogits_dtype);
    if (!counts || !n_tokens || !dlogits || !aligned(counts, 4) || !aligned(n_tokens, 4) || !aligned(dloss, 4) ||
        !aligned(dlogits, eb))
        return FE_ERR_INVALID_ARG;
    const size_t nd = eb * (size_t)T * E, nl = 4 * (size_t)T * E;
    // dlogits may be the logits themselves (fp32): a row is read before it is written
    if ((overlap(dlogits, nd, logits, nl) && (dlogits != (const void*)logits || eb != 4)) ||
        overlap(dlogits, nd, counts, 4 * (size_t)E) || overlap(dlogits, nd, n_tokens, 4) ||
        overlap(dlogits, nd, mask, (size_t)T) || overlap(dlogits, nd, dloss, 4))
        return FE_ERR_INVALID_ARG;
    fe::BalanceParams p{};
    p.logits = logits;
    p.mask = mask;
    p.T = T;
    p.E = E;
    p.k = top_k;
    p.a = balance_coef;
    p.b = z_coef;
    p.counts = const_cast<int32_t*>(counts);
    p.n_tokens = const_cast<int32_t*>(n_tokens);
    p.dloss = dloss;
    p.dlogits = dlogits;
    p.dl_bf16 = dlogits_dtype == FE_DTYPE_BF16;
    const int sms = sm_count();
    if (sms < 1) return record_cuda(cudaErrorInvalidDevice, "device");
    const int rows = fe::kBalWarps * (32 / balance_lanes(E));
    const int grid = (int)std::min<int64_t>((T + rows - 1) / rows, 8 * (int64_t)sms);
    FE_CUDA_TRY(balance_dispatch(p, true, grid, E % 4 == 0 && aligned(logits, 16) && aligned(dlogits, 4 * eb),
                                 (cudaStream_t)stream));
    return FE_OK;
}

fe_status fe_moe_linear(const void* x, int64_t ldx, const void* w, const void* bias, const void* residual, int64_t ldr,
                        int64_t M, int N, int K, int act, void* y, int64_t ldy, void* z, fe_stream_t stream)
{
    const fe_status st = fe_host::check_linear(x, ldx, w, bias, residual, ldr, M, N, K, act, y, ldy, z);
    if (st != FE_OK) return st;
    if (M == 0) return FE_OK;
    const cudaStream_t s = (cudaStream_t)stream;
    const int cols = out_cols(act, N);
    if (M <= fe::kSkinnyMaxM) {
        fe::LinRowsParams p{};
        p.x = static_cast<const uint16_t*>(x);
        p.ldx = ldx;
        p.w = static_cast<const uint16_t*>(w);
        p.bias = static_cast<const uint16_t*>(bias);
        p.res = static_cast<const uint16_t*>(residual);
        p.ldr = ldr;
        p.y = static_cast<uint16_t*>(y);
        p.ldy = ldy;
        p.z = static_cast<uint16_t*>(z);
        p.M = (int)M;
        p.N = N;
        p.K = K;
        p.act = act;
        p.cols = cols;
        FE_CUDA_TRY(act == FE_ACT_SWIGLU ? rows_launch<true>(p, s) : rows_launch<false>(p, s));
        return FE_OK;
    }
    const Product f{{x, M, K, ldx}, {w, N, K, K}, false, false, (int)M, N, K};
    fe::LinParams P{};
    fe::LinProblem& p = P.p[0];
    p.act = act;
    p.cols = cols;
    p.bias = static_cast<const uint16_t*>(bias);
    p.res = static_cast<const uint16_t*>(residual);
    p.ldr = ldr;
    p.out = static_cast<uint16_t*>(y);
    p.ldo = ldy;
    p.z = static_cast<uint16_t*>(z);
    int BN = 0, ways = 0;
    FE_CUDA_TRY(split_ways(p, f, &ways, &BN));
    if (ways > 0) FE_CUDA_TRY(act == FE_ACT_SWIGLU ? split_run<true>(p, f, BN, ways, s) : split_run<false>(p, f, BN, ways, s));
    else FE_CUDA_TRY(lin_run(P, &f, 1, s));
    return FE_OK;
}

size_t fe_moe_linear_workspace(int64_t M, int N, int K, int act)
{
    return fe_moe_linear_backward_workspace(M, N, K, act, 0, 1, 1, 1);
}

size_t fe_moe_linear_backward_workspace(int64_t M, int N, int K, int act, int dy_rows16, int dx, int dw, int db)
{
    if (check_linear_shape(M, N, K, act) != FE_OK) return 0;
    return dz_bytes(M, N, dz_written(act, dy_rows16, dx, dw)) + db_bytes(M, N, db);
}

fe_status fe_moe_linear_backward(const void* dy, int64_t lddy, const void* x, int64_t ldx, const void* w, const void* z,
                                 int64_t M, int N, int K, int act, void* dx, int64_t lddx, void* dw, float* db,
                                 void* workspace, size_t workspace_bytes, fe_stream_t stream)
{
    const fe_status st = check_linear_shape(M, N, K, act);
    if (st != FE_OK) return st;
    const int cols = out_cols(act, N);
    if (M > 0 && !dx && !dw && !db) return FE_ERR_INVALID_ARG;   // dx of no rows may have no address
    const size_t nx = span(M, ldx, K), ndx = span(M, lddx, K), nw = 2 * (size_t)N * K, nz = 2 * (size_t)M * N;
    const size_t ndy = span(M, lddy, cols);
    const bool rows16 = lddy % 8 == 0 && aligned(dy, 16), dz_buf = dz_written(act, rows16, dx, dw);
    const size_t need = M > 0 ? dz_bytes(M, N, dz_buf) + db_bytes(M, N, db) : 0;
    if (M > 0) {
        if (!dy || lddy < cols || (act != FE_ACT_NONE && !z) || (dx && (!w || lddx < K)) || (dw && (!x || ldx < K)) ||
            (need > 0 && (!workspace || !aligned(workspace, 16))))
            return FE_ERR_INVALID_ARG;
        if (dw && ldx % 8 != 0) return FE_ERR_UNSUPPORTED;
        if (!aligned(dy, 2) || !aligned(z, 2) || (dw && !aligned(x, 16)) || (dx && !aligned(w, 16))) return FE_ERR_INVALID_ARG;
        if (workspace_bytes < need) return FE_ERR_CAPACITY;
    }
    if (!aligned(dx, 2) || !aligned(dw, 2) || !aligned(db, 4)) return FE_ERR_INVALID_ARG;
    const void* ins[4] = {dy, dw ? x : nullptr, dx ? w : nullptr, act != FE_ACT_NONE ? z : nullptr};
    const size_t in_n[4] = {ndy, nx, nw, nz};
    const void* outs[4] = {dx, dw, db, need > 0 ? workspace : nullptr};
    const size_t out_n[4] = {ndx, nw, 4 * (size_t)N, need};
    const size_t ld[2] = {2 * (size_t)lddy, 2 * (size_t)ldx}, width[2] = {2 * (size_t)cols, 2 * (size_t)K};
    for (int i = 0; i < 4; ++i) {
        for (int j = 0; j < 4; ++j)   // dx may lie beside dy or x
            if (i == 0 && j < 2 ? overlap_rows(dx, ndx, 2 * (size_t)lddx, 2 * (size_t)K, ins[j], in_n[j], ld[j], width[j])
                                : overlap(outs[i], out_n[i], ins[j], in_n[j]))
                return FE_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i], out_n[i], outs[j], out_n[j])) return FE_ERR_INVALID_ARG;
    }
    const cudaStream_t s = (cudaStream_t)stream;
    if (M == 0) {   // sums over no rows
        if (dw) FE_CUDA_TRY(cudaMemsetAsync(dw, 0, nw, s));
        if (db) FE_CUDA_TRY(cudaMemsetAsync(db, 0, 4 * (size_t)N, s));
        return FE_OK;
    }
    const bool direct = act == FE_ACT_NONE && rows16;   // dZ is dY itself
    const int64_t lddz = direct ? lddy : ((int64_t)N + 7) / 8 * 8;
    uint16_t* dzbuf = static_cast<uint16_t*>(workspace);
    const void* dz = direct ? dy : dzbuf;
    float* part = reinterpret_cast<float*>(static_cast<char*>(workspace) + dz_bytes(M, N, dz_buf));
    int partials = 0;
    if (!direct || db) {
        fe::LinDzParams p{};
        p.dy = static_cast<const uint16_t*>(dy);
        p.lddy = lddy;
        p.z = static_cast<const uint16_t*>(z);
        p.dz = dz_buf ? dzbuf : nullptr;
        p.lddz = lddz;
        p.part = db ? part : nullptr;
        p.M = M;
        p.N = N;
        p.cols = cols;
        p.rows_per_cta = dz_rows(M);
        const int used = (int)((M + p.rows_per_cta - 1) / p.rows_per_cta);
        const bool vec = cols % 8 == 0 && lddy % 8 == 0 && aligned(dy, 16) && (act == FE_ACT_NONE || aligned(z, 16));
        const int per = 32 * (vec ? 8 : 1);
        const dim3 grid((cols + per - 1) / per, used);
        FE_CUDA_TRY(vec ? dz_launch<8>(act, grid, p, s) : dz_launch<1>(act, grid, p, s));
        partials = used;
    }
    if (dx || dw) {
        // dW [N][K] = dZ^T X (longest tiles first), dX [M][K] = dZ W: one launch of whole tiles.  Neither
        // contraction is split: where there are fewer tiles than CTA pairs, a pair walks a tile's rows alone (dW of
        // 16384 rows, N = K = 64: one tile, 48 us; N = 128, K = 2048: 50 us).
        fe::LinParams P{};
        Product prod[2];
        int n = 0;
        if (dw) {
            prod[n] = {{dz, M, N, lddz}, {x, M, K, ldx}, true, true, N, K, (int)M};
            P.p[n].out = static_cast<uint16_t*>(dw);
            P.p[n].ldo = P.p[n].cols = K;
            ++n;
        }
        if (dx) {
            prod[n] = {{dz, M, N, lddz}, {w, N, K, K}, false, true, (int)M, K, N};
            P.p[n].out = static_cast<uint16_t*>(dx);
            P.p[n].ldo = lddx;
            P.p[n].cols = K;
            ++n;
        }
        FE_CUDA_TRY(lin_run(P, prod, n, s));
    }
    if (db)   // last: the products need not wait for it
        FE_CUDA_TRY(launch(fe::column_sum_kernel, dim3((N + 31) / 32, 1), dim3(1024), 0, s,
                           static_cast<const float*>(part), partials, N, 1, db, static_cast<float*>(nullptr),
                           static_cast<float*>(nullptr)));
    return FE_OK;
}

fe_status fe_moe_get_op_status(uint32_t* bits)
{
    uint32_t v = 0;
    const uint32_t zero = 0;
    FE_CUDA_TRY(cudaDeviceSynchronize());
    FE_CUDA_TRY(cudaMemcpyFromSymbol(&v, fe::g_op_status, sizeof(v)));
    if (v) FE_CUDA_TRY(cudaMemcpyToSymbol(fe::g_op_status, &zero, sizeof(v)));
    if (bits) *bits = v;
    return v ? FE_ERR_DEVICE_STATUS : FE_OK;
}

}  // extern "C"
