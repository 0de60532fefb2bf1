// Host helpers shared by the translation units of the library.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/fe_moe.h"

namespace fe_host {

// Whether [a, a + na) and [b, b + nb) share a byte; null ranges share none.
inline bool overlap(const void* a, size_t na, const void* b, size_t nb)
{
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

// The same for the first ca (cb) of every la (lb) bytes over ranges of na and nb bytes: rows of the same stride lie
// beside each other where their columns do.
inline bool overlap_rows(const void* a, size_t na, size_t la, size_t ca, const void* b, size_t nb, size_t lb, size_t cb)
{
    if (!overlap(a, na, b, nb)) return false;
    if (la != lb || ca > la || cb > lb || la == 0) return true;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    const size_t d = y >= x ? (y - x) % la : (la - (x - y) % la) % la;   // from a row's start to the other's next one
    return d < ca || d + cb > la;
}

// Keeps the text of a CUDA failure for fe_moe_last_error and maps it to a status.
fe_status record_cuda(cudaError_t e, const char* where);

// fe_moe_block_norm and fe_moe_linear with their arguments checked only (nothing is enqueued).
fe_status check_block_norm(const void* r, int r_dtype, const void* y, const void* w_post, const void* gate,
                           int gate_kind, const void* w_pre, float eps, int64_t T, int H, const void* r_out,
                           const void* u);
fe_status check_linear(const void* x, int64_t ldx, const void* w, const void* bias, const void* residual, int64_t ldr,
                       int64_t M, int N, int K, int act, const void* y, int64_t ldy, const void* z);

}  // namespace fe_host
