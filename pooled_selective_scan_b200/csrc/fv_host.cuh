// fv_host.cuh -- host helpers shared by the library's entry points.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <atomic>

#include "fastvim_ssm.h"

namespace fv {

// Keeps the message that fastvim_last_error() returns (defined beside it).
__attribute__((visibility("hidden"))) void note_cuda_error(cudaError_t e, const char* where);

inline bool ptr_aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline size_t round_up256(size_t v) { return (v + 255) & ~(size_t)255; }
inline bool ranges_overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return a && b && na && nb && x < y + nb && y < x + na;
}

// The status of the launch just made.
inline fv_status launch_status(const char* where) {
    const cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess) return FV_OK;
    note_cuda_error(e, where);
    return FV_ERR_CUDA;
}

// Kernels that take more than 48 KB of dynamic shared memory need an opt-in, once per kernel and device
// (a driver call of about a microsecond, so it is remembered; such a kernel's bytes are the same in every call).
template <auto KERNEL>
fv_status opt_in_smem(size_t bytes, const char* where) {
    if (bytes <= 48 * 1024) return FV_OK;
    static std::atomic<unsigned long long> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
    if (e == cudaSuccess && (done.load(std::memory_order_relaxed) & bit)) return FV_OK;
    if (e == cudaSuccess) e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) {
        done.fetch_or(bit, std::memory_order_relaxed);
        return FV_OK;
    }
    note_cuda_error(e, where);
    return FV_ERR_CUDA;
}

}  // namespace fv
