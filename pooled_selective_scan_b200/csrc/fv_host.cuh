// fv_host.cuh -- host helpers shared by the library's entry points.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

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

// Kernels that take more than 48 KB of dynamic shared memory need an opt-in per device.
template <typename Kern>
fv_status opt_in_smem(Kern kernel, size_t bytes, const char* where) {
    if (bytes <= 48 * 1024) return FV_OK;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess) return FV_OK;
    note_cuda_error(e, where);
    return FV_ERR_CUDA;
}

}  // namespace fv
