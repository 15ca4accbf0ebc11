// Helpers shared by the serving kernels: page tables and cache writes
// (afx_kv.cu), attention (afx_attention.cu) and sampling (afx_sample.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "afx_internal.h"

#define AFX_SERVE_TRY(call, what)                                       \
    do {                                                                \
        const cudaError_t serve_err_ = (call);                          \
        if (serve_err_ != cudaSuccess) return afx_fail(AFX_E_CUDA, what, serve_err_); \
    } while (0)

namespace afx {
namespace serve {

// Kernels index device memory the caller names, so every pointer is checked
// on the host first: device (or managed) memory and the alignment its loads
// need.  Returns false for null, host memory or a misaligned address.
inline bool device_ptr(const void* p, uintptr_t align) {
    if (!p || (reinterpret_cast<uintptr_t>(p) & (align - 1))) return false;
    cudaPointerAttributes at{};
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return at.type == cudaMemoryTypeDevice || at.type == cudaMemoryTypeManaged;
}

inline int current_sms() {
    int dev = -1, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    return sms;
}

// Launches a kernel that may start while the one before it on the stream is
// still running: it has to call wait_for_earlier() before it touches memory
// that earlier work writes or reads.
template <typename... Params, typename... Args>
cudaError_t launch_early(void (*kernel)(Params...), uint32_t grid, uint32_t block, size_t smem, cudaStream_t stream, Args... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Returns once all work before this kernel on the stream is done and visible.
__device__ __forceinline__ void wait_for_earlier() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
// From here on (in every CTA) the next kernel on the stream may start.
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

__device__ __forceinline__ void raise(int32_t* status, int32_t bits) {
    if (status) atomicOr(status, bits);
}

__device__ __forceinline__ uint32_t smem_addr(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__host__ __device__ inline uint32_t ceil_div(uint32_t a, uint32_t b) { return a / b + (a % b != 0); }

}  // namespace serve
}  // namespace afx
