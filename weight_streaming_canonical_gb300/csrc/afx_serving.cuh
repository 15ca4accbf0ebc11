// Helpers shared by the serving kernels: page tables and cache writes
// (afx_kv.cu), attention (afx_attention.cu) and sampling (afx_sample.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>
#include <type_traits>

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

// The same, and on the current device, where the kernel is going to run.
inline bool device_ptr_here(const void* p, uintptr_t align) {
    if (!p || (reinterpret_cast<uintptr_t>(p) & (align - 1))) return false;
    cudaPointerAttributes at{};
    int dev = -1;
    if (cudaPointerGetAttributes(&at, p) != cudaSuccess || cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return false;
    }
    return at.type == cudaMemoryTypeManaged || (at.type == cudaMemoryTypeDevice && at.device == dev);
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

// Four elements from i on, of a row's up to end (past it: none), as they lie in
// memory, so that they can be under way while others are worked on.  wide: the
// row is aligned for a load of all four.
template <typename T>
struct RawFour {
    uint32_t w[sizeof(T)];  // 4 sizeof(T) bytes
    __device__ __forceinline__ void load(const T* row, bool wide, uint32_t i, uint32_t end, float none) {
        if (wide && i + 4 <= end) {
            if constexpr (sizeof(T) == 4) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + i));
                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
            } else {
                const uint2 v = __ldg(reinterpret_cast<const uint2*>(row + i));
                w[0] = v.x, w[1] = v.y;
            }
        } else if constexpr (sizeof(T) == 4) {
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c) w[c] = i + c < end ? __ldg(reinterpret_cast<const uint32_t*>(row + i + c)) : __float_as_uint(none);
        } else {
            const uint32_t other = std::is_same<T, __half>::value ? __half_as_ushort(__float2half_rn(none)) : __float_as_uint(none) >> 16;
            uint32_t h[4];
#pragma unroll
            for (uint32_t c = 0; c < 4; ++c) h[c] = i + c < end ? __ldg(reinterpret_cast<const uint16_t*>(row + i + c)) : other;
            w[0] = h[0] | h[1] << 16, w[1] = h[2] | h[3] << 16;
        }
    }
    __device__ __forceinline__ float get(uint32_t c) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[c]);
        const uint32_t h = c % 2 ? w[c / 2] >> 16 : w[c / 2] & 0xFFFFu;
        if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(static_cast<unsigned short>(h)));
        return __uint_as_float(h << 16);
    }
};

__host__ __device__ inline uint32_t ceil_div(uint32_t a, uint32_t b) { return a / b + (a % b != 0); }

}  // namespace serve
}  // namespace afx
