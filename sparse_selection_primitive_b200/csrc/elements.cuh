// Element types of the routing, expert-row and cache kernels: fp32, bf16 and
// fp16 values widened exactly to fp32 and rounded to nearest even on the way out.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "../../include/lapsum.h"

namespace lapsum {

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float widen(__half x) { return __half2float(x); }
template <class T>
__device__ __forceinline__ T narrow(float x);
template <>
__device__ __forceinline__ float narrow<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float x) {
    return __float2bfloat16_rn(x);
}
template <>
__device__ __forceinline__ __half narrow<__half>(float x) { return __float2half_rn(x); }

// N consecutive elements moved with one load or store (N * sizeof(T) is 2, 4, 8
// or 16 bytes and the address a multiple of it).
template <class T, int N>
struct alignas(sizeof(T) * N) Pack {
    T v[N];
};

inline int dtype_size(int dtype) { return dtype == LAPSUM_DTYPE_F32 ? 4 : 2; }
inline bool known_dtype(int dtype) {
    return dtype == LAPSUM_DTYPE_F32 || dtype == LAPSUM_DTYPE_BF16 || dtype == LAPSUM_DTYPE_F16;
}
inline bool aligned_to(const void* p, size_t bytes) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0;
}

// Calls f with a null pointer of the element type `dtype` names.
template <class F>
inline cudaError_t with_dtype(int dtype, F f) {
    switch (dtype) {
        case LAPSUM_DTYPE_BF16: return f((const __nv_bfloat16*)nullptr);
        case LAPSUM_DTYPE_F16: return f((const __half*)nullptr);
        default: return f((const float*)nullptr);
    }
}

}  // namespace lapsum
