// Element types of the inner-step calls and their conversions to fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "dl_common.cuh"

namespace dl {

inline size_t type_size(int32_t type) { return type == DL_F32 ? 4 : type == DL_E4M3 ? 1 : 2; }

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
    return __float2bfloat16_rn(v);
}
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// A run of N elements as one load or store (N * sizeof(T) bytes, aligned so).
template <typename T, int N>
struct __align__(sizeof(T) * N) Pack {
    T v[N];
};

}  // namespace dl
