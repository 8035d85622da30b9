// Element types of the inner-step calls and their conversions to fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>
#include <stdlib.h>

#include <atomic>

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

// Asynchronous copies of BYTES (4, 8 or 16) from global to shared memory; the
// bytes past `valid` are not read and become zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, int valid = BYTES) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src),
                     "r"(valid)
                     : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(smem_addr(dst)), "l"(src),
                     "n"(BYTES), "r"(valid)
                     : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// until at most N of this thread's groups are in flight
template <int N>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two products, sums or fused products at once, each rounded.
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ uint64_t bits2(float2 v) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
    return r;
}
__device__ __forceinline__ float2 floats2(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 x, float2 y) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(x)), "l"(bits2(y)));
    return floats2(r);
}
__device__ __forceinline__ float2 add2(float2 x, float2 y) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(x)), "l"(bits2(y)));
    return floats2(r);
}
__device__ __forceinline__ float2 fma2(float2 x, float2 y, float2 z) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(bits2(x)), "l"(bits2(y)), "l"(bits2(z)));
    return floats2(r);
}

// no more blocks than DL_GRID_LIMIT (environment; tests use it to make single
// blocks cover much)
inline int64_t limited(int64_t blocks) {
    if (const char* cap = getenv("DL_GRID_LIMIT")) {
        const long v = strtol(cap, nullptr, 10);
        if (v > 0 && v < blocks) return v;
    }
    return blocks;
}

// Launch geometry of one kernel with its threads and dynamic shared memory:
// the blocks that fit the current device at once, asked for on the first call
// per device and kept; 0 (and no error left behind for a later call) when the
// device refuses. The shared memory is allowed on every call, so a launch
// after a device reset finds it so. One object per kernel: a static local of
// the function that launches it.
class Resident {
public:
    int blocks(const void* kernel, int threads, size_t smem) {
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices) return 0;
        if (smem > 48 * 1024 && cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     static_cast<int>(smem)) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        int b = kept_[dev].load(std::memory_order_acquire);
        if (b == 0) {
            int per_sm = 0;
            if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem) != cudaSuccess) {
                cudaGetLastError();
                return 0;
            }
            b = per_sm * sm_count();
            kept_[dev].store(b, std::memory_order_release);
        }
        return b;
    }
    // a persistent grid: no more blocks than work items
    int grid(const void* kernel, int threads, size_t smem, int64_t work_items) {
        const int64_t g = limited(blocks(kernel, threads, smem));
        return static_cast<int>(work_items < g ? work_items : g);
    }

private:
    static constexpr int kDevices = 64;
    std::atomic<int> kept_[kDevices] = {};
};

// DL_WAIT_POLLS=0 (environment; tests use it): waits for copies run out at once
inline bool waits_run_out() {
    const char* v = getenv("DL_WAIT_POLLS");
    return v && v[0] == '0' && v[1] == 0;
}

// p is a multiple of a (a power of two); null is
inline bool aligned_to(const void* p, size_t a) {
    return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0;
}

}  // namespace dl
