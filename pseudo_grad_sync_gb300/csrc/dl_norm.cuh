// Layer norm: what the forward and the backward kernels share.
//
// A row is held by TPR consecutive threads (a part of a warp, a warp, or up
// to the whole block), each with VPT packs of N neighbouring elements: pack k
// of thread t starts at column (k * TPR + t) * N, so that a warp's loads are
// contiguous. A block of 256 threads (512 for the widest rows) works on
// several rows at once when TPR is smaller.
//
// Rows stream in: each thread keeps the packs of the next AHEAD rows of its
// own in flight with asynchronous copies into a ring in shared memory that no
// other thread reads, so no barrier belongs to the loads.
#pragma once

#include "dl_types.cuh"

namespace dl {

template <typename T, int N>
__device__ __forceinline__ void unpack(const Pack<T, N>& p, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = to_f32(p.v[i]);
}

// Stores `count` leading elements of a pack; `vec`: the address is a multiple of the pack's size.
template <typename T, int N>
__device__ __forceinline__ void store_pack(T* dst, const float (&v)[N], int count, bool vec) {
    Pack<T, N> p;
#pragma unroll
    for (int i = 0; i < N; ++i) p.v[i] = from_f32<T>(v[i]);
    if (vec && count >= N)
        *reinterpret_cast<Pack<T, N>*>(dst) = p;
    else
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (i < count) dst[i] = p.v[i];
}

__device__ __forceinline__ float load_param(const void* p, int32_t type, int64_t i) {
    return type == DL_F32 ? __ldg(static_cast<const float*>(p) + i)
                          : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p) + i));
}

// Sum of one or two values over the TPR threads of a row. Rows of more than a
// warp pass through shared memory: red holds two sets of partial sums used in
// turn, so that one barrier per sum is enough (the set written now was read
// before the barrier of the sum before this one).
template <int TPR, int BLOCK>
struct RowSum {
    static constexpr int kW = TPR / 32;
    float2* red;
    int set = 0;
    static constexpr size_t kBytes = TPR > 32 ? 2 * (BLOCK / 32) * sizeof(float2) : 0;
    __device__ __forceinline__ float2 operator()(float2 v) {
        constexpr int L = TPR < 32 ? TPR : 32;
#pragma unroll
        for (int sh = L / 2; sh; sh >>= 1) {
            v.x += __shfl_xor_sync(kFull, v.x, sh);
            v.y += __shfl_xor_sync(kFull, v.y, sh);
        }
        if constexpr (TPR > 32) {
            float2* r = red + set * (BLOCK / 32);
            set ^= 1;
            if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v;
            __syncthreads();
            const float2* mine = r + (threadIdx.x / TPR) * kW;
            v = mine[0];
#pragma unroll
            for (int w = 1; w < kW; ++w) v.x += mine[w].x, v.y += mine[w].y;
        }
        return v;
    }
    __device__ __forceinline__ float operator()(float x) {
        constexpr int L = TPR < 32 ? TPR : 32;
#pragma unroll
        for (int sh = L / 2; sh; sh >>= 1) x += __shfl_xor_sync(kFull, x, sh);
        if constexpr (TPR > 32) {
            float* r = reinterpret_cast<float*>(red + set * (BLOCK / 32));
            set ^= 1;
            if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = x;
            __syncthreads();
            const float* mine = r + (threadIdx.x / TPR) * kW;
            x = mine[0];
#pragma unroll
            for (int w = 1; w < kW; ++w) x += mine[w];
        }
        return x;
    }
};

}  // namespace dl
