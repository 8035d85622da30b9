// Token log probabilities: what the forward and the backward kernels share.
//
// A row of logits is cut at 16-byte boundaries into packs of N elements; pack 0
// and the last one may lie partly outside the row. Column of element i of
// pack p: p * N + i - skew, skew being the elements between the boundary and
// the row's start.
#pragma once

#include <math.h>

#include <type_traits>

#include "dl_norm.cuh"

namespace dl {

constexpr float kLog2E = 1.44269504f, kLn2 = 0.693147181f;
constexpr float kLeast = -200.f;  // an exponent of 2 that is 0 in fp32, and no infinity

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// the larger, NaN if one is
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// A row's packs. `base` is the boundary at or before its start.
template <typename T>
struct RowPacks {
    static constexpr int N = 16 / sizeof(T);
    const T* base;
    int skew, packs;
    int64_t end;  // skew + width: elements from base to the row's end

    __device__ __forceinline__ RowPacks(const T* row, int64_t width) {
        skew = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
        base = row - skew;
        end = skew + width;
        packs = static_cast<int>((end + N - 1) / N);
    }
    __device__ __forceinline__ bool whole(int p) const {
        return (p > 0 || skew == 0) && (int64_t(p) + 1) * N <= end;
    }
    __device__ __forceinline__ bool inside(int64_t place) const { return place >= skew && place < end; }
    // pack p of `base`, `fill` where it lies outside the row; element by element
    // into whole words, as a pack in registers is words
    __device__ __forceinline__ Pack<T, N> edge(int64_t p, uint32_t fill) const {
        Pack<T, N> r;
        uint32_t* const w = reinterpret_cast<uint32_t*>(r.v);
        if constexpr (sizeof(T) == 2) {
            const uint16_t* from = reinterpret_cast<const uint16_t*>(base);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t at = p * N + 2 * i;
                const uint32_t low = inside(at) ? from[at] : fill, high = inside(at + 1) ? from[at + 1] : fill;
                w[i] = low | high << 16;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                w[i] = inside(p * N + i) ? reinterpret_cast<const uint32_t*>(base)[p * N + i] : fill;
        }
        return r;
    }
};

// the bits of -inf
template <typename T>
constexpr uint32_t kNone = sizeof(T) == 4 ? 0xff800000u : std::is_same<T, __half>::value ? 0xfc00u : 0xff80u;
template <typename T, int N>
__device__ __forceinline__ Pack<T, N> filled(uint32_t fill) {
    Pack<T, N> r;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        reinterpret_cast<uint32_t*>(r.v)[i] = sizeof(T) == 4 ? fill : fill | fill << 16;
    return r;
}

// A cluster's blocks.
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// what block `rank` has at this block's shared address p
__device__ __forceinline__ uint32_t cluster_address(const void* p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_addr(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ float load_cluster(const float* p, int rank) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_address(p, rank)) : "memory");
    return v;
}
__device__ __forceinline__ uint64_t load_cluster(const uint64_t* p, int rank) {
    uint64_t v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(cluster_address(p, rank)) : "memory");
    return v;
}

__device__ __forceinline__ int64_t token_at(const void* tokens, int32_t type, int64_t row) {
    return type == DL_I64 ? static_cast<const int64_t*>(tokens)[row] : static_cast<const int32_t*>(tokens)[row];
}

}  // namespace dl
