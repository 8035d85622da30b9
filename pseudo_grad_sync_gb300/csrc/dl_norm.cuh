// Layer norm: what the forward and the backward kernels share.
//
// A row is held by TPR consecutive threads (a part of a warp, a warp, or up
// to the whole block), each with VPT packs of N neighbouring elements: pack k
// of thread t starts at column (k * TPR + t) * N, so that a warp's loads are
// contiguous. A block of 256 threads (512 for the widest rows) works on
// several rows at once when TPR is smaller.
//
// A block takes a run of consecutive rows in rounds of one row per group of
// TPR threads. Long runs of 16-byte aligned rows come in by bulk copies into a
// ring of stages in shared memory, issued by one warp; the barrier of the row
// sums also tells that a stage has been read. Short runs and other alignments
// are loaded straight into registers.
#pragma once

#include <float.h>

#include "dl_phase.h"
#include "dl_types.cuh"

namespace dl {

// two 16-bit elements, the first in the low half
__device__ __forceinline__ float2 unpack2(uint32_t w, __nv_bfloat16) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
__device__ __forceinline__ float2 unpack2(uint32_t w, __half) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}

// The packs of a thread as pairs of elements: neighbours of one pack, or for
// packs of one element those of two packs in a row.
template <typename T, int N>
__device__ __forceinline__ float2 pair_of(const Pack<T, N>* q, int p) {
    if constexpr (N == 1) {
        return make_float2(to_f32(q[2 * p].v[0]), to_f32(q[2 * p + 1].v[0]));
    } else {
        constexpr int H = N / 2;
        if constexpr (sizeof(T) == 2) {
            const uint32_t w = reinterpret_cast<const uint32_t*>(q[p / H].v)[p % H];
            return unpack2(w, T());
        } else {
            return make_float2(q[p / H].v[2 * (p % H)], q[p / H].v[2 * (p % H) + 1]);
        }
    }
}

__device__ __forceinline__ uint32_t pack2(float2 v, __nv_bfloat16) {
    const __nv_bfloat162 p = __float22bfloat162_rn(v);
    return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t pack2(float2 v, __half) {
    const __half2 p = __float22half2_rn(v);
    return *reinterpret_cast<const uint32_t*>(&p);
}

template <typename T, int N>
__device__ __forceinline__ Pack<T, N> pack_of(const float2* v) {
    Pack<T, N> p;
    if constexpr (N == 1) {
        p.v[0] = from_f32<T>(v[0].x);
    } else if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) reinterpret_cast<uint32_t*>(p.v)[i] = pack2(v[i], T());
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) p.v[2 * i] = v[i].x, p.v[2 * i + 1] = v[i].y;
    }
    return p;
}

// Stores a thread's pairs: whole packs at once where the rows are aligned
// (`vec`), the elements of a last, partial pack one by one.
template <typename T, int N, int TPR, int VPT, bool FULL>
__device__ __forceinline__ void store_row(T* row, const float2 (&v)[VPT * N / 2], int t, int width, bool vec) {
#pragma unroll
    for (int k = 0; k < VPT; ++k) {
        const int c = (k * TPR + t) * N;
        if (FULL || (N > 1 && vec && c + N <= width)) {
            *(reinterpret_cast<Pack<T, N>*>(row) + k * TPR + t) = pack_of<T, N>(v + k * N / 2);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int e = k * N + i;
                if (c + i < width) row[c + i] = from_f32<T>(e % 2 ? v[e / 2].y : v[e / 2].x);
            }
        }
    }
}

__device__ __forceinline__ float load_param(const void* p, int32_t type, int64_t i) {
    return type == DL_F32 ? __ldg(static_cast<const float*>(p) + i)
                          : __bfloat162float(__ldg(static_cast<const __nv_bfloat16*>(p) + i));
}

// Sums over the TPR threads of a row, in two halves, so that other rows' work
// can lie between them: give() leaves the warp's sums, take() joins the warps
// of the row. Rows of more than a warp need a block barrier between the two;
// there are two sets of slots, used in turn. With CLUSTER blocks per row every
// warp leaves its sums in each block's slots, and the barrier is the cluster's.
template <int TPR, int BLOCK, int CLUSTER = 1>
struct RowSum {
    static constexpr int kW = TPR / 32 * CLUSTER;            // warps of a row
    static constexpr int kSlots = BLOCK / 32 * CLUSTER;      // of a set
    static constexpr bool kShared = TPR > 32;
    static constexpr size_t kBytes = kShared ? 2 * kSlots * sizeof(float2) : 0;
    static_assert(CLUSTER == 1 || TPR == BLOCK, "a cluster shares one row");
    float2* red;
    float2 own;
    __device__ __forceinline__ static void barrier() {
        if constexpr (CLUSTER > 1)
            asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
        else
            __syncthreads();
    }
    __device__ __forceinline__ void give(float2 v, int set) {
        if constexpr (kShared) {
            // after the first exchange the lower half of the warp has only x
            // left to sum and the upper half only y
            const bool up = threadIdx.x & 16;
            float k = (up ? v.y : v.x) + __shfl_xor_sync(kFull, up ? v.x : v.y, 16);
#pragma unroll
            for (int sh = 8; sh; sh >>= 1) k += __shfl_xor_sync(kFull, k, sh);
            if ((threadIdx.x & 15) == 0) {
                if constexpr (CLUSTER == 1) {
                    reinterpret_cast<float*>(red + set * kSlots + (threadIdx.x >> 5))[up] = k;
                } else {
                    const int slot = static_cast<int>(blockIdx.x % CLUSTER) * (BLOCK / 32) + (threadIdx.x >> 5);
                    const uint32_t to = smem_addr(reinterpret_cast<float*>(red + set * kSlots + slot) + up);
#pragma unroll
                    for (int c = 0; c < CLUSTER; ++c)
                        asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
                                     "st.shared::cluster.f32 [a], %2;\n\t}" ::"r"(to), "r"(c), "f"(k)
                                     : "memory");
                }
            }
        } else {
#pragma unroll
            for (int sh = TPR / 2; sh; sh >>= 1)
                v = add2(v, make_float2(__shfl_xor_sync(kFull, v.x, sh), __shfl_xor_sync(kFull, v.y, sh)));
            own = v;
        }
    }
    // single sums
    __device__ __forceinline__ void give(float x, int set) {
        constexpr int L = TPR < 32 ? TPR : 32;
#pragma unroll
        for (int sh = L / 2; sh; sh >>= 1) x += __shfl_xor_sync(kFull, x, sh);
        if constexpr (kShared) {
            if ((threadIdx.x & 31) == 0)
                reinterpret_cast<float*>(red + set * kSlots)[threadIdx.x >> 5] = x;
        } else {
            own.x = x;
        }
    }
    __device__ __forceinline__ float take1(int set) const {
        if constexpr (kShared) {
            const float2* mine = reinterpret_cast<const float2*>(
                reinterpret_cast<const float*>(red + set * kSlots) + (threadIdx.x / TPR) * kW);
            float2 v = mine[0];
#pragma unroll
            for (int w = 1; w < kW / 2; ++w) v = add2(v, mine[w]);
            return v.x + v.y;
        } else {
            return own.x;
        }
    }
    __device__ __forceinline__ float2 take(int set) const {
        if constexpr (kShared) {
            const float4* mine = reinterpret_cast<const float4*>(red + set * kSlots + (threadIdx.x / TPR) * kW);
            float2 v = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kW / 2; ++w) {
                const float4 q = mine[w];
                v = add2(v, add2(make_float2(q.x, q.y), make_float2(q.z, q.w)));
            }
            return v;
        } else {
            return own;
        }
    }
};

// s / n with its rounding corrected by the remainder (inv = 1 / n): a
// constant row's mean is then the constant itself, whatever the width. The
// remainder of an infinite sum is NaN, for which the larger operand is the
// other one: the mean stays infinite.
__device__ __forceinline__ float divided(float s, float n, float inv) {
    const float q = s * inv;
    return fmaf(fmaxf(fmaf(-q, n, s), -FLT_MAX), inv, q);
}

// Sum over the whole block, for rows that a block reads several times.
__device__ __forceinline__ float2 block_sum(float2 v, float2* red) {
    for (int sh = 16; sh; sh >>= 1)
        v = add2(v, make_float2(__shfl_xor_sync(kFull, v.x, sh), __shfl_xor_sync(kFull, v.y, sh)));
    __syncthreads();  // red may still be read from the sum before
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = make_float2(0.f, 0.f);
    for (int w = 0; w < static_cast<int>(blockDim.x / 32); ++w) v = add2(v, red[w]);
    return v;
}

// Rows loaded straight into registers: warp 0 has the next round's rows brought
// to L2 meanwhile, a lane per row (the 16-byte aligned inside of each). It pays
// where a round is few long rows.
template <typename T>
__device__ __forceinline__ void prefetch_rows(int64_t first, int groups, int64_t end, const T* p, int64_t stride,
                                              int width) {
    if (threadIdx.x >= 32) return;
    const int64_t r = first + threadIdx.x;
    if (static_cast<int>(threadIdx.x) >= groups || r >= end) return;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p + r * stride);
    const uintptr_t lo = (at + 15) & ~uintptr_t(15), hi = (at + width * sizeof(T)) & ~uintptr_t(15);
    if (hi > lo)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(lo), "r"(static_cast<uint32_t>(hi - lo))
                     : "memory");
}

constexpr int kRowPolls = 1 << 17;  // of a wait for a round's rows: about a second

// Where a ring reports a wait that ran out (either may be null), and whether to
// take the first one for such.
struct RingReport {
    uint32_t* word;
    uint32_t* second;
    bool lost;
};

// The end of a block with a wait that ran out: sets the status words, and warp
// 0, which issued the copies, waits (bounded too) until those in flight at its
// own failed wait have landed. `record` is what RowRing::record left of it. Out
// of line, and the record in shared memory: carried in registers, or with the
// reports in the loop, rows of 5632 took up to 10% longer backward.
template <int STAGES>
__device__ __noinline__ void ring_drain(uint64_t* full, const uint64_t* record, const RingReport& report) {
    if (report.word) atomicOr(report.word, kDevErrCopyTimeout);
    if (report.second) atomicOr(report.second, kDevErrCopyTimeout);
    if (threadIdx.x >= 32) return;
    __syncwarp();
    const int at = static_cast<int>(*record);
    RingPhase<STAGES> phase;
    phase.stage = at % STAGES;
    phase.parity = at / STAGES % 2;
    for (int i = 0; i < at / (2 * STAGES); ++i)
        mbar_wait_bounded(full + phase.stage_of(i), phase.parity_of(i), kRowPolls);
}

// The ring of a block's rounds: each stage holds ARRAYS arrays' rows of one
// round. Rows that follow each other in memory come in one copy per array,
// others in one copy per row.
template <typename T, int TPR, int EPT, int BLOCK, int ARRAYS, int STAGES>
struct RowRing {
    static constexpr int kGroups = BLOCK / TPR;
    static_assert(kGroups <= 32, "a lane of warp 0 copies a row");
    static constexpr size_t kRow = size_t(TPR) * EPT * sizeof(T);
    static constexpr size_t kStage = kGroups * ARRAYS * kRow;
    static constexpr size_t kBytes = STAGES * kStage;
    unsigned char* base;
    uint64_t* full;  // a barrier per stage, and a word
    const RingReport& report;  // of the kernel's arguments
    int64_t end;               // of the block's rows
    // bytes of a row that a bulk copy takes: a last, partial pack is loaded by its owner
    uint32_t bytes;
    uint32_t pitch;  // between a stage's rows: `bytes` when they come in one copy, else kRow
    RingPhase<STAGES> phase;
    bool ok = true;

    __device__ __forceinline__ void init() {
        if (threadIdx.x == 0) {
            for (int i = 0; i < STAGES; ++i) mbar_init(full + i, 1);
            fence_barrier_init();
        }
        __syncthreads();
    }
    __device__ __forceinline__ unsigned char* row(int st, int group, int which) const {
        return base + st * kStage + which * (kGroups * kRow) + group * pitch;
    }
    // Warp 0: copies the rows of the round from `first` on, a lane per row.
    __device__ __forceinline__ void issue(int st, int64_t first, const T* p0, int64_t s0, const T* p1, int64_t s1) {
        if (threadIdx.x >= 32) return;
        const int64_t left = end - first;
        if (left <= 0 || !ok) return;
        const int n = left < kGroups ? static_cast<int>(left) : kGroups, j = threadIdx.x;
        if (j == 0) {
            fence_proxy_async();
            mbar_arrive_expect_tx(full + st, n * ARRAYS * bytes);
        }
        __syncwarp();
        const uint32_t size = pitch == kRow ? bytes : n * bytes;
        if (j < (pitch == kRow ? n : 1) && bytes) {
            bulk_copy_g2s(row(st, j, 0), p0 + (first + j) * s0, size, full + st);
            if (ARRAYS > 1) bulk_copy_g2s(row(st, j, 1), p1 + (first + j) * s1, size, full + st);
        }
    }
    // the stage of the round being read, and the one of the round before it
    __device__ __forceinline__ int stage() const { return phase.stage; }
    __device__ __forceinline__ int before() const { return phase.before(); }
    __device__ __forceinline__ void advance() { phase.advance(); }
    // Until the current stage holds the round from row `first` on. After a wait
    // that ran out the warp neither waits nor copies any more, and the block's
    // outputs are undefined.
    __device__ __forceinline__ void wait(int64_t first) {
        if (!ok) return;
        ok = __all_sync(kFull, mbar_wait_bounded(full + phase.stage, phase.parity, kRowPolls));
        if (!ok) record(first);
    }
    // The wait for the first round as one that ran out.
    __device__ __forceinline__ void lose(int64_t first) {
        ok = false;
        record(first);
    }
    // Before the block ends or uses the ring's memory for something else.
    __device__ __forceinline__ void drain() {
        if (!ok) ring_drain<STAGES>(full, full + STAGES, report);
    }

private:
    // behind the barriers: what warp 0 has in flight
    __device__ __forceinline__ void record(int64_t first) {
        if (threadIdx.x == 0)
            full[STAGES] = (phase.in_flight((end - first + kGroups - 1) / kGroups) * 2 + phase.parity) * STAGES +
                           phase.stage;
    }
};

}  // namespace dl
