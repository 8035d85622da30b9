// Layer norm backward: the input's gradient and the sums over rows that are
// the weight's and the bias's gradients, in one pass over dy and x.
#include <math.h>
#include <stdint.h>

#include "dl_norm.cuh"

namespace dl {
namespace {

constexpr int kMostBlocks = 456;  // partial sums: 3 blocks on each of 152 SMs
constexpr int kWideParts = 32;    // parts of the rows for the widest rows' sums

template <typename T>
struct BwdArgs {
    const T* dy;
    const T* x;
    T* dx;
    const void* weight;
    const float* mean;
    const float* rstd;
    float* part;  // [blocks][2][width]
    RingReport report;
    int64_t ds, xs, os, rows;
    int64_t run;  // rows of a block
    int width;
    int32_t ptype;
    bool rms, vec_out;
};

constexpr int kStatRows = 512;  // rows whose mean and rstd a block holds at a time

template <typename T, int TPR, int BLOCK, bool BULK, int CLUSTER>
struct BwdGeometry {
    static constexpr int kEPT = 16, kGroups = BLOCK / TPR, kStages = sizeof(T) == 4 ? 3 : 4;
    using Ring = RowRing<T, TPR, kEPT, BLOCK, 2, kStages>;
    static constexpr size_t kSums = kGroups > 1 ? size_t(BLOCK) * kEPT * 2 * sizeof(float) : 0;
    static constexpr size_t kFixed = 128 + kStatRows * sizeof(float2) + RowSum<TPR, BLOCK, CLUSTER>::kBytes;
    static constexpr size_t kBytes = kFixed + (BULK && Ring::kBytes > kSums ? Ring::kBytes : kSums);
};

// A round: the row's terms of its two sums and of the thread's columns' sums,
// the exchange of the row sums (one barrier), then dx from the packs, still
// in registers. FULL: the threads' packs cover the width exactly and dx's rows
// are aligned. CLUSTER blocks share rows too wide for one block's registers,
// 8192 columns each, and exchange the row sums through each other's shared
// memory.
//
// Reads dy and x once: the columns' sums stay in registers over a block's
// whole run (a pass of its own for them took 555 us with the rest), so few
// blocks mean few partial sums: one block of 512 threads per SM (131 us)
// against two of 256 (139 us). Rows come by bulk copies: copies by every
// thread kept the shared-memory pipe at 63% and the call at 180 us. The row
// sums' exchange halves its shuffles by giving each half of the warp one sum.
// 32768 x 4096 bf16: 127 us with the join, 6.3 TB/s (93% of the copy rate);
// fp32 248 us (96%); 8192 x 14336 bf16 195 us (53%: one barrier of the
// cluster per row; clusters of four blocks of 256 threads: 598 us).
template <typename T, int N, int TPR, int BLOCK, bool BULK, bool FULL, int CLUSTER>
__global__ void __launch_bounds__(BLOCK) k_norm_bwd(const __grid_constant__ BwdArgs<T> a) {
    using Geo = BwdGeometry<T, TPR, BLOCK, BULK, CLUSTER>;
    constexpr int EPT = Geo::kEPT, VPT = EPT / N, kGroups = Geo::kGroups, kPairs = EPT / 2;
    extern __shared__ __align__(128) unsigned char smem[];
    using P = Pack<T, N>;
    float2* stats = reinterpret_cast<float2*>(smem + 128);
    RowSum<TPR, BLOCK, CLUSTER> sum{stats + kStatRows};
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    // the block's rows, and with a cluster its part of their columns
    const int64_t part_of = blockIdx.x / CLUSTER, begin = a.run * part_of, end = min(a.rows, begin + a.run);
    const int off = CLUSTER > 1 ? static_cast<int>(blockIdx.x % CLUSTER) * TPR * EPT : 0;
    const int width = CLUSTER > 1 ? max(0, min(a.width - off, TPR * EPT)) : a.width;
    const T* const dy = a.dy + off;
    const T* const x = a.x + off;
    auto column = [&](int k) { return (k * TPR + t) * N; };
    const uint32_t bytes = static_cast<uint32_t>(width * sizeof(T)) & ~15u;
    const bool together = bytes == width * sizeof(T) && a.ds == width && a.xs == width;
    typename Geo::Ring ring{smem + Geo::kFixed, reinterpret_cast<uint64_t*>(smem), a.report, end, bytes,
                            together ? bytes : static_cast<uint32_t>(Geo::Ring::kRow)};
    if constexpr (CLUSTER > 1) sum.barrier();  // the other block runs before its memory is written
    if constexpr (BULK) {
        ring.init();
#pragma unroll
        for (int i = 0; i < Geo::kStages - 1; ++i) ring.issue(i, begin + i * kGroups, dy, a.ds, x, a.xs);
        if (a.report.lost) ring.lose(begin);
    }
    float2 w[kPairs], dw[kPairs], db[kPairs];
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = 2 * p + i, c = column(e / N) + e % N;
            f[i] = c < width ? load_param(a.weight, a.ptype, off + c) : 0.f;
        }
        w[p] = make_float2(f[0], f[1]);
        dw[p] = db[p] = make_float2(0.f, 0.f);
    }
    const float inv = 1.0f / static_cast<float>(a.width);
    int set = 0, at = kStatRows;
    for (int64_t first = begin; first < end; first += kGroups, at += kGroups) {
        const int64_t r = first + group;
        // off 16 bytes, 32768 x 4096 bf16 267 -> 184 us, but 60000 x 501 48 -> 63 without the bound
        if constexpr (!BULK && TPR >= 64) {
            prefetch_rows(first + kGroups, kGroups, end, dy, a.ds, width);
            prefetch_rows(first + kGroups, kGroups, end, x, a.xs, width);
        }
        const bool in = kGroups == 1 || r < end;
        if (at == kStatRows) {  // the next rows' statistics
            __syncthreads();
            for (int i = threadIdx.x; i < kStatRows && first + i < end; i += BLOCK)
                stats[i] = make_float2(a.rms ? 0.f : __ldg(a.mean + first + i), __ldg(a.rstd + first + i));
            __syncthreads();
            at = 0;
        }
        const float2 st = stats[at + group];
        const float mu = in ? st.x : 0.f, rs = in ? st.y : 0.f;
        P dyp[VPT], xp[VPT];
        if constexpr (BULK) ring.wait(first);
        const P* from0 = (BULK ? reinterpret_cast<const P*>(ring.row(ring.stage(), group, 0))
                               : reinterpret_cast<const P*>(dy + r * a.ds)) + t;
        const P* from1 = (BULK ? reinterpret_cast<const P*>(ring.row(ring.stage(), group, 1))
                               : reinterpret_cast<const P*>(x + r * a.xs)) + t;
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = column(k);
            if (in && (FULL || c + N <= width)) {
                dyp[k] = from0[k * TPR], xp[k] = from1[k * TPR];
            } else {  // zeros past the width and the rows
#pragma unroll
                for (int i = 0; i < N; ++i) dyp[k].v[i] = xp[k].v[i] = from_f32<T>(0.f);
                if (N > 1 && in && c < width)  // a last, partial pack
#pragma unroll
                    for (int i = 0; i < N - 1; ++i)
                        if (c + i < width) {
                            dyp[k].v[i] = dy[r * a.ds + c + i];
                            xp[k].v[i] = x[r * a.xs + c + i];
                        }
            }
        }
        float2 s2 = make_float2(0.f, 0.f), q2 = s2;
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
            const float2 g = pair_of<T, N>(dyp, p);
            const float2 h = mul2(add2(pair_of<T, N>(xp, p), both(-mu)), both(rs));
            const float2 wg = mul2(g, w[p]);
            s2 = add2(s2, wg);
            q2 = fma2(wg, h, q2);
            dw[p] = fma2(g, h, dw[p]);
            db[p] = add2(db[p], g);
        }
        sum.give(make_float2(s2.x + s2.y, q2.x + q2.y), set);
        if constexpr (RowSum<TPR, BLOCK, CLUSTER>::kShared || BULK) sum.barrier();
        if constexpr (BULK) {  // every thread has read this round's stage, and the one before it long ago
            ring.issue(ring.before(), first + (Geo::kStages - 1) * kGroups, dy, a.ds, x, a.xs);
            ring.advance();
        }
        const float2 total = sum.take(set);
        set ^= 1;
        if (in) {
            // dx = rs (w dy - s - (x - mu) rs q): x - mu first, as the definition
            // has it, then two fused steps per element. With mu in the constant
            // (x c1 + (c0 - mu c1), an add less) the two large terms of a row on
            // an offset cancel: off by some 2000 u of its terms at mean 1000, spread 1.
            const float s = a.rms ? 0.f : total.x * inv, rq = rs * (total.y * inv);
            const float2 c1 = both(-rs * rq), c0 = both(-rs * s), r2 = both(rs), off_mu = both(-mu);
            float2 out[kPairs];
#pragma unroll
            for (int p = 0; p < kPairs; ++p)
                out[p] = fma2(mul2(pair_of<T, N>(dyp, p), w[p]), r2,
                              fma2(add2(pair_of<T, N>(xp, p), off_mu), c1, c0));
            store_row<T, N, TPR, VPT, FULL>(a.dx + off + r * a.os, out, t, width, a.vec_out);
        }
    }
    if constexpr (BULK) ring.drain();
    // the join's blocks may take the place of those that end from here on
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    // the block's sums over its rows
    float* part = a.part + part_of * 2 * a.width + off;
    if constexpr (kGroups == 1) {
#pragma unroll
        for (int p = 0; p < kPairs; ++p)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int e = 2 * p + i, c = column(e / N) + e % N;
                if (c < width) {
                    part[c] = i ? dw[p].y : dw[p].x;
                    part[a.width + c] = i ? db[p].y : db[p].x;
                }
            }
    } else {
        constexpr int kCols = TPR * EPT;
        __syncthreads();  // the ring's last reads and copies are done
        float* acc = reinterpret_cast<float*>(smem + Geo::kFixed);  // [groups][2][columns]
#pragma unroll
        for (int p = 0; p < kPairs; ++p)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int e = 2 * p + i, c = column(e / N) + e % N;
                acc[(2 * group) * kCols + c] = i ? dw[p].y : dw[p].x;
                acc[(2 * group + 1) * kCols + c] = i ? db[p].y : db[p].x;
            }
        __syncthreads();
        for (int e = threadIdx.x; e < 2 * a.width; e += BLOCK) {
            const int which = e >= a.width, c = e - which * a.width;
            float v = 0.f;
            for (int g = 0; g < kGroups; ++g) v += acc[(2 * g + which) * kCols + c];
            part[e] = v;
        }
    }
}

// Sums of the blocks' partial sums: 32 columns and 8 shares of the blocks per
// block of threads, in a fixed order.
__global__ void __launch_bounds__(kThreads)
    k_norm_join(const float* part, int parts, int width, int32_t ptype, bool accumulate, void* dw,
                void* db) {
    __shared__ float red[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const float* from = part + int64_t(blockIdx.y) * width + c;
    float s = 0.f;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // until the partial sums are all there
    if (c < width) {
        int p = warp;
        for (; p + 3 * kWarps < parts; p += 4 * kWarps) {
            float v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = __ldcg(from + int64_t(p + u * kWarps) * 2 * width);
            s += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; p < parts; p += kWarps) s += __ldcg(from + int64_t(p) * 2 * width);
    }
    red[warp][lane] = s;
    __syncthreads();
    if (warp || c >= width) return;
#pragma unroll
    for (int k = 1; k < kWarps; ++k) s += red[k][lane];
    void* out = blockIdx.y ? db : dw;
    if (accumulate) s += ptype == DL_F32 ? static_cast<float*>(out)[c] : __bfloat162float(static_cast<__nv_bfloat16*>(out)[c]);
    if (ptype == DL_F32)
        static_cast<float*>(out)[c] = s;
    else
        static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(s);
}

// Rows wider than 16384 columns: dx row by row, read again for the second
// phase, and the sums by strips of 32 columns in a pass of their own, all
// element by element (6000 x 20000 bf16: 615 us, 17% of the copy rate).
template <typename T>
__global__ void __launch_bounds__(1024) k_norm_dx_wide(const __grid_constant__ BwdArgs<T> a) {
    __shared__ float2 red[32];
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const float mu = a.rms ? 0.f : a.mean[r], rs = a.rstd[r];
        float2 v = make_float2(0.f, 0.f);
        for (int c = threadIdx.x; c < a.width; c += 1024) {
            const float w = to_f32(a.dy[r * a.ds + c]) * load_param(a.weight, a.ptype, c);
            v.x += w;
            v.y = fmaf(w, (to_f32(a.x[r * a.xs + c]) - mu) * rs, v.y);
        }
        v = block_sum(v, red);
        const float s = a.rms ? 0.f : v.x / a.width, q = v.y / a.width;
        for (int c = threadIdx.x; c < a.width; c += 1024) {
            const float w = to_f32(a.dy[r * a.ds + c]) * load_param(a.weight, a.ptype, c);
            const float h = (to_f32(a.x[r * a.xs + c]) - mu) * rs;
            a.dx[r * a.os + c] = from_f32<T>((w - s - h * q) * rs);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) k_norm_dw_wide(const __grid_constant__ BwdArgs<T> a) {
    __shared__ float sw[kWarps][32], sb[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const int64_t r0 = a.rows * blockIdx.y / kWideParts, r1 = a.rows * (blockIdx.y + 1) / kWideParts;
    float w = 0.f, b = 0.f;
    if (c < a.width)
        for (int64_t r = r0 + warp; r < r1; r += kWarps) {
            const float g = to_f32(a.dy[r * a.ds + c]);
            const float h = (to_f32(a.x[r * a.xs + c]) - (a.rms ? 0.f : a.mean[r])) * a.rstd[r];
            w = fmaf(g, h, w);
            b += g;
        }
    sw[warp][lane] = w;
    sb[warp][lane] = b;
    __syncthreads();
    if (warp == 0 && c < a.width) {
        for (int k = 1; k < kWarps; ++k) w += sw[k][lane], b += sb[k][lane];
        a.part[(2 * blockIdx.y) * int64_t(a.width) + c] = w;
        a.part[(2 * blockIdx.y + 1) * int64_t(a.width) + c] = b;
    }
}

// Launches the pass; returns the number of partial sums or a negative status,
// 0 when nothing was launched: with one round per block, loads straight into
// registers end sooner than copies (64 rows of 4096: 6.1 us on the device
// against 6.4, 300 rows: 9.2 both).
template <typename T, int N, int TPR, int BLOCK, int CLUSTER, bool BULK, bool FULL>
int launch_form(BwdArgs<T> a, cudaStream_t s) {
    using Geo = BwdGeometry<T, TPR, BLOCK, BULK, CLUSTER>;
    auto* kernel = k_norm_bwd<T, N, TPR, BLOCK, BULK, FULL, CLUSTER>;
    static Resident resident;
    const int64_t rounds = (a.rows + Geo::kGroups - 1) / Geo::kGroups;
    int64_t parts = resident.grid(reinterpret_cast<const void*>(kernel), BLOCK, Geo::kBytes, rounds * CLUSTER);
    if (parts == 0) return DL_ERR_CUDA;
    parts = parts < CLUSTER ? 1 : parts / CLUSTER;
    if (parts > kMostBlocks) parts = kMostBlocks;
    if (BULK && rounds <= parts) return 0;
    if (BULK && library_status_word(&a.report.second) != DL_OK) return DL_ERR_CUDA;
    if (BULK) a.report.lost = waits_run_out();
    a.run = (rounds + parts - 1) / parts * Geo::kGroups;
    parts = (a.rows + a.run - 1) / a.run;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(static_cast<unsigned>(parts * CLUSTER));
    config.blockDim = dim3(BLOCK);
    config.dynamicSmemBytes = Geo::kBytes;
    config.stream = s;
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = CLUSTER;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    config.attrs = &cluster;
    config.numAttrs = CLUSTER > 1 ? 1 : 0;
    if (cudaLaunchKernelEx(&config, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return DL_ERR_CUDA;
    }
    return static_cast<int>(parts);
}

template <typename T, int N, int TPR, int BLOCK, int CLUSTER = 1>
int launch(const BwdArgs<T>& a, cudaStream_t s) {
    if constexpr (N > 1) {
        const bool full = a.width == TPR * 16 * CLUSTER && a.vec_out;
        const int parts = full ? launch_form<T, N, TPR, BLOCK, CLUSTER, true, true>(a, s)
                               : launch_form<T, N, TPR, BLOCK, CLUSTER, true, false>(a, s);
        if (parts != 0) return parts;
    }
    return launch_form<T, N, TPR, BLOCK, CLUSTER, false, false>(a, s);
}

// 16 elements per thread: the columns' sums and the packs of 32 would not fit
// the registers of two warps per scheduler. Threads per row follow the width
// (300000 x 200: 289 us with 32, 98 with 16; 16384 x 5632: 155 us with 512,
// 122 with 384).
template <typename T, int N>
int by_width(const BwdArgs<T>& a, cudaStream_t s) {
    if (a.width <= 128) return launch<T, N, 8, 256>(a, s);
    if (a.width <= 256) return launch<T, N, 16, 512>(a, s);
    if (a.width <= 512) return launch<T, N, 32, 512>(a, s);
    if (a.width <= 1024) return launch<T, N, 64, 512>(a, s);
    if (a.width <= 2048) return launch<T, N, 128, 512>(a, s);
    if (a.width <= 4096) return launch<T, N, 256, 512>(a, s);
    if (a.width <= 6144) return launch<T, N, 384, 384>(a, s);
    if (a.width <= 8192) return launch<T, N, 512, 512>(a, s);
    if (a.width <= 16384) return launch<T, N, 512, 512, 2>(a, s);
    // the sums first: dx may overwrite dy
    k_norm_dw_wide<T><<<dim3((a.width + 31) / 32, kWideParts), kThreads, 0, s>>>(a);
    const int64_t most = int64_t(sm_count()) * 2;
    k_norm_dx_wide<T><<<static_cast<int>(a.rows < most ? a.rows : most), 1024, 0, s>>>(a);
    const int st = launch_status();
    return st == DL_OK ? kWideParts : st;
}

template <typename T>
int backward(BwdArgs<T> a, cudaStream_t s) {
    a.vec_out = aligned16(a.dx) && a.os * sizeof(T) % 16 == 0;
    if (aligned16(a.dy) && aligned16(a.x) && a.ds * sizeof(T) % 16 == 0 && a.xs * sizeof(T) % 16 == 0)
        return by_width<T, 16 / sizeof(T)>(a, s);
    return by_width<T, 1>(a, s);
}

}  // namespace
}  // namespace dl

using namespace dl;

extern "C" size_t dl_layernorm_workspace_bytes(int64_t rows, int32_t width) {
    if (rows < 0 || width < 1) return 0;
    const int64_t parts = rows > kMostBlocks ? kMostBlocks : rows < kWideParts ? kWideParts : rows;
    return align256(kWsHeader + size_t(2) * parts * static_cast<size_t>(width) * sizeof(float));
}

extern "C" int dl_layernorm_backward(const void* dy, int64_t dy_stride, const void* x,
                                     int64_t x_stride, int32_t x_type, int64_t rows, int32_t width,
                                     const void* weight, int32_t param_type, const float* mean,
                                     const float* rstd, int32_t flags, void* dx, int64_t dx_stride,
                                     void* dweight, void* dbias, void* d_workspace,
                                     size_t workspace_bytes, void* stream) {
    if ((x_type != DL_F32 && x_type != DL_BF16 && x_type != DL_F16) ||
        (param_type != DL_F32 && param_type != DL_BF16) || rows < 0 || width < 1 ||
        dy_stride < width || x_stride < width || dx_stride < width ||
        (flags & ~(DL_NORM_RMS | DL_NORM_ACCUMULATE)) || !dweight)
        return DL_ERR_ARG;
    const bool rms = flags & DL_NORM_RMS;
    if (rows > 0 && (!dy || !x || !dx || !weight || !rstd || (!rms && !mean))) return DL_ERR_ARG;
    const size_t xa = type_size(x_type), pa = type_size(param_type);
    if (!aligned_to(dy, xa) || !aligned_to(x, xa) || !aligned_to(dx, xa) || !aligned_to(weight, pa) ||
        !aligned_to(dweight, pa) || !aligned_to(dbias, pa) || (!rms && !aligned_to(mean, 4)) ||
        !aligned_to(rstd, 4))
        return DL_ERR_ALIGN;
    if (!d_workspace || workspace_bytes < dl_layernorm_workspace_bytes(rows, width))
        return DL_ERR_WORKSPACE;
    if (!aligned_to(d_workspace, 256)) return DL_ERR_ALIGN;
    const bool accumulate = flags & DL_NORM_ACCUMULATE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    float* part = reinterpret_cast<float*>(static_cast<char*>(d_workspace) + kWsHeader);
    auto call = [&](auto zero) {
        using T = decltype(zero);
        return backward<T>(BwdArgs<T>{static_cast<const T*>(dy), static_cast<const T*>(x),
                                      static_cast<T*>(dx), weight, mean, rstd, part,
                                      RingReport{static_cast<uint32_t*>(d_workspace), nullptr, false},
                                      dy_stride, x_stride, dx_stride, rows, 0, width, param_type, rms,
                                      false},
                           s);
    };
    int parts = 0;
    if (rows > 0)
        parts = x_type == DL_F32 ? call(float()) : x_type == DL_BF16 ? call(__nv_bfloat16()) : call(__half());
    if (parts < 0) return parts;
    // Launched while the pass before it runs (its blocks wait for that pass's
    // end): the launch's latency is not added to the call.
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3((width + 31) / 32, dbias ? 2 : 1);
    config.blockDim = dim3(kThreads);
    config.stream = s;
    cudaLaunchAttribute early;
    early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    early.val.programmaticStreamSerializationAllowed = 1;
    config.attrs = &early;
    config.numAttrs = 1;
    if (cudaLaunchKernelEx(&config, k_norm_join, static_cast<const float*>(part), parts, static_cast<int>(width),
                           param_type, accumulate, dweight, dbias) != cudaSuccess) {
        cudaGetLastError();
        return DL_ERR_CUDA;
    }
    return DL_OK;
}
