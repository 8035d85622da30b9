// Layer norm (centred or RMS) forward.
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "dl_norm.cuh"

namespace dl {
namespace {

template <typename T>
struct FwdArgs {
    const T* x;
    T* y;
    const void* weight;
    const void* bias;
    float* mean;
    float* rstd;
    RingReport report;
    int64_t xs, ys, rows;
    int64_t run;  // rows of a block
    int width;
    int32_t ptype;
    float eps;
    bool rms, vec_out;
};

template <typename T, int TPR, int EPT, int BLOCK, bool BULK>
struct FwdGeometry {
    static constexpr int kGroups = BLOCK / TPR, kStages = 3;
    using Ring = RowRing<T, TPR, EPT, BLOCK, 1, kStages>;
    static constexpr size_t kFixed = 128 + RowSum<TPR, BLOCK>::kBytes;
    static constexpr size_t kBytes = kFixed + (BULK ? Ring::kBytes : 0);
};

// A round: the row's sum, a barrier, the sum of its squared deviations, a
// barrier, and the result from the deviations, still in registers. FULL: the
// threads' packs cover the width exactly and y's rows are aligned.
//
// Bound by HBM on paper (two passes of the row's bytes); what it fights is
// the latency of two dependent sums per row. 32 elements per thread halve the
// instructions per element against 16 (92 us at three blocks per SM); two
// blocks of 256 threads per SM work on four rows of 4096 at once; three
// stages (two: 120 us, four: 101 us).
// 32768 x 4096 bf16: 89 us, 6.1 TB/s (89% of the copy rate), RMS 84 us (94%);
// fp16 the same, fp32 177 us (89%).
// A few rows (5 x 2048): 3.9 us on the device.
template <typename T, int N, int TPR, int EPT, int BLOCK, bool BULK, bool FULL>
__global__ void __launch_bounds__(BLOCK, 512 / BLOCK) k_norm_fwd(const __grid_constant__ FwdArgs<T> a) {
    using Geo = FwdGeometry<T, TPR, EPT, BLOCK, BULK>;
    constexpr int VPT = EPT / N, kGroups = Geo::kGroups, kPairs = EPT / 2;
    constexpr bool kBarrier = RowSum<TPR, BLOCK>::kShared;
    extern __shared__ __align__(128) unsigned char smem[];
    using P = Pack<T, N>;
    RowSum<TPR, BLOCK> sum{reinterpret_cast<float2*>(smem + 128)};
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int64_t begin = a.run * blockIdx.x, end = min(a.rows, begin + a.run);
    const uint32_t bytes = static_cast<uint32_t>(a.width * sizeof(T)) & ~15u;
    const bool together = bytes == a.width * sizeof(T) && a.xs == a.width;
    typename Geo::Ring ring{smem + Geo::kFixed, reinterpret_cast<uint64_t*>(smem), a.report, end, bytes,
                            together ? bytes : static_cast<uint32_t>(Geo::Ring::kRow)};
    if constexpr (BULK) {
        ring.init();
#pragma unroll
        for (int i = 0; i < Geo::kStages - 1; ++i) ring.issue(i, begin + i * kGroups, a.x, a.xs, a.x, a.xs);
        if (a.report.lost) ring.lose(begin);
    }
    float2 w[kPairs], b[kPairs];
    uint32_t valid = 0;  // a bit per element below the width
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
        float f[2], g[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = 2 * p + i, c = ((e / N) * TPR + t) * N + e % N;
            const bool in = c < a.width;
            if (!FULL) valid |= static_cast<uint32_t>(in) << e;
            f[i] = in ? load_param(a.weight, a.ptype, c) : 0.f;
            g[i] = in && a.bias ? load_param(a.bias, a.ptype, c) : 0.f;
        }
        w[p] = make_float2(f[0], f[1]), b[p] = make_float2(g[0], g[1]);
    }
    // 1 for packs with elements below the width, 0 for the others: their zeros
    // have no deviation
    float has[VPT];
#pragma unroll
    for (int k = 0; k < VPT; ++k) has[k] = (k * TPR + t) * N < a.width ? 1.f : 0.f;
    // a last, partial pack; the elements of a pack of one are covered by `has`
    const bool cut = !FULL && N > 1 && a.width % N != 0 && (a.width / N) % TPR == t;
    const float width = static_cast<float>(a.width), inv = 1.0f / width;
    int set = 0;
    for (int64_t first = begin; first < end; first += kGroups) {
        const int64_t r = first + group;
        // off 16 bytes, 16384 x 5001 bf16 131 -> 111 us, but 60000 x 501 54 -> 56 and RMS 39 -> 45 without the bound
        if constexpr (!BULK && TPR >= 192) prefetch_rows(first + kGroups, kGroups, end, a.x, a.xs, a.width);
        const bool in = kGroups == 1 || r < end;
        float2 x[kPairs];
        if constexpr (BULK) ring.wait(first);
        {
            P raw[VPT];
            const P* from = (BULK ? reinterpret_cast<const P*>(ring.row(ring.stage(), group, 0))
                                  : reinterpret_cast<const P*>(a.x + r * a.xs)) + t;
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = (k * TPR + t) * N;
                if (FULL || (in && c + N <= a.width)) {
                    raw[k] = from[k * TPR];  // FULL: a stage's rows past the last are stale and not used
                } else {  // zeros past the width and the rows
#pragma unroll
                    for (int i = 0; i < N; ++i) raw[k].v[i] = from_f32<T>(0.f);
                    if (N > 1 && in && c < a.width)  // a last, partial pack
#pragma unroll
                        for (int i = 0; i < N - 1; ++i)
                            if (c + i < a.width) raw[k].v[i] = a.x[r * a.xs + c + i];
                }
            }
#pragma unroll
            for (int p = 0; p < kPairs; ++p) x[p] = pair_of<T, N>(raw, p);
        }
        float mu = 0.f;
        if (!a.rms) {
            float2 s = x[0];
#pragma unroll
            for (int p = 1; p < kPairs; ++p) s = add2(s, x[p]);
            sum.give(s.x + s.y, set);
            if constexpr (kBarrier) __syncthreads();
            mu = divided(sum.take1(set), width, inv);
            set ^= 1;
#pragma unroll
            for (int p = 0; p < kPairs; ++p)
                x[p] = FULL ? add2(x[p], both(-mu))
                            : fma2(make_float2(has[2 * p / N], has[(2 * p + 1) / N]), both(-mu), x[p]);
            if (cut) {
#pragma unroll
                for (int p = 0; p < kPairs; ++p) {
                    if (!(valid >> (2 * p) & 1)) x[p].x = 0.f;
                    if (!(valid >> (2 * p + 1) & 1)) x[p].y = 0.f;
                }
            }
        }
        float2 q = mul2(x[0], x[0]);
#pragma unroll
        for (int p = 1; p < kPairs; ++p) q = fma2(x[p], x[p], q);
        sum.give(q.x + q.y, set);
        if constexpr (kBarrier || BULK) __syncthreads();
        if constexpr (BULK) {  // every thread has read this round's stage, and the one before it long ago
            ring.issue(ring.before(), first + (Geo::kStages - 1) * kGroups, a.x, a.xs, a.x, a.xs);
            ring.advance();
        }
        const float rs = rsqrtf(fmaf(sum.take1(set), inv, a.eps));
        set ^= 1;
        if (in) {
#pragma unroll
            for (int p = 0; p < kPairs; ++p) x[p] = fma2(mul2(x[p], both(rs)), w[p], b[p]);
            store_row<T, N, TPR, VPT, FULL>(a.y + r * a.ys, x, t, a.width, a.vec_out);
            if (t == 0) {
                if (!a.rms) a.mean[r] = mu;
                a.rstd[r] = rs;
            }
        }
    }
    if constexpr (BULK) ring.drain();
}

// Rows too wide for a block's registers: the row is read three times (from
// L2 after the first), element by element: 6000 x 20000 bf16 257 us (27% of the
// copy rate). Columns count in 64 bits: a step past a width near 2^31
// would not fit 32.
template <typename T>
__global__ void __launch_bounds__(1024) k_norm_fwd_wide(const __grid_constant__ FwdArgs<T> a) {
    __shared__ float2 red[32];
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* xr = a.x + r * a.xs;
        float mu = 0.f;
        if (!a.rms) {
            float s = 0.f;
            for (int64_t c = threadIdx.x; c < a.width; c += 1024) s += to_f32(xr[c]);
            mu = block_sum(make_float2(s, 0.f), red).x / a.width;
        }
        float q = 0.f;
        for (int64_t c = threadIdx.x; c < a.width; c += 1024) {
            const float d = to_f32(xr[c]) - mu;
            q = fmaf(d, d, q);
        }
        const float rs = rsqrtf(block_sum(make_float2(q, 0.f), red).x / a.width + a.eps);
        for (int64_t c = threadIdx.x; c < a.width; c += 1024) {
            const float h = (to_f32(xr[c]) - mu) * rs * load_param(a.weight, a.ptype, c);
            a.y[r * a.ys + c] = from_f32<T>(a.bias ? h + load_param(a.bias, a.ptype, c) : h);
        }
        if (threadIdx.x == 0) {
            if (!a.rms) a.mean[r] = mu;
            a.rstd[r] = rs;
        }
    }
}

// False when nothing was launched: with one round per block there is nothing
// to stage ahead, and loads straight into registers end sooner (64 rows of
// 4096: 5.1 us on the device against 5.4; at two rounds the copies win, 7.4
// against 7.6).
template <typename T, int N, int TPR, int EPT, int BLOCK, bool BULK, bool FULL>
bool launch(FwdArgs<T> a, cudaStream_t s, int* status) {
    using Geo = FwdGeometry<T, TPR, EPT, BLOCK, BULK>;
    const void* kernel = reinterpret_cast<const void*>(k_norm_fwd<T, N, TPR, EPT, BLOCK, BULK, FULL>);
    *status = DL_ERR_CUDA;
    static Resident resident;
    const int64_t rounds = (a.rows + Geo::kGroups - 1) / Geo::kGroups;
    int64_t grid = resident.grid(kernel, BLOCK, Geo::kBytes, rounds);
    if (grid == 0) return true;
    if (BULK && rounds <= grid) return false;
    if (BULK && library_status_word(&a.report.word) != DL_OK) return true;
    if (BULK) a.report.lost = waits_run_out();
    a.run = (rounds + grid - 1) / grid * Geo::kGroups;
    grid = (a.rows + a.run - 1) / a.run;
    k_norm_fwd<T, N, TPR, EPT, BLOCK, BULK, FULL><<<static_cast<int>(grid), BLOCK, Geo::kBytes, s>>>(a);
    *status = launch_status();
    return true;
}

template <typename T, int N, int TPR, int EPT, int BLOCK>
int launch(const FwdArgs<T>& a, cudaStream_t s) {
    int status;
    if constexpr (N > 1) {
        const bool full = a.width == TPR * EPT && a.vec_out;
        if (full ? launch<T, N, TPR, EPT, BLOCK, true, true>(a, s, &status)
                 : launch<T, N, TPR, EPT, BLOCK, true, false>(a, s, &status))
            return status;
    }
    launch<T, N, TPR, EPT, BLOCK, false, false>(a, s, &status);
    return status;
}

// 32 elements per thread where a row has them: half of a round's work is the
// same for a thread of 16. Narrower rows take fewer (500000 rows of 64: 161 us
// with 32, 46 with 8), rows to 6144 three quarters of the threads of 8192
// (16384 x 5632: 96 -> 78 us).
template <typename T, int N>
int by_width(const FwdArgs<T>& a, cudaStream_t s) {
    if (a.width <= 64) return launch<T, N, 8, 8, 256>(a, s);
    if (a.width <= 128) return launch<T, N, 8, 16, 256>(a, s);
    if (a.width <= 256) return launch<T, N, 8, 32, 256>(a, s);
    if (a.width <= 1024) return launch<T, N, 32, 32, 256>(a, s);
    if (a.width <= 2048) return launch<T, N, 64, 32, 256>(a, s);
    if (a.width <= 4096) return launch<T, N, 128, 32, 256>(a, s);
    if (a.width <= 6144) return launch<T, N, 192, 32, 384>(a, s);
    if (a.width <= 8192) return launch<T, N, 256, 32, 256>(a, s);
    if (a.width <= 16384) return launch<T, N, 512, 32, 512>(a, s);
    const int64_t most = int64_t(sm_count()) * 2;
    k_norm_fwd_wide<T><<<static_cast<int>(a.rows < most ? a.rows : most), 1024, 0, s>>>(a);
    return launch_status();
}

template <typename T>
int forward(const void* x, int64_t xs, int64_t rows, int width, const void* w, const void* b,
            int32_t pt, float eps, bool rms, void* y, int64_t ys, float* mean, float* rstd,
            cudaStream_t s) {
    FwdArgs<T> a{static_cast<const T*>(x), static_cast<T*>(y), w, b, mean, rstd, {}, xs, ys,
                 rows, 0, width, pt, eps, rms, false};
    a.vec_out = aligned16(y) && ys * sizeof(T) % 16 == 0;
    if (aligned16(x) && xs * sizeof(T) % 16 == 0) return by_width<T, 16 / sizeof(T)>(a, s);
    return by_width<T, 1>(a, s);
}

}  // namespace

}  // namespace dl

using namespace dl;

extern "C" int dl_layernorm_forward(const void* x, int64_t x_stride, int32_t x_type, int64_t rows,
                                    int32_t width, const void* weight, const void* bias,
                                    int32_t param_type, double eps, int32_t flags, void* y,
                                    int64_t y_stride, float* mean, float* rstd, void* stream) {
    if ((x_type != DL_F32 && x_type != DL_BF16 && x_type != DL_F16) ||
        (param_type != DL_F32 && param_type != DL_BF16) || rows < 0 || width < 1 ||
        x_stride < width || y_stride < width || !(eps >= 0.0 && eps <= FLT_MAX) ||
        (flags & ~DL_NORM_RMS))
        return DL_ERR_ARG;
    if (rows == 0) return DL_OK;
    const bool rms = flags & DL_NORM_RMS;
    if (!x || !y || !weight || !rstd || (!rms && !mean)) return DL_ERR_ARG;
    if (!aligned_to(x, type_size(x_type)) || !aligned_to(y, type_size(x_type)) ||
        !aligned_to(weight, type_size(param_type)) || !aligned_to(bias, type_size(param_type)) ||
        (!rms && !aligned_to(mean, 4)) || !aligned_to(rstd, 4))
        return DL_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const float e = static_cast<float>(eps);
    switch (x_type) {
        case DL_F32:
            return forward<float>(x, x_stride, rows, width, weight, bias, param_type, e, rms, y,
                                  y_stride, mean, rstd, s);
        case DL_BF16:
            return forward<__nv_bfloat16>(x, x_stride, rows, width, weight, bias, param_type, e, rms,
                                          y, y_stride, mean, rstd, s);
        default:
            return forward<__half>(x, x_stride, rows, width, weight, bias, param_type, e, rms, y,
                                   y_stride, mean, rstd, s);
    }
}
