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
    int64_t xs, ys, rows;
    int width;
    int32_t ptype;
    float eps;
    bool rms, vec_out;
};

// Rows in flight per thread beyond the three being worked on. Threads of 32
// fp32 elements take none: their ring would pass 227 KB.
template <typename T, int EPT>
constexpr int kRowsAhead = EPT * sizeof(T) > 64 ? 0 : 2;

// A block's rounds take one row of each group of TPR threads. A round sums
// its row, sums the squared deviations of the row before (whose mean is known
// by then) and finishes the row before that: the two sums of a round travel
// together, with one barrier, and the wait for it is spent on other rows.
template <typename T, int N, int TPR, int VPT, int BLOCK>
__global__ void __launch_bounds__(BLOCK) k_norm_fwd(const __grid_constant__ FwdArgs<T> a) {
    constexpr int kAhead = kRowsAhead<T, VPT * N>, kStages = kAhead + 3;
    constexpr bool kAsync = N * sizeof(T) >= 4 && kAhead > 0;
    constexpr int kGroups = BLOCK / TPR, kPairs = VPT * N / 2;
    extern __shared__ __align__(16) unsigned char smem[];
    using P = Pack<T, N>;
    RowSum<TPR, BLOCK> sum{reinterpret_cast<float2*>(smem)};
    P* ring = reinterpret_cast<P*>(smem + RowSum<TPR, BLOCK>::kBytes) + threadIdx.x;
    const int t = threadIdx.x % TPR;
    const int64_t step = int64_t(gridDim.x) * kGroups;  // from one of a group's rows to its next
    const int64_t r0 = int64_t(blockIdx.x) * kGroups;
    const int64_t mine = r0 + threadIdx.x / TPR;
    auto issue = [&](int64_t r, int stage) {
        if (r < a.rows) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = (k * TPR + t) * N;
                if (c < a.width)
                    copy_async<N * sizeof(T)>(ring + (stage * VPT + k) * BLOCK, a.x + r * a.xs + c,
                                              static_cast<int>(min(N, a.width - c) * sizeof(T)));
            }
        }
        copy_commit();
    };
    if constexpr (kAsync) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) issue(mine + i * step, i);
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
            valid |= static_cast<uint32_t>(in) << e;
            f[i] = in ? load_param(a.weight, a.ptype, c) : 0.f;
            g[i] = in && a.bias ? load_param(a.bias, a.ptype, c) : 0.f;
        }
        w[p] = make_float2(f[0], f[1]), b[p] = make_float2(g[0], g[1]);
    }
    const bool whole = valid == (VPT * N == 32 ? ~0u : (1u << (VPT * N % 32)) - 1u);
    const float width = static_cast<float>(a.width), inv = 1.0f / width;
    // row r's deviations from mu; zeros past the width (where the ring's slots are stale)
    auto read = [&](int64_t r, int stage, float mu, float2 (&x)[kPairs]) {
        P raw[VPT];
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            if constexpr (kAsync) {
                raw[k] = ring[(stage * VPT + k) * BLOCK];
            } else {
                const int c = (k * TPR + t) * N;
#pragma unroll
                for (int i = 0; i < N; ++i) raw[k].v[i] = from_f32<T>(0.f);
                if (r >= 0 && r < a.rows) {
                    if (N > 1 && c + N <= a.width) {
                        raw[k] = *reinterpret_cast<const P*>(a.x + r * a.xs + c);
                    } else {
#pragma unroll
                        for (int i = 0; i < N; ++i)
                            if (c + i < a.width) raw[k].v[i] = a.x[r * a.xs + c + i];
                    }
                }
            }
        }
#pragma unroll
        for (int p = 0; p < kPairs; ++p) x[p] = add2(pair_of<T, N>(raw, p), both(-mu));
        if (!whole) {
#pragma unroll
            for (int p = 0; p < kPairs; ++p) {
                if (!(valid >> (2 * p) & 1)) x[p].x = 0.f;
                if (!(valid >> (2 * p + 1) & 1)) x[p].y = 0.f;
            }
        }
    };
    int stage = 0, stage1 = kStages - 1, stage2 = kStages - 2, set = 0;  // of this row and the two before
    float mu = 0.f;                                                      // of the row before
    const int64_t rounds = r0 < a.rows ? (a.rows - r0 + step - 1) / step : 0;
    int64_t r = mine;
    for (int64_t i = 0; i < rounds + 2; ++i, r += step) {
        const float2 total = sum.take(set ^ 1);
        float2 x[kPairs], part = make_float2(0.f, 0.f);
        if constexpr (kAsync) {
            copy_wait<kAhead - 1>();
            issue(r + kAhead * step, stage + kAhead < kStages ? stage + kAhead : stage + kAhead - kStages);
        }
        if (!a.rms && i < rounds) {
            read(r, stage, 0.f, x);
            float2 s = x[0];
#pragma unroll
            for (int p = 1; p < kPairs; ++p) s = add2(s, x[p]);
            part.x = s.x + s.y;
        }
        const float mu2 = mu;
        if (i >= 1 && i <= rounds) {
            mu = a.rms ? 0.f : divided(total.x, width, inv);
            read(r - step, stage1, mu, x);
            float2 q = mul2(x[0], x[0]);
#pragma unroll
            for (int p = 1; p < kPairs; ++p) q = fma2(x[p], x[p], q);
            part.y = q.x + q.y;
        }
        sum.give(part, set);
        if (i >= 2) {
            const int64_t row = r - 2 * step;
            const float rs = rsqrtf(fmaf(total.y, inv, a.eps));
            read(row, stage2, mu2, x);
            if (row < a.rows) {
#pragma unroll
                for (int p = 0; p < kPairs; ++p) x[p] = fma2(mul2(x[p], both(rs)), w[p], b[p]);
                store_row<T, N, TPR, VPT>(a.y + row * a.ys, x, t, a.width, whole && a.vec_out);
                if (t == 0) {
                    if (!a.rms) a.mean[row] = mu2;
                    a.rstd[row] = rs;
                }
            }
        }
        if constexpr (RowSum<TPR, BLOCK>::kShared) __syncthreads();
        set ^= 1;
        stage2 = stage1, stage1 = stage;
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
}

// Rows too wide for a block's registers: the row is read three times (from
// L2 after the first).
template <typename T>
__global__ void __launch_bounds__(1024) k_norm_fwd_wide(const __grid_constant__ FwdArgs<T> a) {
    __shared__ float2 red[32];
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* xr = a.x + r * a.xs;
        float mu = 0.f;
        if (!a.rms) {
            float s = 0.f;
            for (int c = threadIdx.x; c < a.width; c += 1024) s += to_f32(xr[c]);
            mu = block_sum(make_float2(s, 0.f), red).x / a.width;
        }
        float q = 0.f;
        for (int c = threadIdx.x; c < a.width; c += 1024) {
            const float d = to_f32(xr[c]) - mu;
            q = fmaf(d, d, q);
        }
        const float rs = rsqrtf(block_sum(make_float2(q, 0.f), red).x / a.width + a.eps);
        for (int c = threadIdx.x; c < a.width; c += 1024) {
            const float h = (to_f32(xr[c]) - mu) * rs * load_param(a.weight, a.ptype, c);
            a.y[r * a.ys + c] = from_f32<T>(a.bias ? h + load_param(a.bias, a.ptype, c) : h);
        }
        if (threadIdx.x == 0) {
            if (!a.rms) a.mean[r] = mu;
            a.rstd[r] = rs;
        }
    }
}

template <typename T, int N, int TPR, int VPT, int BLOCK>
int launch(const FwdArgs<T>& a, cudaStream_t s) {
    const void* kernel = reinterpret_cast<const void*>(k_norm_fwd<T, N, TPR, VPT, BLOCK>);
    const size_t smem = RowSum<TPR, BLOCK>::kBytes +
                        (N * sizeof(T) >= 4 && kRowsAhead<T, VPT * N> > 0
                             ? size_t(kRowsAhead<T, VPT * N> + 3) * VPT * BLOCK * N * sizeof(T)
                             : 0);
    if (!allow_shared(kernel, smem)) return DL_ERR_CUDA;
    constexpr int at_once = BLOCK / TPR;
    const int grid = grid_for(kernel, BLOCK, smem, (a.rows + at_once - 1) / at_once);
    k_norm_fwd<T, N, TPR, VPT, BLOCK><<<grid, BLOCK, smem, s>>>(a);
    return launch_status();
}

// 16 elements per thread up to 8192 columns, 32 above.
template <typename T, int N>
int by_width(const FwdArgs<T>& a, cudaStream_t s) {
    if (a.width <= 128) return launch<T, N, 8, 16 / N, 256>(a, s);
    if (a.width <= 512) return launch<T, N, 32, 16 / N, 256>(a, s);
    if (a.width <= 1024) return launch<T, N, 64, 16 / N, 256>(a, s);
    if (a.width <= 2048) return launch<T, N, 128, 16 / N, 256>(a, s);
    if (a.width <= 4096) return launch<T, N, 256, 16 / N, 256>(a, s);
    if (a.width <= 8192) return launch<T, N, 512, 16 / N, 512>(a, s);
    if (a.width <= 16384) return launch<T, N, 512, 32 / N, 512>(a, s);
    const int64_t most = int64_t(sm_count()) * 2;
    k_norm_fwd_wide<T><<<static_cast<int>(a.rows < most ? a.rows : most), 1024, 0, s>>>(a);
    return launch_status();
}

template <typename T>
int forward(const void* x, int64_t xs, int64_t rows, int width, const void* w, const void* b,
            int32_t pt, float eps, bool rms, void* y, int64_t ys, float* mean, float* rstd,
            cudaStream_t s) {
    FwdArgs<T> a{static_cast<const T*>(x), static_cast<T*>(y), w, b, mean, rstd, xs, ys, rows, width,
                 pt, eps, rms, false};
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
