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

// Rows in flight per thread; its ring holds one more, the one being read.
// Threads of 32 fp32 elements take one: three would need 256 KB.
template <typename T, int EPT>
constexpr int kRowsAhead = EPT * sizeof(T) > 64 ? 1 : 3;

template <typename T, int N, int TPR, int VPT, int BLOCK>
__global__ void __launch_bounds__(BLOCK) k_norm_fwd(const __grid_constant__ FwdArgs<T> a) {
    constexpr bool kAsync = N * sizeof(T) >= 4;
    constexpr int kAhead = kRowsAhead<T, VPT * N>, kRing = kAhead + 1;
    constexpr int kRowsAtOnce = BLOCK / TPR;
    extern __shared__ __align__(16) unsigned char smem[];
    using P = Pack<T, N>;
    RowSum<TPR, BLOCK> sum{reinterpret_cast<float2*>(smem)};
    P* ring = reinterpret_cast<P*>(smem + RowSum<TPR, BLOCK>::kBytes);
    const int t = threadIdx.x % TPR;
    const int64_t step = int64_t(gridDim.x) * kRowsAtOnce;
    const int64_t r0 = int64_t(blockIdx.x) * kRowsAtOnce;  // of the block
    const int64_t mine = r0 + threadIdx.x / TPR;
    auto issue = [&](int64_t r, int stage) {
        if (r < a.rows) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = (k * TPR + t) * N;
                if (c < a.width)
                    copy_async<N * sizeof(T)>(ring + (stage * VPT + k) * BLOCK + threadIdx.x,
                                              a.x + r * a.xs + c,
                                              static_cast<int>(min(N, a.width - c) * sizeof(T)));
            }
        }
        copy_commit();
    };
    if constexpr (kAsync) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) issue(mine + i * step, i);
    }
    float w[VPT * N], b[VPT * N];
#pragma unroll
    for (int k = 0; k < VPT; ++k)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (k * TPR + t) * N + i;
            w[k * N + i] = c < a.width ? load_param(a.weight, a.ptype, c) : 0.f;
            b[k * N + i] = c < a.width && a.bias ? load_param(a.bias, a.ptype, c) : 0.f;
        }
    const float width = static_cast<float>(a.width);
    int stage = 0;
    for (int64_t first = r0; first < a.rows; first += step) {
        const int64_t r = first + threadIdx.x / TPR;
        float x[VPT * N];
        if constexpr (kAsync) {
            copy_wait<kAhead - 1>();
            // the slot read in the round before this one
            issue(r + kAhead * step, (stage + kAhead) % kRing);
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const int c = (k * TPR + t) * N;
            float v[N];
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] = 0.f;
            if (r < a.rows && c < a.width) {
                if constexpr (kAsync)
                    unpack<T, N>(ring[(stage * VPT + k) * BLOCK + threadIdx.x], v);
                else
                    v[0] = to_f32(a.x[r * a.xs + c]);
            }
#pragma unroll
            for (int i = 0; i < N; ++i) x[k * N + i] = v[i];
        }
        stage = (stage + 1) % kRing;
        float mu = 0.f;
        if (!a.rms) {
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < VPT * N; ++i) s += x[i];
            mu = sum(s) / width;
        }
        float q = 0.f;
#pragma unroll
        for (int k = 0; k < VPT; ++k)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const bool in = (k * TPR + t) * N + i < a.width;
                const float d = in ? x[k * N + i] - mu : 0.f;
                x[k * N + i] = d;
                q = fmaf(d, d, q);
            }
        const float rs = rsqrtf(sum(q) / width + a.eps);
        if (r < a.rows) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = (k * TPR + t) * N;
                float v[N];
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = fmaf(x[k * N + i] * rs, w[k * N + i], b[k * N + i]);
                if (c < a.width) store_pack<T, N>(a.y + r * a.ys + c, v, a.width - c, a.vec_out);
            }
            if (t == 0) {
                if (!a.rms) a.mean[r] = mu;
                a.rstd[r] = rs;
            }
        }
    }
}

// Rows too wide for a block's registers: the row is read three times (from
// L2 after the first).
template <typename T>
__global__ void __launch_bounds__(1024) k_norm_fwd_wide(const __grid_constant__ FwdArgs<T> a) {
    __shared__ float2 red[2 * 32];
    RowSum<1024, 1024> sum{red};
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const T* xr = a.x + r * a.xs;
        float mu = 0.f;
        if (!a.rms) {
            float s = 0.f;
            for (int c = threadIdx.x; c < a.width; c += 1024) s += to_f32(xr[c]);
            mu = sum(s) / a.width;
        }
        float q = 0.f;
        for (int c = threadIdx.x; c < a.width; c += 1024) {
            const float d = to_f32(xr[c]) - mu;
            q = fmaf(d, d, q);
        }
        const float rs = rsqrtf(sum(q) / a.width + a.eps);
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
                        (N * sizeof(T) >= 4 ? size_t(kRowsAhead<T, VPT * N> + 1) * VPT * BLOCK * N * sizeof(T) : 0);
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
