// Layer norm (centred or RMS) forward and backward.
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "dl_types.cuh"

namespace dl {
namespace {

__device__ __forceinline__ float load_param(const void* p, int32_t type, int64_t i) {
    return type == DL_F32 ? static_cast<const float*>(p)[i]
                          : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

__device__ __forceinline__ float block_sum(float v, float* red) {
    for (int sh = 16; sh; sh >>= 1) v += __shfl_xor_sync(kFull, v, sh);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.f;
    for (int w = 0; w < kWarps; ++w) s += red[w];
    return s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_norm_fwd(const T* x, int64_t xs, int64_t rows, int width, const void* weight,
               const void* bias, int32_t ptype, float eps, bool rms, T* y, int64_t ys, float* mean,
               float* rstd) {
    __shared__ float red[kWarps];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const T* xr = x + r * xs;
        float mu = 0.f;
        if (!rms) {
            float s = 0.f;
            for (int c = threadIdx.x; c < width; c += kThreads) s += to_f32(xr[c]);
            mu = block_sum(s, red) / width;
        }
        float q = 0.f;
        for (int c = threadIdx.x; c < width; c += kThreads) {
            const float d = to_f32(xr[c]) - mu;
            q = fmaf(d, d, q);
        }
        const float rs = 1.0f / sqrtf(block_sum(q, red) / width + eps);
        for (int c = threadIdx.x; c < width; c += kThreads) {
            const float h = (to_f32(xr[c]) - mu) * rs * load_param(weight, ptype, c);
            y[r * ys + c] = from_f32<T>(bias ? h + load_param(bias, ptype, c) : h);
        }
        if (threadIdx.x == 0) {
            if (!rms) mean[r] = mu;
            rstd[r] = rs;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_norm_dx(const T* dy, int64_t ds, const T* x, int64_t xs, int64_t rows, int width,
              const void* weight, int32_t ptype, const float* mean, const float* rstd, bool rms,
              T* dx, int64_t os) {
    __shared__ float red[kWarps];
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
        const float mu = rms ? 0.f : mean[r], rs = rstd[r];
        float s = 0.f, q = 0.f;
        for (int c = threadIdx.x; c < width; c += kThreads) {
            const float w = to_f32(dy[r * ds + c]) * load_param(weight, ptype, c);
            s += w;
            q = fmaf(w, (to_f32(x[r * xs + c]) - mu) * rs, q);
        }
        s = rms ? 0.f : block_sum(s, red) / width;
        q = block_sum(q, red) / width;
        for (int c = threadIdx.x; c < width; c += kThreads) {
            const float w = to_f32(dy[r * ds + c]) * load_param(weight, ptype, c);
            const float h = (to_f32(x[r * xs + c]) - mu) * rs;
            dx[r * os + c] = from_f32<T>((w - s - h * q) * rs);
        }
    }
}

// Sums over rows: block (strip of 32 columns, part of the rows); warp w takes
// every eighth row of the part; partial sums go to the workspace.
constexpr int kParts = 32;

template <typename T>
__global__ void __launch_bounds__(kThreads)
    k_norm_dw(const T* dy, int64_t ds, const T* x, int64_t xs, int64_t rows, int width,
              const float* mean, const float* rstd, bool rms, float* part) {
    __shared__ float sw[kWarps][32], sb[kWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int c = blockIdx.x * 32 + lane;
    const int64_t r0 = rows * blockIdx.y / kParts, r1 = rows * (blockIdx.y + 1) / kParts;
    float w = 0.f, b = 0.f;
    if (c < width)
        for (int64_t r = r0 + warp; r < r1; r += kWarps) {
            const float g = to_f32(dy[r * ds + c]);
            const float h = (to_f32(x[r * xs + c]) - (rms ? 0.f : mean[r])) * rstd[r];
            w = fmaf(g, h, w);
            b += g;
        }
    sw[warp][lane] = w;
    sb[warp][lane] = b;
    __syncthreads();
    if (warp == 0 && c < width) {
        for (int k = 1; k < kWarps; ++k) w += sw[k][lane], b += sb[k][lane];
        part[(2 * blockIdx.y) * int64_t(width) + c] = w;
        part[(2 * blockIdx.y + 1) * int64_t(width) + c] = b;
    }
}

__global__ void __launch_bounds__(kThreads)
    k_norm_join(const float* part, int width, int32_t ptype, bool accumulate, void* dw, void* db) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= width) return;
    for (int k = 0; k < (db ? 2 : 1); ++k) {
        float s = 0.f;
        for (int p = 0; p < kParts; ++p) s += part[(2 * p + k) * int64_t(width) + c];
        void* out = k ? db : dw;
        if (accumulate) s += load_param(out, ptype, c);
        if (ptype == DL_F32)
            static_cast<float*>(out)[c] = s;
        else
            static_cast<__nv_bfloat16*>(out)[c] = __float2bfloat16_rn(s);
    }
}

bool aligned_to(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int grid_rows(int64_t rows) {
    const int64_t most = int64_t(sm_count()) * 8;
    return static_cast<int>(rows < most ? rows : most);
}

template <typename T>
int forward(const void* x, int64_t xs, int64_t rows, int width, const void* w, const void* b,
            int32_t pt, float eps, bool rms, void* y, int64_t ys, float* mean, float* rstd,
            cudaStream_t s) {
    k_norm_fwd<T><<<grid_rows(rows), kThreads, 0, s>>>(static_cast<const T*>(x), xs, rows, width, w,
                                                       b, pt, eps, rms, static_cast<T*>(y), ys, mean,
                                                       rstd);
    return launch_status();
}

template <typename T>
int backward(const void* dy, int64_t ds, const void* x, int64_t xs, int64_t rows, int width,
             const void* w, int32_t pt, const float* mean, const float* rstd, bool rms,
             bool accumulate, void* dx, int64_t os, void* dw, void* db, float* part,
             cudaStream_t s) {
    const T* dyt = static_cast<const T*>(dy);
    const T* xt = static_cast<const T*>(x);
    // the sums first: dx may overwrite dy
    k_norm_dw<T><<<dim3((width + 31) / 32, kParts), kThreads, 0, s>>>(dyt, ds, xt, xs, rows, width,
                                                                      mean, rstd, rms, part);
    if (rows > 0)
        k_norm_dx<T><<<grid_rows(rows), kThreads, 0, s>>>(dyt, ds, xt, xs, rows, width, w, pt, mean,
                                                          rstd, rms, static_cast<T*>(dx), os);
    k_norm_join<<<(width + kThreads - 1) / kThreads, kThreads, 0, s>>>(part, width, pt, accumulate,
                                                                       dw, db);
    return launch_status();
}

bool activation_type(int32_t t) { return t == DL_F32 || t == DL_BF16 || t == DL_F16; }
bool param_type_ok(int32_t t) { return t == DL_F32 || t == DL_BF16; }

}  // namespace
}  // namespace dl

using namespace dl;

extern "C" int dl_layernorm_forward(const void* x, int64_t x_stride, int32_t x_type, int64_t rows,
                                    int32_t width, const void* weight, const void* bias,
                                    int32_t param_type, double eps, int32_t flags, void* y,
                                    int64_t y_stride, float* mean, float* rstd, void* stream) {
    if (!activation_type(x_type) || !param_type_ok(param_type) || rows < 0 || width < 1 ||
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

extern "C" size_t dl_layernorm_workspace_bytes(int64_t rows, int32_t width) {
    if (rows < 0 || width < 1) return 0;
    return align256(kWsHeader + size_t(2) * kParts * static_cast<size_t>(width) * sizeof(float));
}

extern "C" int dl_layernorm_backward(const void* dy, int64_t dy_stride, const void* x,
                                     int64_t x_stride, int32_t x_type, int64_t rows, int32_t width,
                                     const void* weight, int32_t param_type, const float* mean,
                                     const float* rstd, int32_t flags, void* dx, int64_t dx_stride,
                                     void* dweight, void* dbias, void* d_workspace,
                                     size_t workspace_bytes, void* stream) {
    if (!activation_type(x_type) || !param_type_ok(param_type) || rows < 0 || width < 1 ||
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
    const bool acc = flags & DL_NORM_ACCUMULATE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    float* part = reinterpret_cast<float*>(static_cast<char*>(d_workspace) + kWsHeader);
    switch (x_type) {
        case DL_F32:
            return backward<float>(dy, dy_stride, x, x_stride, rows, width, weight, param_type, mean,
                                   rstd, rms, acc, dx, dx_stride, dweight, dbias, part, s);
        case DL_BF16:
            return backward<__nv_bfloat16>(dy, dy_stride, x, x_stride, rows, width, weight,
                                           param_type, mean, rstd, rms, acc, dx, dx_stride, dweight,
                                           dbias, part, s);
        default:
            return backward<__half>(dy, dy_stride, x, x_stride, rows, width, weight, param_type,
                                    mean, rstd, rms, acc, dx, dx_stride, dweight, dbias, part, s);
    }
}
