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
    int64_t ds, xs, os, rows;
    int width;
    int32_t ptype;
    bool rms, vec_out;
};

template <typename T, int N, int TPR, int VPT, int BLOCK, int AHEAD>
__global__ void __launch_bounds__(BLOCK) k_norm_bwd(const __grid_constant__ BwdArgs<T> a) {
    constexpr bool kAsync = N * sizeof(T) >= 4;
    constexpr int kRing = AHEAD + 1;
    constexpr int kRowsAtOnce = BLOCK / TPR;
    // Elements are handled in pairs: of one pack, or for single elements of
    // two neighbouring packs of the thread.
    constexpr int kPairs = VPT * N / 2;
    extern __shared__ __align__(16) unsigned char smem[];
    using P = Pack<T, N>;
    RowSum<TPR, BLOCK> sum{reinterpret_cast<float2*>(smem)};
    P* ring = reinterpret_cast<P*>(smem + RowSum<TPR, BLOCK>::kBytes);
    const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
    const int64_t step = int64_t(gridDim.x) * kRowsAtOnce;
    const int64_t r0 = int64_t(blockIdx.x) * kRowsAtOnce;
    auto column = [&](int k) { return (k * TPR + t) * N; };
    auto issue = [&](int64_t r, int stage) {
        if (r < a.rows) {
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                const int c = column(k);
                if (c < a.width) {
                    const int valid = static_cast<int>(min(N, a.width - c) * sizeof(T));
                    P* to = ring + (stage * 2 * VPT + k) * BLOCK + threadIdx.x;
                    copy_async<N * sizeof(T)>(to, a.dy + r * a.ds + c, valid);
                    copy_async<N * sizeof(T)>(to + VPT * BLOCK, a.x + r * a.xs + c, valid);
                }
            }
        }
        copy_commit();
    };
    if constexpr (kAsync) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) issue(r0 + group + i * step, i);
    }
    float2 w[kPairs], dw[kPairs], db[kPairs];
#pragma unroll
    for (int p = 0; p < kPairs; ++p) {
        float f[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int e = 2 * p + i, c = column(e / N) + e % N;
            f[i] = c < a.width ? load_param(a.weight, a.ptype, c) : 0.f;
        }
        w[p] = make_float2(f[0], f[1]);
        dw[p] = db[p] = make_float2(0.f, 0.f);
    }
    const float width = static_cast<float>(a.width);
    int64_t r = r0 + group;
    float mu = 0.f, rs = 0.f;
    if (r < a.rows) {
        if (!a.rms) mu = __ldg(a.mean + r);
        rs = __ldg(a.rstd + r);
    }
    int stage = 0;
    for (int64_t first = r0; first < a.rows; first += step, r += step) {
        const bool in = r < a.rows;
        float mu_next = 0.f, rs_next = 0.f;
        if (r + step < a.rows) {
            if (!a.rms) mu_next = __ldg(a.mean + r + step);
            rs_next = __ldg(a.rstd + r + step);
        }
        P dyp[VPT], xp[VPT];
        if constexpr (kAsync) {
            copy_wait<AHEAD - 1>();
            issue(r + AHEAD * step, (stage + AHEAD) % kRing);  // the slot read one round ago
        }
#pragma unroll
        for (int k = 0; k < VPT; ++k) {
            const bool there = in && column(k) < a.width;
            if constexpr (kAsync) {
                const P* from = ring + (stage * 2 * VPT + k) * BLOCK + threadIdx.x;
                if (there) dyp[k] = from[0], xp[k] = from[VPT * BLOCK];
            } else {
                if (there) dyp[k].v[0] = a.dy[r * a.ds + column(k)], xp[k].v[0] = a.x[r * a.xs + column(k)];
            }
            if (!there) {
#pragma unroll
                for (int i = 0; i < N; ++i) dyp[k].v[i] = xp[k].v[i] = from_f32<T>(0.f);
            }
        }
        stage = stage + 1 == kRing ? 0 : stage + 1;
        // xhat and dy of pair p (columns past the width: dy and the weight are zero)
        auto pair = [&](const P* q, int p) {
            if constexpr (N == 1) {
                return make_float2(to_f32(q[2 * p].v[0]), to_f32(q[2 * p + 1].v[0]));
            } else {
                constexpr int H = N / 2;
                return make_float2(to_f32(q[p / H].v[2 * (p % H)]), to_f32(q[p / H].v[2 * (p % H) + 1]));
            }
        };
        float2 s2 = make_float2(0.f, 0.f), q2 = s2;
#pragma unroll
        for (int p = 0; p < kPairs; ++p) {
            const float2 g = pair(dyp, p);
            const float2 h = mul2(add2(pair(xp, p), both(-mu)), both(rs));
            const float2 wg = mul2(g, w[p]);
            s2 = add2(s2, wg);
            q2 = fma2(wg, h, q2);
            dw[p] = fma2(g, h, dw[p]);
            db[p] = add2(db[p], g);
        }
        const float2 total = sum(make_float2(s2.x + s2.y, q2.x + q2.y));
        const float2 s = both(a.rms ? 0.f : -(total.x / width)), q = both(-(total.y / width));
        if (in) {
            float out[VPT * N];
#pragma unroll
            for (int p = 0; p < kPairs; ++p) {
                const float2 wg = mul2(pair(dyp, p), w[p]);
                const float2 h = mul2(add2(pair(xp, p), both(-mu)), both(rs));
                const float2 d = mul2(fma2(h, q, add2(wg, s)), both(rs));
                out[2 * p] = d.x, out[2 * p + 1] = d.y;
            }
#pragma unroll
            for (int k = 0; k < VPT; ++k) {
                float v[N];
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = out[k * N + i];
                const int c = column(k);
                if (c < a.width) store_pack<T, N>(a.dx + r * a.os + c, v, a.width - c, a.vec_out);
            }
        }
        mu = mu_next, rs = rs_next;
    }
    // the block's sums over its rows
    float* part = a.part + int64_t(blockIdx.x) * 2 * a.width;
    if constexpr (kRowsAtOnce == 1) {
#pragma unroll
        for (int p = 0; p < kPairs; ++p)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int e = 2 * p + i, c = column(e / N) + e % N;
                if (c < a.width) {
                    part[c] = i ? dw[p].y : dw[p].x;
                    part[a.width + c] = i ? db[p].y : db[p].x;
                }
            }
    } else {
        constexpr int kCols = TPR * VPT * N;
        if constexpr (kAsync) copy_wait<0>();
        __syncthreads();  // the ring's last reads and copies are done
        float* acc = reinterpret_cast<float*>(smem);  // [rows at once][2][columns]
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
            for (int g = 0; g < kRowsAtOnce; ++g) v += acc[(2 * g + which) * kCols + c];
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
    if (c < width) {
        int p = warp;
        for (; p + 3 * kWarps < parts; p += 4 * kWarps) {
            float v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = __ldg(from + int64_t(p + u * kWarps) * 2 * width);
            s += (v[0] + v[1]) + (v[2] + v[3]);
        }
        for (; p < parts; p += kWarps) s += __ldg(from + int64_t(p) * 2 * width);
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

// Rows wider than 8192 columns: dx row by row, read again for the second
// phase, and the sums by strips of 32 columns in a pass of their own.
template <typename T>
__global__ void __launch_bounds__(1024) k_norm_dx_wide(const __grid_constant__ BwdArgs<T> a) {
    __shared__ float2 red[2 * 32];
    RowSum<1024, 1024> sum{red};
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
        const float mu = a.rms ? 0.f : a.mean[r], rs = a.rstd[r];
        float2 v = make_float2(0.f, 0.f);
        for (int c = threadIdx.x; c < a.width; c += 1024) {
            const float w = to_f32(a.dy[r * a.ds + c]) * load_param(a.weight, a.ptype, c);
            v.x += w;
            v.y = fmaf(w, (to_f32(a.x[r * a.xs + c]) - mu) * rs, v.y);
        }
        v = sum(v);
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

// launches the pass; returns the number of partial sums or a negative status
template <typename T, int N, int TPR, int BLOCK>
int launch(const BwdArgs<T>& a, cudaStream_t s) {
    constexpr int VPT = 16 / N, AHEAD = sizeof(T) == 4 ? 1 : 3;
    const void* kernel = reinterpret_cast<const void*>(k_norm_bwd<T, N, TPR, VPT, BLOCK, AHEAD>);
    size_t smem = RowSum<TPR, BLOCK>::kBytes +
                  (N * sizeof(T) >= 4 ? size_t(AHEAD + 1) * 2 * VPT * BLOCK * N * sizeof(T) : 0);
    if (TPR < BLOCK && smem < size_t(BLOCK) * 16 * 2 * sizeof(float)) smem = size_t(BLOCK) * 16 * 2 * sizeof(float);
    if (!allow_shared(kernel, smem)) return DL_ERR_CUDA;
    constexpr int at_once = BLOCK / TPR;
    int grid = grid_for(kernel, BLOCK, smem, (a.rows + at_once - 1) / at_once);
    if (grid > kMostBlocks) grid = kMostBlocks;
    k_norm_bwd<T, N, TPR, VPT, BLOCK, AHEAD><<<grid, BLOCK, smem, s>>>(a);
    const int st = launch_status();
    return st == DL_OK ? grid : st;
}

template <typename T, int N>
int by_width(const BwdArgs<T>& a, cudaStream_t s) {
    if (a.width <= 128) return launch<T, N, 8, 256>(a, s);
    if (a.width <= 512) return launch<T, N, 32, 256>(a, s);
    if (a.width <= 1024) return launch<T, N, 64, 256>(a, s);
    if (a.width <= 2048) return launch<T, N, 128, 256>(a, s);
    if (a.width <= 4096) return launch<T, N, 256, 256>(a, s);
    if (a.width <= 8192) return launch<T, N, 512, 512>(a, s);
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
                                      static_cast<T*>(dx), weight, mean, rstd, part, dy_stride,
                                      x_stride, dx_stride, rows, width, param_type, rms, false},
                           s);
    };
    int parts = 0;
    if (rows > 0)
        parts = x_type == DL_F32 ? call(float()) : x_type == DL_BF16 ? call(__nv_bfloat16()) : call(__half());
    if (parts < 0) return parts;
    k_norm_join<<<dim3((width + 31) / 32, dbias ? 2 : 1), kThreads, 0, s>>>(part, parts, width, param_type,
                                                                          accumulate, dweight, dbias);
    return launch_status();
}
