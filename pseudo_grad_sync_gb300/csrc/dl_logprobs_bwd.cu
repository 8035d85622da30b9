// The logits' gradient of token log probabilities, entropy and alternatives.
#include <stdint.h>

#include "dl_logprobs.cuh"

namespace dl {
namespace {

template <typename T>
struct BackwardArgs {
    const T* logits;
    T* out;
    const void* tokens;
    const float *row_max, *log_sum, *entropy, *d_logp, *d_entropy, *d_lse;
    const int64_t* top_tokens;
    const float* d_top;
    int64_t stride, out_stride, rows, items;
    int32_t vocab, token_type, n_top, chunks;
};

// dlogits[j] = e^(z_j - m) * (c0 + c1 * (z_j - m)) + what the tokens named in
// the row add; 1 / S is part of c0 and c1.
struct Row {
    float m, c0, c1;

    __device__ __forceinline__ float2 at(float2 z) const {
        const float2 d = add2(z, both(-m)), t = mul2(d, both(kLog2E));
        float2 c = both(c0);
        // a probability of 0 has no part in the entropy, however far below its logit is
        if (c1 != 0.f) c = fma2(make_float2(max_nan(d.x, kLeast), max_nan(d.y, kLeast)), both(c1), c);
        return mul2(make_float2(exp2_fast(t.x), exp2_fast(t.y)), c);
    }
};

// A block takes a chunk of a row: U packs per thread. Every logit's value is
// p_j times a polynomial of the row; the few columns named by the token and
// the alternatives get their own gradients on top, before the one rounding:
// the thread whose chunk has such a column computes it aside and stores it
// after its packs.
template <typename T, int N, int BLOCK, int U>
__global__ void __launch_bounds__(BLOCK) k_logprobs_bwd(const __grid_constant__ BackwardArgs<T> a) {
    __shared__ float aside[DL_LOGPROBS_MAX_TOP + 1];
    using P = Pack<T, N>;
    for (int64_t item = blockIdx.x; item < a.items; item += gridDim.x) {
        const int64_t row = item / a.chunks;
        const int chunk = static_cast<int>(item - row * a.chunks);
        const T* x = a.logits + row * a.stride;
        T* y = a.out + row * a.out_stride;
        const int64_t token = a.tokens ? token_at(a.tokens, a.token_type, row) : 0;
        const float g = a.d_logp ? a.d_logp[row] : 0.f, h = a.d_entropy ? a.d_entropy[row] : 0.f,
                    l = a.d_lse ? a.d_lse[row] : 0.f, log_sum = a.log_sum[row];
        float named = 0.f;
        bool any = g != 0.f || h != 0.f || l != 0.f;
        for (int i = 0; i < a.n_top; ++i) {
            const int64_t k = a.top_tokens[row * a.n_top + i];
            const float q = a.d_top[row * a.n_top + i];
            if (k >= 0 && k < a.vocab) {
                named += q;
                any = any || q != 0.f;
            }
        }
        const bool zero = token < 0 || log_sum == -INFINITY || !any;
        Row r;
        r.m = a.row_max[row];
        const float inverse = expf(-log_sum);
        r.c1 = -h * inverse;
        r.c0 = (l - g - named - (h != 0.f ? h * (a.entropy[row] - log_sum) : 0.f)) * inverse;
        if (g != 0.f && token >= a.vocab) r.c0 = NAN;

        const int64_t skew = N == 1 ? 0 : static_cast<int64_t>((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
        const int64_t end = skew + a.vocab, first = (int64_t(chunk) * U * BLOCK + threadIdx.x) * N;
        const T* xb = x - skew;
        T* yb = y - skew;
        // this thread's columns among the named ones (place: element from the boundary)
        auto mine = [&](int64_t column) {
            const int64_t pack = (column + skew) / N - int64_t(chunk) * U * BLOCK;
            return pack >= 0 && pack < U * BLOCK && pack % BLOCK == threadIdx.x;
        };
        auto name = [&](int i) { return i == 0 ? (a.d_logp ? token : -1) : a.top_tokens[row * a.n_top + i - 1]; };
        if (!zero)
            for (int i = 0; i <= a.n_top; ++i) {
                const int64_t k = name(i);
                if (k < 0 || k >= a.vocab || !mine(k)) continue;
                float more = 0.f;
                for (int j = 0; j <= a.n_top; ++j)
                    if (name(j) == k) more += j == 0 ? g : a.d_top[row * a.n_top + j - 1];
                aside[i] = r.at(both(to_f32(x[k]))).x + more;
            }
        P q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = first + int64_t(u) * BLOCK * N;
            if (zero) {
#pragma unroll
                for (int i = 0; i < N; ++i) q[u].v[i] = from_f32<T>(0.f);
            } else if (at >= skew && at + N <= end) {
                q[u] = *reinterpret_cast<const P*>(xb + at);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    q[u].v[i] = at + i >= skew && at + i < end ? xb[at + i] : from_f32<T>(0.f);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t at = first + int64_t(u) * BLOCK * N;
            if (!zero) {
                if constexpr (N == 1) {
                    q[u].v[0] = from_f32<T>(r.at(both(to_f32(q[u].v[0]))).x);
                } else {
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) {
                        const float2 v = r.at(pair_of(&q[u], i));
                        q[u].v[2 * i] = from_f32<T>(v.x), q[u].v[2 * i + 1] = from_f32<T>(v.y);
                    }
                }
            }
            if (at >= skew && at + N <= end) {
                *reinterpret_cast<P*>(yb + at) = q[u];
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (at + i >= skew && at + i < end) yb[at + i] = q[u].v[i];
            }
        }
        if (!zero)
            for (int i = 0; i <= a.n_top; ++i) {
                const int64_t k = name(i);
                if (k >= 0 && k < a.vocab && mine(k)) y[k] = from_f32<T>(aside[i]);
            }
        __syncthreads();  // the next item's threads write aside
    }
}

template <typename T, int N, int BLOCK, int U>
int launch(BackwardArgs<T> a, cudaStream_t s) {
    const int64_t per = int64_t(BLOCK) * U * N;
    a.chunks = static_cast<int32_t>((int64_t(a.vocab) + (N - 1) + per - 1) / per);
    if (a.rows > INT64_MAX / a.chunks) return DL_ERR_ARG;
    a.items = a.rows * a.chunks;
    k_logprobs_bwd<T, N, BLOCK, U><<<static_cast<unsigned>(a.items < INT32_MAX ? a.items : INT32_MAX), BLOCK, 0, s>>>(a);
    return launch_status();
}

template <typename T>
int backward(const BackwardArgs<T>& a, cudaStream_t s) {
    constexpr int N = 16 / sizeof(T);
    // packs need every row of dlogits to lie on its 16-byte boundary as its logits do
    const bool alike = (reinterpret_cast<uintptr_t>(a.logits) - reinterpret_cast<uintptr_t>(a.out)) % 16 == 0 &&
                       (a.rows == 1 || (a.stride - a.out_stride) % N == 0);
    return alike ? launch<T, N, 256, 8>(a, s) : launch<T, 1, 256, 8>(a, s);
}

}  // namespace
}  // namespace dl

using namespace dl;

extern "C" int dl_logprobs_backward(const void* logits, int64_t stride, int32_t type, int64_t rows, int32_t vocab,
                                    const void* tokens, int32_t token_type, const float* row_max,
                                    const float* log_sum, const float* entropy, const float* d_logp,
                                    const float* d_entropy, const float* d_lse, int32_t n_top,
                                    const int64_t* top_tokens, const float* d_top, void* dlogits,
                                    int64_t dlogits_stride, void* stream) {
    if ((type != DL_F32 && type != DL_BF16 && type != DL_F16) || rows < 0 || vocab < 1 || stride < vocab ||
        dlogits_stride < vocab || (tokens && token_type != DL_I32 && token_type != DL_I64) || n_top < 0 ||
        n_top > DL_LOGPROBS_MAX_TOP || (logits == dlogits && stride != dlogits_stride))
        return DL_ERR_ARG;
    if (rows == 0) return DL_OK;
    if (!logits || !dlogits || !row_max || !log_sum || (d_entropy && !entropy) || (d_logp && !tokens) ||
        (n_top > 0 && (!top_tokens || !d_top)))
        return DL_ERR_ARG;
    const size_t size = type_size(type);
    if (!aligned_to(logits, size) || !aligned_to(dlogits, size) ||
        (tokens && !aligned_to(tokens, token_type == DL_I64 ? 8 : 4)) || !aligned_to(row_max, 4) ||
        !aligned_to(log_sum, 4) || !aligned_to(entropy, 4) || !aligned_to(d_logp, 4) || !aligned_to(d_entropy, 4) ||
        !aligned_to(d_lse, 4) || (n_top > 0 && (!aligned_to(top_tokens, 8) || !aligned_to(d_top, 4))))
        return DL_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto call = [&](auto zero) {
        using T = decltype(zero);
        return backward<T>(BackwardArgs<T>{static_cast<const T*>(logits), static_cast<T*>(dlogits), tokens, row_max,
                                           log_sum, entropy, d_logp, d_entropy, d_lse, top_tokens, d_top, stride,
                                           dlogits_stride, rows, 0, vocab, token_type, n_top, 0},
                           s);
    };
    return type == DL_F32 ? call(float()) : type == DL_BF16 ? call(__nv_bfloat16()) : call(__half());
}
