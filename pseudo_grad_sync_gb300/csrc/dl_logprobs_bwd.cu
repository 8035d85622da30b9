// The logits' gradient of token log probabilities, entropy and alternatives.
#include <stdint.h>

#include "dl_logprobs.cuh"

namespace dl {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kThreads = 128;

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

// 16 bytes from `shift` elements on in two neighbouring packs
template <typename T, int N>
__device__ __forceinline__ Pack<T, N> shifted(const Pack<T, N>& p, const Pack<T, N>& q, int shift) {
    const uint32_t* a = reinterpret_cast<const uint32_t*>(p.v);
    const uint32_t* b = reinterpret_cast<const uint32_t*>(q.v);
    uint32_t w[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    const int bytes = shift * static_cast<int>(sizeof(T));
    if (bytes & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (bytes & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    if (bytes & 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(w[i], w[i + 1], 16);
    }
    Pack<T, N> r;
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<uint32_t*>(r.v)[i] = w[i];
    return r;
}

// A warp takes a chunk of a row: U packs per lane, cut where dlogits has its
// 16-byte boundaries. Logits that lie otherwise on theirs (SHIFT) are read as
// two packs each and shifted. Every logit's value is a factor of the row times
// its probability; the few columns named by the token and the alternatives
// get their own gradients on top, before the one rounding: a lane for each
// computes that value aside and stores it after the chunk's packs.
//
// Bound by HBM: each logit is read once and written once. 8192 x 128256 bf16 with
// entropy 617 us (100% of the copy rate), without 597; 16384 x 32000 308 (100%);
// 8192 x 32000 fp32 with entropy and 5 alternatives 310 (100%). Shifted: 8192 x 32003
// fp32 with both 341 us (91%), bf16 173 (89%; element by element 491). The shifted
// forms and the aligned ones with alternatives spill 20 to 64 bytes. Chunks of a
// warp need no barrier (a block's chunk with its token's column patched by the
// thread that owns it: 635 us, and 3983 us instead of 155 for 262144 x 512). Eight
// packs per lane (four: 753 us), blocks of 128 threads (256: 636); the edges go
// element by element because a select per pack between a whole and a partial load
// serialises the loads (1041 us).
template <typename T, bool TOP, bool SHIFT>
__global__ void __launch_bounds__(kThreads, TOP && !SHIFT ? 8 : 7) k_logprobs_bwd(const __grid_constant__ BackwardArgs<T> a) {
    constexpr int N = 16 / sizeof(T), U = 8;
    using P = Pack<T, N>;
    const int lane = threadIdx.x % 32;
    for (int64_t item = int64_t(blockIdx.x) * (kThreads / 32) + threadIdx.x / 32; item < a.items;
         item += int64_t(gridDim.x) * (kThreads / 32)) {
        const int64_t row = a.chunks == 1       ? item
                            : a.items >> 32 == 0 ? static_cast<uint32_t>(item) / static_cast<uint32_t>(a.chunks)
                                                 : item / a.chunks;
        const int chunk = static_cast<int>(item - row * a.chunks);
        const T* x = a.logits + row * a.stride;
        T* y = a.out + row * a.out_stride;
        const int64_t token = a.tokens ? token_at(a.tokens, a.token_type, row) : 0;
        const float g = a.d_logp ? a.d_logp[row] : 0.f, h = a.d_entropy ? a.d_entropy[row] : 0.f,
                    l = a.d_lse ? a.d_lse[row] : 0.f, log_sum = a.log_sum[row];
        Row r;
        r.m = a.row_max[row];
        // this lane's alternative
        int64_t mine = -1;
        float q = 0.f, named = 0.f;
        if constexpr (TOP) {
            if (lane < a.n_top) {
                mine = a.top_tokens[row * a.n_top + lane];
                if (mine >= 0 && mine < a.vocab)
                    q = a.d_top[row * a.n_top + lane];
                else
                    mine = -1;
            }
            named = q;
#pragma unroll
            for (int j = 16; j > 0; j /= 2) named += __shfl_xor_sync(kAll, named, j);
        }
        const bool any = g != 0.f || h != 0.f || l != 0.f || (TOP && __any_sync(kAll, q != 0.f));
        const bool zero = token < 0 || log_sum == -INFINITY || !any;
        const float inverse = expf(-log_sum);
        r.c1 = -h * inverse;
        r.c0 = (l - g - named - (h != 0.f ? h * (a.entropy[row] - log_sum) : 0.f)) * inverse;
        if (g != 0.f && token >= a.vocab) r.c0 = NAN;

        const RowPacks<T> out(y, a.vocab);
        const int first = chunk * U * 32;
        // [low, high): packs read and written whole. What is before and behind them, up to
        // 2 N columns, is done element by element, a lane for each, by the row's first and last chunk.
        P v[U];
        const RowPacks<T> in(x, a.vocab);
        int low = out.skew > 0, high = static_cast<int>(out.end / N);
        if constexpr (SHIFT) {
            // column p * N - out.skew is element p * N + in.skew - out.skew from x's boundary: the
            // packs from there on, of which each lane reads one and takes the next from its neighbour
            const int shift = in.skew - out.skew, back = shift < 0;
            // packs that lie between the logits' first and last place
            const int begin = in.base < a.logits;
            const int end = in.packs - (in.base + int64_t(in.packs) * N > a.logits + (a.rows - 1) * a.stride + a.vocab);
            low = max(low, begin + back), high = min(high, end - 1 + back);
            P w[U + 1];
#pragma unroll
            for (int u = 0; u <= U; ++u) {
                w[u] = filled<T, N>(0);
                const int p = first - back + lane + u * 32;
                if (p >= begin && p < (zero ? 0 : end) && (u < U || lane == 0))
                    w[u] = reinterpret_cast<const P*>(in.base)[p];
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                P next;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t give = lane == 0 ? reinterpret_cast<const uint32_t*>(w[u + 1].v)[i]
                                                    : reinterpret_cast<const uint32_t*>(w[u].v)[i];
                    reinterpret_cast<uint32_t*>(next.v)[i] = __shfl_sync(kAll, give, (lane + 1) % 32);
                }
                v[u] = shifted(w[u], next, shift + back * N);
            }
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                v[u] = filled<T, N>(0);
                const int p = first + u * 32 + lane;
                if (p >= low && p < (zero ? 0 : high)) v[u] = reinterpret_cast<const P*>(in.base)[p];
            }
        }
        int64_t edge = -1;  // this lane's column of those
        if (lane < 16) {
            if (chunk == 0 && lane < low * N - out.skew) edge = lane;
        } else if (chunk == a.chunks - 1) {
            edge = int64_t(max(low, high)) * N - out.skew + lane - 16;  // behind the last of them
        }
        if (edge >= a.vocab) edge = -1;
        const float at_edge = edge >= 0 && !zero ? to_f32(x[edge]) : 0.f;
        // a named column is its pack's chunk's; behind the last whole pack the last chunk's, as its edge is
        const int64_t behind = int64_t(max(low, high)) * N - out.skew;
        auto within = [&](int64_t column) {
            if (column < 0 || column >= a.vocab) return false;
            if (column >= behind) return chunk == a.chunks - 1;
            const int64_t pack = (column + out.skew) / N - first;
            return pack >= 0 && pack < U * 32;
        };
        const bool has_token = !zero && a.d_logp && within(token), has_top = TOP && !zero && within(mine);
        float at_token = 0.f, at_top = 0.f;
        if (has_token) {  // in every lane alike
            float more = g;
            if constexpr (TOP) {
                float same = mine == token ? q : 0.f;
#pragma unroll
                for (int j = 16; j > 0; j /= 2) same += __shfl_xor_sync(kAll, same, j);
                more += same;
            }
            at_token = r.at(both(to_f32(x[token]))).x + more;
        }
        if (TOP && __any_sync(kAll, has_top)) {
            float more = a.d_logp && mine == token ? g : 0.f;
            for (int i = 0; i < a.n_top; ++i) {
                const int64_t other = __shfl_sync(kAll, mine, i);
                const float its = __shfl_sync(kAll, q, i);
                if (other == mine) more += its;
            }
            if (has_top) at_top = r.at(both(to_f32(x[mine]))).x + more;
        }
        if (a.logits == a.out) __syncwarp();  // named logits are read before their packs are written

        if (!zero) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (first + u * 32 >= high) break;  // a short row
                float2 f[N / 2];
#pragma unroll
                for (int i = 0; i < N / 2; ++i) f[i] = r.at(pair_of(&v[u], i));
                v[u] = pack_of<T, N>(f);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int p = first + u * 32 + lane;
            if (p >= low && p < high) reinterpret_cast<P*>(y - out.skew)[p] = v[u];
        }
        if (edge >= 0) y[edge] = from_f32<T>(zero ? 0.f : r.at(both(at_edge)).x);
        if (has_token || (TOP && __any_sync(kAll, has_top))) {
            __syncwarp();
            if (has_top && !(has_token && mine == token)) y[mine] = from_f32<T>(at_top);
            if (has_token && lane == 0) y[token] = from_f32<T>(at_token);
        }
    }
}

template <typename T, bool TOP, bool SHIFT>
int launch(BackwardArgs<T> a, cudaStream_t s) {
    constexpr int N = 16 / sizeof(T), kPer = 32 * 8;
    a.chunks = static_cast<int32_t>(((int64_t(a.vocab) + 2 * N - 2) / N + kPer - 1) / kPer);
    if (a.rows > INT64_MAX / a.chunks) return DL_ERR_ARG;
    a.items = a.rows * a.chunks;
    const int64_t blocks = (a.items + kThreads / 32 - 1) / (kThreads / 32);
    const int64_t grid = limited(blocks < INT32_MAX ? blocks : INT32_MAX);
    k_logprobs_bwd<T, TOP, SHIFT><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a);
    return launch_status();
}

template <typename T>
int backward(const BackwardArgs<T>& a, cudaStream_t s) {
    constexpr int N = 16 / sizeof(T);
    // every row of dlogits lies on its 16-byte boundary as its logits do
    const bool alike = (reinterpret_cast<uintptr_t>(a.logits) - reinterpret_cast<uintptr_t>(a.out)) % 16 == 0 &&
                       (a.rows == 1 || (a.stride - a.out_stride) % N == 0);
    if (a.n_top) return alike ? launch<T, true, false>(a, s) : launch<T, true, true>(a, s);
    return alike ? launch<T, false, false>(a, s) : launch<T, false, true>(a, s);
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
