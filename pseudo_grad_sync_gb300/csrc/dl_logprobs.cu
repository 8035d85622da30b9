// Token log probabilities, entropy and most probable alternatives of rows of logits.
#include <float.h>
#include <stdint.h>

#include "dl_logprobs.cuh"

namespace dl {
namespace {

constexpr unsigned kAll = 0xffffffffu;

template <typename T>
struct ForwardArgs {
    const T* logits;
    const void* tokens;
    float *logp, *entropy, *lse;
    int64_t* top_tokens;
    float* top_logp;
    float *row_max, *log_sum;
    int64_t stride, rows;
    int32_t vocab, token_type, n_top;
};

// A part of a row's softmax: its largest logit m, s = sum e^(z - m) and, in
// units of log 2, a = sum e^(z - m) (z - m). Nothing yet: m lowest and s zero,
// so that -inf - m is -inf and adds nothing.
struct Part {
    float m = -FLT_MAX, s = 0.f, a = 0.f;

    // to a larger maximum
    __device__ __forceinline__ void raise(float top) {
        const float t = max_nan((m - top) * kLog2E, kLeast), f = exp2_fast(t);
        a = fmaf(s, t, a) * f;
        s *= f;
        m = top;
    }
    __device__ __forceinline__ void add(Part o) {
        const float top = max_nan(m, o.m);
        raise(top);
        o.raise(top);
        s += o.s;
        a += o.a;
    }
};

template <typename T, int N>
__device__ __forceinline__ float largest(const Pack<T, N>& p) {
    if constexpr (sizeof(T) == 2) {
        using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
        const T2* q = reinterpret_cast<const T2*>(p.v);
        T2 r = q[0];
#pragma unroll
        for (int i = 1; i < N / 2; ++i) r = __hmax2_nan(r, q[i]);
        const float2 f = as_floats(*reinterpret_cast<const uint32_t*>(&r), T());
        return max_nan(f.x, f.y);
    } else {
        return max_nan(max_nan(p.v[0], p.v[1]), max_nan(p.v[2], p.v[3]));
    }
}

// Adds U packs: the maximum first, then every term relative to it.
template <bool ENTROPY, typename T, int N, int U>
__device__ __forceinline__ void add_packs(Part& part, const Pack<T, N> (&p)[U], float top) {
    part.raise(max_nan(part.m, top));
    float2 s = make_float2(0.f, 0.f), a = s;
    const float2 minus = both(-part.m), unit = both(kLog2E);
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            float2 t = mul2(add2(pair_at(p[u], i), minus), unit);
            if (ENTROPY) t = make_float2(max_nan(t.x, kLeast), max_nan(t.y, kLeast));
            const float2 e = make_float2(exp2_fast(t.x), exp2_fast(t.y));
            s = add2(s, e);
            if (ENTROPY) a = fma2(e, t, a);
        }
    part.s += s.x + s.y;
    part.a += a.x + a.y;
}

// Logits as keys: a larger key is a larger logit, of equal ones the lower
// column; 0 is none, and -inf is none.
__device__ __forceinline__ uint64_t key_of(float v, uint32_t column) {
    if (!(v > -INFINITY)) return 0;
    const uint32_t b = __float_as_uint(v + 0.f);  // one zero
    const uint32_t o = b & 0x80000000u ? ~b : b | 0x80000000u;
    return uint64_t(o) << 32 | (0xffffffffu - column);
}
__device__ __forceinline__ float logit_of(uint64_t key) {
    const uint32_t o = static_cast<uint32_t>(key >> 32);
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint32_t column_of(uint64_t key) { return 0xffffffffu - static_cast<uint32_t>(key); }

// A warp's 32 largest keys, one per lane, the largest in lane 0.
struct WarpTop {
    uint64_t key = 0;

    __device__ __forceinline__ void exchange(int lane, int j, bool descending) {
        const uint64_t o = __shfl_xor_sync(kAll, key, j);
        const bool first = (lane & j) == 0;
        key = (first == descending) == (key > o) ? key : o;
    }
    // any keys in any order (bitonic)
    __device__ __forceinline__ void sort(int lane) {
        for (int k = 2; k <= 32; k *= 2)
            for (int j = k / 2; j > 0; j /= 2) exchange(lane, j, (lane & k) == 0 || k == 32);
    }
    // the 32 largest of these and another list's, given in reverse order
    __device__ __forceinline__ void merge(int lane, uint64_t reversed) {
        key = key > reversed ? key : reversed;
        for (int j = 16; j > 0; j /= 2) exchange(lane, j, true);
    }
    // one more key, the same in every lane
    __device__ __forceinline__ void insert(int lane, uint64_t k) {
        const int place = __popc(__ballot_sync(kAll, key > k));
        const uint64_t before = __shfl_up_sync(kAll, key, 1);
        key = lane < place ? key : lane == place ? k : before;
    }
};

template <int WARPS>
struct Scratch {
    Part part[WARPS];
    uint64_t list[WARPS][32];
    uint64_t threshold;
    int chosen, threads[WARPS * 32];
};

// One block per row at a time. Every thread keeps the running maximum and sums
// of its packs; warps and then the block join them.
//
// Alternatives: each thread also remembers its best pack and that pack's
// largest logit. The n_top-th largest of the threads' best is a bound that no
// alternative lies below, and only n_top threads have an element that reaches
// it: their packs alone are read again, a warp per thread, and what reaches
// the bound goes into the warps' sorted lists, which are merged.
template <typename T, int BLOCK, bool ENTROPY, bool TOP>
__global__ void __launch_bounds__(BLOCK) k_logprobs(const __grid_constant__ ForwardArgs<T> a) {
    constexpr int N = 16 / sizeof(T), U = 4, kWarps = BLOCK / 32;
    __shared__ Scratch<TOP ? kWarps : 1> top;
    __shared__ Part parts[kWarps];
    const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    const T none = from_f32<T>(-INFINITY);
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const int64_t token = a.tokens ? token_at(a.tokens, a.token_type, row) : 0;
        if (token < 0) {
            if (threadIdx.x == 0) {
                a.logp[row] = 0.f;
                if (a.lse) a.lse[row] = 0.f;
                if (a.entropy) a.entropy[row] = 0.f;
                if (a.row_max) a.row_max[row] = 0.f, a.log_sum[row] = 0.f;
            }
            if (TOP && threadIdx.x < a.n_top) {
                a.top_tokens[row * a.n_top + threadIdx.x] = -1;
                a.top_logp[row * a.n_top + threadIdx.x] = -INFINITY;
            }
            continue;
        }
        const RowPacks<T> packs(a.logits + row * a.stride, a.vocab);
        Part part;
        float best = -INFINITY;
        int best_pack = -1;
        for (int64_t p = threadIdx.x; p < packs.packs; p += BLOCK * U) {
            Pack<T, N> q[U];
            float most = -INFINITY;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p + u * BLOCK < packs.packs) {
                    q[u] = packs.load(static_cast<int>(p + u * BLOCK), none);
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) q[u].v[i] = none;
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float m = largest(q[u]);
                if (TOP && m > best) best = m, best_pack = static_cast<int>(p + u * BLOCK);
                most = max_nan(most, m);
            }
            add_packs<ENTROPY>(part, q, most);
        }
#pragma unroll
        for (int j = 16; j > 0; j /= 2) {
            Part o;
            o.m = __shfl_xor_sync(kAll, part.m, j);
            o.s = __shfl_xor_sync(kAll, part.s, j);
            o.a = __shfl_xor_sync(kAll, part.a, j);
            part.add(o);
        }
        if (lane == 0) parts[warp] = part;
        uint64_t low = 0, high = 0;  // between these keys lies the thread's best
        if constexpr (TOP) {
            if (best_pack >= 0) {
                const int64_t first = int64_t(best_pack) * N - packs.skew;
                high = key_of(best, static_cast<uint32_t>(first < 0 ? 0 : first));
                low = key_of(best, static_cast<uint32_t>(min(first + N - 1, int64_t(a.vocab) - 1)));
            }
            WarpTop list{low};
            list.sort(lane);
            top.list[warp][lane] = list.key;
            if (threadIdx.x == 0) top.chosen = 0;
        }
        __syncthreads();
        part = parts[0];
        for (int w = 1; w < kWarps; ++w) part.add(parts[w]);
        WarpTop found;
        if constexpr (TOP) {
            if (warp == 0) {
                WarpTop list{top.list[0][lane]};
                for (int w = 1; w < kWarps; ++w) list.merge(lane, top.list[w][31 - lane]);
                const uint64_t bound = __shfl_sync(kAll, list.key, a.n_top - 1);
                if (lane == 0) top.threshold = bound;
            }
            __syncthreads();
            const uint64_t bound = top.threshold;
            if (high != 0 && high >= bound) top.threads[atomicAdd(&top.chosen, 1)] = threadIdx.x;
            __syncthreads();
            for (int c = warp; c < top.chosen; c += kWarps) {
                for (int64_t p = top.threads[c]; p < packs.packs; p += 32 * BLOCK) {
                    const int64_t mine = p + lane * BLOCK;
                    Pack<T, N> q;
#pragma unroll
                    for (int i = 0; i < N; ++i) q.v[i] = none;
                    if (mine < packs.packs) q = packs.load(static_cast<int>(mine), none);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const uint64_t k = key_of(to_f32(q.v[i]), static_cast<uint32_t>(mine * N + i - packs.skew));
                        unsigned who = __ballot_sync(kAll, k != 0 && k >= bound);
                        while (who) {
                            found.insert(lane, __shfl_sync(kAll, k, __ffs(who) - 1));
                            who &= who - 1;
                        }
                    }
                }
            }
            top.list[warp][lane] = found.key;  // the threshold's lists were read before the last barrier but one
            __syncthreads();
            if (warp == 0)
                for (int w = 1; w < kWarps; ++w) found.merge(lane, top.list[w][31 - lane]);
        }
        if (warp == 0) {
            // nothing but -inf: no sum; NaN or +inf: a sum of NaN
            const bool empty = part.s == 0.f, bad = !(part.s >= 0.f);
            const float m = bad ? NAN : empty ? 0.f : part.m, log_sum = logf(part.s);
            if (lane == 0) {
                if (a.tokens) {
                    float z = NAN;
                    if (token < a.vocab) z = to_f32(a.logits[row * a.stride + token]);
                    a.logp[row] = empty && token < a.vocab ? -INFINITY : (z - m) - log_sum;
                }
                if (a.lse) a.lse[row] = m + log_sum;
                if (a.entropy) a.entropy[row] = empty ? 0.f : log_sum - part.a / part.s * kLn2;
                if (a.row_max) a.row_max[row] = m, a.log_sum[row] = log_sum;
            }
            if (TOP && lane < a.n_top) {
                const bool have = found.key != 0 && !bad;
                a.top_tokens[row * a.n_top + lane] = have ? static_cast<int64_t>(column_of(found.key)) : -1;
                a.top_logp[row * a.n_top + lane] =
                    bad ? NAN : have ? (logit_of(found.key) - m) - log_sum : -INFINITY;
            }
        }
        __syncthreads();  // the next row writes the shared lists
    }
}

template <typename T, int BLOCK, bool ENTROPY, bool TOP>
int launch(const ForwardArgs<T>& a, cudaStream_t s) {
    static Resident resident;
    const int grid =
        resident.grid(reinterpret_cast<const void*>(k_logprobs<T, BLOCK, ENTROPY, TOP>), BLOCK, 0, a.rows);
    if (grid == 0) return DL_ERR_CUDA;
    k_logprobs<T, BLOCK, ENTROPY, TOP><<<grid, BLOCK, 0, s>>>(a);
    return launch_status();
}

template <typename T, int BLOCK>
int launch(const ForwardArgs<T>& a, cudaStream_t s) {
    if (a.entropy) return a.n_top ? launch<T, BLOCK, true, true>(a, s) : launch<T, BLOCK, true, false>(a, s);
    return a.n_top ? launch<T, BLOCK, false, true>(a, s) : launch<T, BLOCK, false, false>(a, s);
}

template <typename T>
int forward(const ForwardArgs<T>& a, cudaStream_t s) {
    return launch<T, 256>(a, s);
}

}  // namespace
}  // namespace dl

using namespace dl;

extern "C" int dl_logprobs_forward(const void* logits, int64_t stride, int32_t type, int64_t rows, int32_t vocab,
                                   const void* tokens, int32_t token_type, float* logp, float* entropy, float* lse,
                                   int32_t n_top, int64_t* top_tokens, float* top_logp, float* row_max,
                                   float* log_sum, void* stream) {
    if ((type != DL_F32 && type != DL_BF16 && type != DL_F16) || rows < 0 || vocab < 1 || stride < vocab ||
        (tokens && token_type != DL_I32 && token_type != DL_I64) || n_top < 0 || n_top > DL_LOGPROBS_MAX_TOP)
        return DL_ERR_ARG;
    if (rows == 0) return DL_OK;
    if (!logits || !tokens != !logp || !row_max != !log_sum || (n_top > 0 && (!top_tokens || !top_logp)))
        return DL_ERR_ARG;
    if (!aligned_to(logits, type_size(type)) || (tokens && !aligned_to(tokens, token_type == DL_I64 ? 8 : 4)) ||
        !aligned_to(logp, 4) || !aligned_to(entropy, 4) || !aligned_to(lse, 4) ||
        (n_top > 0 && (!aligned_to(top_tokens, 8) || !aligned_to(top_logp, 4))) || !aligned_to(row_max, 4) ||
        !aligned_to(log_sum, 4))
        return DL_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    auto call = [&](auto zero) {
        using T = decltype(zero);
        return forward<T>(ForwardArgs<T>{static_cast<const T*>(logits), tokens, logp, entropy, lse, top_tokens,
                                         top_logp, row_max, log_sum, stride, rows, vocab, token_type, n_top},
                          s);
    };
    return type == DL_F32 ? call(float()) : type == DL_BF16 ? call(__nv_bfloat16()) : call(__half());
}
