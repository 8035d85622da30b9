// Rotary positions: pairs of a head's elements turned by their token's position.
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "dl_types.cuh"

namespace dl {
namespace {

constexpr int kThreads = 256;

struct RotaryArgs {
    dl_rotary_job job[DL_ROTARY_MAX_JOBS];
    const uint64_t* turns;
    const void* positions;
    int64_t tokens, total;  // tokens of a batch and of all
    int64_t position_stride, first, tiles;
    float amplitude, direction;  // direction: -1 for the inverse
    int32_t n_jobs, head_dim, pairs, position_type, tile;
};

// cos and sin of position * turns / 2^64 turns. The product wraps to the exact
// fraction of a turn; its nearest quarter turn comes off in integers, and what
// is left (at most an eighth, 31 bits) rounds once on its way to fp32.
__device__ __forceinline__ float2 cos_sin(uint64_t position, uint64_t turns) {
    const uint64_t shifted = position * turns + (1ull << 61);
    const int quarter = static_cast<int>(shifted >> 62);
    const int64_t rest = static_cast<int64_t>(shifted & ((1ull << 62) - 1)) - (1ll << 61);
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(rest >> 31)) * 0x1p-32f, &s, &c);
    if (quarter & 1) {
        const float t = c;
        c = -s, s = t;
    }
    return quarter & 2 ? make_float2(-c, -s) : make_float2(c, s);
}

__device__ __forceinline__ uint64_t position_of(const RotaryArgs& a, int64_t batch, int64_t token) {
    if (!a.positions) return static_cast<uint64_t>(a.first) + static_cast<uint64_t>(token);
    const int64_t at = batch * a.position_stride + token;
    return static_cast<uint64_t>(a.position_type == DL_I64 ? static_cast<const int64_t*>(a.positions)[at]
                                                           : static_cast<const int32_t*>(a.positions)[at]);
}

// (a, b) turned: a product and a fused product each, so that every form of the
// kernel gives the same bits.
__device__ __forceinline__ void turn(float& a, float& b, float2 cs) {
    const float first = fmaf(a, cs.x, -__fmul_rn(b, cs.y));
    b = fmaf(b, cs.x, __fmul_rn(a, cs.y));
    a = first;
}

// A block takes a tile of consecutive tokens, all heads of all tensors. First
// its threads compute the tile's cosines and sines into shared memory, one per
// (token, pair), so that a token's heads share them; then they walk over the
// (token, head) rows, each thread on a fixed unit of the row: a pack of N
// elements (half layout: the pack of its pairs' partners beside it), or a pack
// behind the rotated part that is only copied.
template <typename T, int N, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) k_rotary(const __grid_constant__ RotaryArgs a) {
    extern __shared__ __align__(16) float2 table[];
    using P = Pack<T, N>;
    constexpr int kPairs = INTERLEAVED && N > 1 ? N / 2 : N;  // of a unit
    const int turned = a.pairs / kPairs, rotated = 2 * a.pairs;
    const int units = turned + (a.head_dim - rotated + N - 1) / N;
    const int wide = min(units, kThreads), slots = kThreads / wide, slot = threadIdx.x / wide;
    for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const int64_t begin = tile * a.tile;
        const int count = static_cast<int>(min(static_cast<int64_t>(a.tile), a.total - begin));
        for (int i = threadIdx.x; i < count * a.pairs; i += kThreads) {
            const int64_t at = begin + i / a.pairs, batch = at / a.tokens;
            float2 cs = cos_sin(position_of(a, batch, at - batch * a.tokens), a.turns[i % a.pairs]);
            table[i] = make_float2(cs.x * a.amplitude, cs.y * a.amplitude * a.direction);
        }
        __syncthreads();
        for (int j = 0; j < a.n_jobs; ++j) {
            const dl_rotary_job& job = a.job[j];
            const bool in_place = job.x == job.y;
            if (slot >= slots) continue;
            for (int64_t row = slot; row < int64_t(count) * job.heads; row += slots) {
                const int64_t local = row / job.heads, head = row - local * job.heads;
                const int64_t at = begin + local, batch = at / a.tokens, token = at - batch * a.tokens;
                const T* x = static_cast<const T*>(job.x) + batch * job.x_batch + token * job.x_token + head * job.x_head;
                T* y = static_cast<T*>(job.y) + batch * job.y_batch + token * job.y_token + head * job.y_head;
                for (int u = threadIdx.x % wide; u < units; u += wide) {
                    if (u >= turned) {
                        if (in_place) continue;
                        const int c = rotated + (u - turned) * N;
                        if (c + N <= a.head_dim) {
                            *reinterpret_cast<P*>(y + c) = *reinterpret_cast<const P*>(x + c);
                        } else {
                            for (int i = c; i < a.head_dim; ++i) y[i] = x[i];
                        }
                        continue;
                    }
                    const float2* cs = table + local * a.pairs + u * kPairs;
                    if constexpr (INTERLEAVED && N > 1) {
                        P v = *reinterpret_cast<const P*>(x + u * N);
#pragma unroll
                        for (int i = 0; i < kPairs; ++i) {
                            float p = to_f32(v.v[2 * i]), q = to_f32(v.v[2 * i + 1]);
                            turn(p, q, cs[i]);
                            v.v[2 * i] = from_f32<T>(p), v.v[2 * i + 1] = from_f32<T>(q);
                        }
                        *reinterpret_cast<P*>(y + u * N) = v;
                    } else {
                        const int low = INTERLEAVED ? 2 * u : u * N, high = INTERLEAVED ? 2 * u + 1 : a.pairs + u * N;
                        P v = *reinterpret_cast<const P*>(x + low), w = *reinterpret_cast<const P*>(x + high);
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            float p = to_f32(v.v[i]), q = to_f32(w.v[i]);
                            turn(p, q, cs[i]);
                            v.v[i] = from_f32<T>(p), w.v[i] = from_f32<T>(q);
                        }
                        *reinterpret_cast<P*>(y + low) = v;
                        *reinterpret_cast<P*>(y + high) = w;
                    }
                }
            }
        }
        __syncthreads();
    }
}

template <typename T, int N, bool INTERLEAVED>
int launch(RotaryArgs a, cudaStream_t s) {
    const size_t bytes = size_t(a.tile) * a.pairs * sizeof(float2);
    const int64_t most = INT32_MAX;
    k_rotary<T, N, INTERLEAVED><<<static_cast<unsigned>(a.tiles < most ? a.tiles : most), kThreads, bytes, s>>>(a);
    return launch_status();
}

template <typename T>
int apply(const RotaryArgs& a, bool interleaved, cudaStream_t s) {
    constexpr int N = 16 / sizeof(T);
    // whole packs: of pairs' first elements beside packs of their second ones
    // (half layout), or of neighbouring pairs
    bool packs = (interleaved ? 2 * a.pairs : a.pairs) % N == 0;
    for (int j = 0; j < a.n_jobs && packs; ++j) {
        const dl_rotary_job& q = a.job[j];
        packs = aligned16(q.x) && aligned16(q.y) &&
                (q.x_batch | q.x_token | q.x_head | q.y_batch | q.y_token | q.y_head) % N == 0;
    }
    if (interleaved) return packs ? launch<T, N, true>(a, s) : launch<T, 1, true>(a, s);
    return packs ? launch<T, N, false>(a, s) : launch<T, 1, false>(a, s);
}

// Whether [n0][n1][n2][width] at these strides has every element at a place of
// its own: each dimension steps past what the ones of smaller strides cover.
bool apart(int64_t n0, int64_t s0, int64_t n1, int64_t s1, int64_t n2, int64_t s2, int64_t width) {
    int64_t n[3] = {n0, n1, n2}, s[3] = {s0, s1, s2};
    for (int i = 0; i < 2; ++i)
        for (int j = 0; j < 2 - i; ++j)
            if (s[j] > s[j + 1]) {
                const int64_t sn = n[j], ss = s[j];
                n[j] = n[j + 1], s[j] = s[j + 1], n[j + 1] = sn, s[j + 1] = ss;
            }
    int64_t covered = width;
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) continue;
        if (s[i] < covered || s[i] > (INT64_MAX - covered) / (n[i] - 1)) return false;
        covered += s[i] * (n[i] - 1);
    }
    return true;
}

}  // namespace
}  // namespace dl

using namespace dl;

extern "C" int dl_rotary_frequencies(int32_t dim, double base, int32_t scaling, double factor, double context,
                                     double low, double high, uint64_t* turns) {
    const double kTau = 6.283185307179586476925287;
    if (dim < 2 || dim % 2 || dim > DL_ROTARY_MAX_DIM || !(base >= 1.0 && base <= DBL_MAX) || !turns ||
        scaling < DL_ROTARY_PLAIN || scaling > DL_ROTARY_PARTS)
        return DL_ERR_ARG;
    if (scaling != DL_ROTARY_PLAIN && !(factor >= 1.0 && factor <= DBL_MAX)) return DL_ERR_ARG;
    if (scaling == DL_ROTARY_BASE) {
        if (dim == 2) return DL_ERR_ARG;
        base *= pow(factor, static_cast<double>(dim) / (dim - 2));
        if (!(base <= DBL_MAX)) return DL_ERR_ARG;
    }
    if (scaling == DL_ROTARY_PARTS && !(context > 0.0 && context <= DBL_MAX && low >= 0.0 && high > low && high <= DBL_MAX))
        return DL_ERR_ARG;
    for (int32_t i = 0; i < dim / 2; ++i) {
        double f = pow(base, -2.0 * i / dim);
        if (scaling == DL_ROTARY_LINEAR) f /= factor;
        if (scaling == DL_ROTARY_PARTS) {
            const double keep = fmin(1.0, fmax(0.0, (context * f / kTau - low) / (high - low)));
            f = f * keep + (1.0 - keep) * f / factor;
        }
        turns[i] = static_cast<uint64_t>(rint(f / kTau * 0x1p64));
    }
    return DL_OK;
}

extern "C" int dl_rotary_apply(const dl_rotary_job* jobs, int32_t n_jobs, int32_t type, int64_t batch,
                               int64_t tokens, int32_t head_dim, int32_t rotary_dim, const uint64_t* d_turns,
                               double amplitude, const void* positions, int32_t position_type,
                               int64_t position_stride, int64_t first, int32_t flags, void* stream) {
    if (!jobs || n_jobs < 1 || n_jobs > DL_ROTARY_MAX_JOBS ||
        (type != DL_F32 && type != DL_BF16 && type != DL_F16) || batch < 0 || tokens < 0 || head_dim < 2 ||
        rotary_dim < 2 || rotary_dim % 2 || rotary_dim > head_dim || rotary_dim > DL_ROTARY_MAX_DIM ||
        !(fabs(amplitude) <= FLT_MAX) || (flags & ~(DL_ROTARY_INTERLEAVED | DL_ROTARY_INVERSE)) ||
        (positions && ((position_type != DL_I32 && position_type != DL_I64) || position_stride < 0)))
        return DL_ERR_ARG;
    for (int32_t j = 0; j < n_jobs; ++j)
        if (jobs[j].heads < 0) return DL_ERR_ARG;
    if (batch == 0 || tokens == 0) return DL_OK;
    if (batch > INT64_MAX / tokens) return DL_ERR_ARG;
    RotaryArgs a = {};
    const size_t size = type_size(type);
    bool aligned = aligned_to(d_turns, 8) && aligned_to(positions, position_type == DL_I64 ? 8 : 4);
    for (int32_t j = 0; j < n_jobs; ++j) {
        const dl_rotary_job& q = jobs[j];
        if (q.heads == 0) continue;
        if (!q.x || !q.y || (q.x_batch | q.x_token | q.x_head | q.y_batch | q.y_token | q.y_head) < 0 ||
            (q.x == q.y && (q.x_batch != q.y_batch || q.x_token != q.y_token || q.x_head != q.y_head)) ||
            !apart(batch, q.y_batch, tokens, q.y_token, q.heads, q.y_head, head_dim))
            return DL_ERR_ARG;
        for (int32_t i = 0; i < n_jobs; ++i)  // in place or apart, never another tensor's
            if (i != j && jobs[i].heads > 0 && (q.y == jobs[i].y || q.y == jobs[i].x)) return DL_ERR_ARG;
        aligned = aligned && aligned_to(q.x, size) && aligned_to(q.y, size);
        a.job[a.n_jobs++] = q;
    }
    if (a.n_jobs == 0) return DL_OK;
    if (!d_turns) return DL_ERR_ARG;
    if (!aligned) return DL_ERR_ALIGN;
    a.turns = d_turns, a.positions = positions;
    a.tokens = tokens, a.total = batch * tokens;
    a.position_stride = position_stride, a.first = first;
    a.amplitude = static_cast<float>(amplitude), a.direction = flags & DL_ROTARY_INVERSE ? -1.f : 1.f;
    a.head_dim = head_dim, a.pairs = rotary_dim / 2, a.position_type = position_type;
    a.tile = 1;
    a.tiles = (a.total + a.tile - 1) / a.tile;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool interleaved = flags & DL_ROTARY_INTERLEAVED;
    switch (type) {
        case DL_F32: return apply<float>(a, interleaved, s);
        case DL_BF16: return apply<__nv_bfloat16>(a, interleaved, s);
        default: return apply<__half>(a, interleaved, s);
    }
}
