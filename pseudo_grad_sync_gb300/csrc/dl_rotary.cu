// Rotary positions: pairs of a head's elements turned by their token's position.
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "dl_norm.cuh"
#include "dl_rotary_form.h"

namespace dl {
namespace {

constexpr int kThreads = 256;

struct RotaryArgs {
    dl_rotary_job job[DL_ROTARY_MAX_JOBS];
    const uint64_t* turns;
    const void* positions;
    int64_t batch, tokens;
    int64_t position_batch, position_token;  // strides
    int64_t first, first_step;               // of the tokens where positions is NULL
    int64_t tiles_per_batch, tiles;
    float amplitude, direction;  // direction: -1 for the inverse
    int32_t n_jobs, head_dim, pairs, position_type;
    int32_t tile, side, lanes;  // tokens of a tile, tokens and heads of a token side by side
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
    if (!a.positions) return static_cast<uint64_t>(a.first) + static_cast<uint64_t>(token * a.first_step);
    const int64_t at = batch * a.position_batch + token * a.position_token;
    return static_cast<uint64_t>(a.position_type == DL_I64 ? static_cast<const int64_t*>(a.positions)[at]
                                                           : static_cast<const int32_t*>(a.positions)[at]);
}

// Two pairs turned: a product and a fused product each, in this order in every
// form of the kernel, so that they all give the same bits.
__device__ __forceinline__ void turn(float2& a, float2& b, float2 c, float2 s) {
    const float2 bs = mul2(b, s), as = mul2(a, s);
    a = fma2(a, c, make_float2(-bs.x, -bs.y));
    b = fma2(b, c, as);
}
__device__ __forceinline__ void turn(float& a, float& b, float c, float s) {
    const float first = fmaf(a, c, -__fmul_rn(b, s));
    b = fmaf(b, c, __fmul_rn(a, s));
    a = first;
}

// elements 2i and 2i + 1 of a pack
template <typename T, int N>
__device__ __forceinline__ void set_pair(Pack<T, N>& p, int i, float2 v) {
    if constexpr (sizeof(T) == 2) {
        reinterpret_cast<uint32_t*>(p.v)[i] = pack2(v, T());
    } else {
        p.v[2 * i] = v.x, p.v[2 * i + 1] = v.y;
    }
}

// A unit's pairs turned in place. Half layout: the pairs' first elements in v,
// the second ones in w; interleaved: the first `pairs` neighbours in v (packs of
// one: in v and w).
template <typename T, int N, bool INTERLEAVED, int PAIRS>
__device__ __forceinline__ void turn_unit(Pack<T, N>& v, Pack<T, N>& w, const float2 (&cs)[PAIRS], int pairs) {
    if constexpr (N == 1) {
        float a = to_f32(v.v[0]), b = to_f32(w.v[0]);
        turn(a, b, cs[0].x, cs[0].y);
        v.v[0] = from_f32<T>(a), w.v[0] = from_f32<T>(b);
    } else if constexpr (INTERLEAVED) {
#pragma unroll
        for (int i = 0; i < PAIRS; ++i) {
            if (i >= pairs) break;
            float2 e = pair_of(&v, i);
            turn(e.x, e.y, cs[i].x, cs[i].y);
            set_pair(v, i, e);
        }
    } else {
#pragma unroll
        for (int i = 0; i < PAIRS / 2; ++i) {
            float2 a = pair_of(&v, i), b = pair_of(&w, i);
            turn(a, b, make_float2(cs[2 * i].x, cs[2 * i + 1].x), make_float2(cs[2 * i].y, cs[2 * i + 1].y));
            set_pair(v, i, a);
            set_pair(w, i, b);
        }
    }
}

// A block takes a tile of consecutive tokens, all heads of all tensors. First
// its threads compute the tile's cosines and sines into shared memory, one per
// (token, pair), so that a token's heads share them. Then each thread keeps
// those of one unit of one token in registers and walks over the heads: a unit
// is a pack of N elements (half layout: with the pack of its pairs' partners),
// or packs behind the rotated part that are only copied.
//
// Bound by HBM (reads and writes mixed, 78% of its peak in the counters): 4 x 8192
// tokens of 32 + 8 heads of 128 bf16 106 us (93% of the copy rate), half of each
// head rotated 110, 4 x 4096 in fp32 103 (96%), interleaved 111. With the cosines
// read from shared memory for every head and an integer division per row it was
// 218 us; one head at a time per thread 118. The next heads' loads ahead of the
// cosines gained nothing on single tokens and cost the batch 8 us. Single tokens
// (5 x 36 heads of 64): 3.4 us. What is left: heads few or narrow (one query and
// one key head of 128: 23%), whose tokens share a cosine among two heads only, and
// packs below 16 bytes (heads of 75: 39-42%). The half layout in 16-bit packs of
// eight spills 20 bytes at the 80 registers that three blocks per SM leave.
template <typename T, int N, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads, 3) k_rotary(const __grid_constant__ RotaryArgs a) {
    extern __shared__ __align__(16) float2 table[];
    using P = Pack<T, N>;
    using F = Form<N, INTERLEAVED>;
    constexpr int kPairs = F::kPairs, kRows = 4;  // heads at a time
    const int turned = F::turned(a.pairs), units = F::units(a.head_dim, a.pairs);
    const int wide = min(units, kThreads);
    const int slot = threadIdx.x / wide, local = slot / a.lanes, head = slot - local * a.lanes;
    const int token0 = threadIdx.x / a.pairs, pair0 = threadIdx.x - token0 * a.pairs;
    const int more_tokens = kThreads / a.pairs, more_pairs = kThreads - more_tokens * a.pairs;
    const int first_unit = threadIdx.x % wide;
    for (int64_t tile = blockIdx.x; tile < a.tiles; tile += gridDim.x) {
        const int64_t batch = a.tiles_per_batch == 1 ? tile : a.batch == 1 ? 0 : tile / a.tiles_per_batch;
        const int64_t begin = (tile - batch * a.tiles_per_batch) * a.tile;
        const int count = static_cast<int>(min(static_cast<int64_t>(a.tile), a.tokens - begin));
        for (int i = threadIdx.x, token = token0, pair = pair0; i < count * a.pairs; i += kThreads) {
            const float2 cs = cos_sin(position_of(a, batch, begin + token), a.turns[pair]);
            table[i] = make_float2(cs.x * a.amplitude, cs.y * a.amplitude * a.direction);
            token += more_tokens, pair += more_pairs;
            if (pair >= a.pairs) pair -= a.pairs, ++token;
        }
        __syncthreads();
        // a token's units (one each but for the widest heads), then the next token
        for (int l = slot < a.side * a.lanes ? local : count, u = first_unit; l < count;
             u + wide < units ? u += wide : (u = first_unit, l += a.side)) {
            const bool turns = u < turned;
            const int pairs = a.pairs - u * kPairs;  // of the unit, where it has fewer than kPairs
            float2 cs[kPairs];
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                cs[i] = i < pairs ? table[l * a.pairs + u * kPairs + i] : make_float2(0.f, 0.f);
            const int low = F::first(u, turned);
            const int apart = turns && !INTERLEAVED ? a.pairs : N;  // between a unit's two packs
            const bool two = F::two(turns, low, a.head_dim);
            for (int j = 0; j < a.n_jobs; ++j) {
                const dl_rotary_job& job = a.job[j];
                if (!turns && job.x == job.y) continue;  // in place: nothing to copy
                const T* x = static_cast<const T*>(job.x) + batch * job.x_batch + (begin + l) * job.x_token + low;
                T* y = static_cast<T*>(job.y) + batch * job.y_batch + (begin + l) * job.y_token + low;
                for (HeadWalk<kRows> h(head, a.lanes, job.heads); h.more(); h.next()) {
                    P v[kRows], w[kRows];
#pragma unroll
                    for (int r = 0; r < kRows; ++r)
                        if (h.has(r)) {
                            const T* from = x + h.row(r) * job.x_head;
                            v[r] = *reinterpret_cast<const P*>(from);
                            if (two) w[r] = *reinterpret_cast<const P*>(from + apart);
                        }
#pragma unroll
                    for (int r = 0; r < kRows; ++r)
                        if (h.has(r)) {
                            T* to = y + h.row(r) * job.y_head;
                            if (turns) turn_unit<T, N, INTERLEAVED>(v[r], w[r], cs, pairs);
                            *reinterpret_cast<P*>(to) = v[r];
                            if (two) *reinterpret_cast<P*>(to + apart) = w[r];
                        }
                }
            }
        }
        // elements behind the last whole pack
        const int tail = F::rest(a.head_dim, a.pairs) % N;
        if (N > 1 && tail > 0)
            for (int j = 0; j < a.n_jobs; ++j) {
                const dl_rotary_job& job = a.job[j];
                if (job.x == job.y) continue;
                for (int64_t i = threadIdx.x; i < int64_t(count) * job.heads * tail; i += kThreads) {
                    const int64_t row = i / tail, token = begin + row / job.heads, h = row % job.heads;
                    const int64_t c = a.head_dim - tail + i % tail;
                    static_cast<T*>(job.y)[batch * job.y_batch + token * job.y_token + h * job.y_head + c] =
                        static_cast<const T*>(job.x)[batch * job.x_batch + token * job.x_token + h * job.x_head + c];
                }
            }
        __syncthreads();
    }
}

// How a block's threads are shared out: `wide` units of a head side by side,
// `lanes` heads, and as many tokens as that leaves room for. Tokens share the
// latency of a tile's cosines, heads need no more of them; where there are few
// tokens the heads spread over the threads instead.
template <typename T, int N, bool INTERLEAVED>
int launch(RotaryArgs a, cudaStream_t s) {
    const int units = Form<N, INTERLEAVED>::units(a.head_dim, a.pairs);
    const int slots = kThreads / (units < kThreads ? units : kThreads);
    int least = INT32_MAX, most = 1;
    for (int j = 0; j < a.n_jobs; ++j) {
        least = a.job[j].heads < least ? a.job[j].heads : least;
        most = a.job[j].heads > most ? a.job[j].heads : most;
    }
    int lanes = 1;
    auto blocks = [&](int tile) { return a.batch * ((a.tokens + tile - 1) / tile); };
    while (2 * lanes <= slots && (lanes * 8 <= least || (lanes * 2 <= least && blocks(slots / lanes) < 16 * sm_count())))
        lanes *= 2;
    while (2 * lanes <= slots && lanes < most && blocks(slots / lanes) < 4 * sm_count()) lanes *= 2;
    a.lanes = lanes, a.side = slots / lanes, a.tile = a.side;
    while (a.tile * a.pairs < 512 && blocks(2 * a.tile) >= 8 * sm_count()) a.tile *= 2;
    const int most_tokens = 4096 / a.pairs;  // 32 KB of cosines and sines
    if (a.tile > most_tokens) a.tile = most_tokens;
    if (a.tile > a.tokens) a.tile = static_cast<int>(a.tokens);
    a.tiles_per_batch = (a.tokens + a.tile - 1) / a.tile;
    a.tiles = a.tiles_per_batch * a.batch;
    const size_t bytes = size_t(a.tile) * a.pairs * sizeof(float2);
    const int64_t grid = limited(a.tiles < INT32_MAX ? a.tiles : INT32_MAX);
    k_rotary<T, N, INTERLEAVED><<<static_cast<unsigned>(grid), kThreads, bytes, s>>>(a);
    return launch_status();
}

// Packs as wide as every address, stride and the pairs allow: 16 bytes, or
// half of that, down to single elements.
template <typename T, int N>
int by_pack(const RotaryArgs& a, bool interleaved, cudaStream_t s) {
    bool fits = interleaved ? Form<N, true>::fits(a.head_dim, a.pairs) : Form<N, false>::fits(a.head_dim, a.pairs);
    for (int j = 0; j < a.n_jobs && fits; ++j) {
        const dl_rotary_job& q = a.job[j];
        fits = aligned_to(q.x, N * sizeof(T)) && aligned_to(q.y, N * sizeof(T)) &&
               (q.x_batch | q.x_token | q.x_head | q.y_batch | q.y_token | q.y_head) % N == 0;
    }
    if constexpr (N > 1) {
        if (!fits) return by_pack<T, N / 2>(a, interleaved, s);
    }
    return interleaved ? launch<T, N, true>(a, s) : launch<T, N, false>(a, s);
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
    a.batch = batch, a.tokens = tokens;
    a.position_batch = position_stride, a.position_token = 1;
    a.first = first, a.first_step = 1;
    a.amplitude = static_cast<float>(amplitude), a.direction = flags & DL_ROTARY_INVERSE ? -1.f : 1.f;
    a.head_dim = head_dim, a.pairs = rotary_dim / 2, a.position_type = position_type;
    if (tokens == 1) {  // single tokens of many sequences: one sequence of them
        a.tokens = batch, a.batch = 1;
        a.position_token = position_stride, a.first_step = 0;
        for (int32_t j = 0; j < a.n_jobs; ++j) {
            a.job[j].x_token = a.job[j].x_batch, a.job[j].y_token = a.job[j].y_batch;
            a.job[j].x_batch = a.job[j].y_batch = 0;
        }
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool interleaved = flags & DL_ROTARY_INTERLEAVED;
    switch (type) {
        case DL_F32: return by_pack<float, 4>(a, interleaved, s);
        case DL_BF16: return by_pack<__nv_bfloat16, 8>(a, interleaved, s);
        default: return by_pack<__half, 8>(a, interleaved, s);
    }
}
