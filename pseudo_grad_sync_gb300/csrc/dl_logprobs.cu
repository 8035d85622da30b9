// Token log probabilities, entropy and most probable alternatives of rows of logits.
#include <float.h>
#include <stdint.h>

#include <type_traits>

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
    float m, s, a;

    static __device__ __forceinline__ Part nothing() { return {-FLT_MAX, 0.f, 0.f}; }
    // to a larger maximum
    __device__ __forceinline__ void raise(float top) {
        const float t = max_nan((m - top) * kLog2E, kLeast), f = exp2_fast(t);
        a = fmaf(s, t, a) * f;
        s *= f;
        m = top;
    }
};

template <typename T, int N, int U>
__device__ __forceinline__ float largest(const Pack<T, N> (&p)[U]) {
    if constexpr (sizeof(T) == 2) {
        using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
        T2 r = reinterpret_cast<const T2*>(p[0].v)[0];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = u == 0; i < N / 2; ++i) r = __hmax2_nan(r, reinterpret_cast<const T2*>(p[u].v)[i]);
        const float2 f = unpack2(*reinterpret_cast<const uint32_t*>(&r), T());
        return max_nan(f.x, f.y);
    } else {
        float r = p[0].v[0];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = u == 0; i < N; ++i) r = max_nan(r, p[u].v[i]);
        return r;
    }
}

// Adds U packs: the maximum first, then every term relative to it. A term
// that is 0 because its logit is -inf makes the entropy's sum NaN; that sum is
// then taken again with exponents kept finite, which costs the packs with
// masked logits a second pass and the others nothing.
//
// Where there are enough of them the exponents are one fused product each,
// x * log2(e) + c with c = -m * log2(e) as rounded: all are off by the same
// `off`, which the fused m * log2(e) + c gives exactly and the sums are
// corrected by (16384 x 32000 bf16 with entropy and 5 alternatives 213 us,
// 224 without). The largest term is then the product of two approximate powers,
// 1 to about 2^-21 only. Not for maxima so large that it is no small number.
template <bool ENTROPY, typename T, int N, int U>
__device__ __forceinline__ void add_packs(Part& part, const Pack<T, N> (&p)[U], float top) {
    part.raise(max_nan(part.m, top));
    float2 s = make_float2(0.f, 0.f), a = s;
    const float2 unit = both(kLog2E);
    if (N * U >= 32 && fabsf(part.m) < 0x1p20f) {
        const float c = -(part.m * kLog2E), off = fmaf(part.m, kLog2E, c), back = exp2_fast(-off);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float2 t = fma2(pair_of(&p[u], i), unit, both(c));
                const float2 e = make_float2(exp2_fast(t.x), exp2_fast(t.y));
                s = add2(s, e);
                if (ENTROPY) a = fma2(e, t, a);
            }
        s.x = (s.x + s.y) * back, s.y = 0.f;
        a.x = fmaf(a.x + a.y, back, -off * s.x), a.y = 0.f;
    } else {
        const float2 minus = both(-part.m);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int i = 0; i < N / 2; ++i) {
                const float2 t = mul2(add2(pair_of(&p[u], i), minus), unit);
                const float2 e = make_float2(exp2_fast(t.x), exp2_fast(t.y));
                s = add2(s, e);
                if (ENTROPY) a = fma2(e, t, a);
            }
    }
    float sum = a.x + a.y;
    if (ENTROPY && !(sum == sum)) {
        sum = 0.f;
        for (int u = 0; u < U; ++u)
            for (int i = 0; i < N; ++i) {
                const float t = max_nan((to_f32(p[u].v[i]) - part.m) * kLog2E, kLeast);
                sum = fmaf(exp2_fast(t), t, sum);
            }
    }
    part.s += s.x + s.y;
    part.a += sum;
}

// the parts of a warp's lanes, joined in every lane
__device__ __forceinline__ void join(Part& part) {
    float top = part.m;
#pragma unroll
    for (int j = 16; j > 0; j /= 2) top = max_nan(top, __shfl_xor_sync(kAll, top, j));
    part.raise(top);
#pragma unroll
    for (int j = 16; j > 0; j /= 2) {
        part.s += __shfl_xor_sync(kAll, part.s, j);
        part.a += __shfl_xor_sync(kAll, part.a, j);
    }
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

// Lists of 32 values, one per lane, the largest in lane 0.
template <typename K>
__device__ __forceinline__ K exchange(K key, int lane, int j, bool descending) {
    const K o = __shfl_xor_sync(kAll, key, j);
    return (((lane & j) == 0) == descending) == (key > o) ? key : o;
}
// L lists of values in any order, each sorted (bitonic)
template <int L, typename K>
__device__ __forceinline__ void sort_lists(K (&key)[L], int lane) {
#pragma unroll
    for (int k = 2; k <= 32; k *= 2)
#pragma unroll
        for (int j = k / 2; j > 0; j /= 2)
#pragma unroll
            for (int l = 0; l < L; ++l) key[l] = exchange(key[l], lane, j, (lane & k) == 0 || k == 32);
}
// the 32 largest of two lists, the second in reverse order
template <typename K>
__device__ __forceinline__ K merge_lists(K key, K reversed, int lane) {
    key = key > reversed ? key : reversed;
#pragma unroll
    for (int j = 16; j > 0; j /= 2) key = exchange(key, lane, j, true);
    return key;
}

// A row, or a block's share of one: packs [begin, end), in stages of U packs
// per thread. [low, high) of them lie between the logits' first and last place
// and are copied whole; one that holds a row's edge is masked.
template <typename T, int TPR, int U>
struct Share {
    RowPacks<T> packs;
    int begin, end, low, high, stages;

    __device__ __forceinline__ Share(const T* row, int vocab, int rank, int ranks, const T* from, const T* to)
        : packs(row, vocab) {
        const int each = (packs.packs + ranks - 1) / ranks;
        begin = min(rank * each, packs.packs);
        end = min(begin + each, packs.packs);
        low = max(begin, packs.base < from ? 1 : 0);
        // no less than low: one pack may hold both of the logits' ends
        high = max(low, min(end, packs.packs - (packs.base + int64_t(packs.packs) * packs.N > to ? 1 : 0)));
        stages = max((end - begin + TPR * U - 1) / (TPR * U), 1);
    }
};

constexpr int kCandidates = 64;

// Slots of a thread's share: the largest logit of each stage, or of as many
// consecutive ones as make the slots suffice.
template <typename T, int WARPS>
constexpr int kSlots = sizeof(T) == 4 && WARPS > 1 ? 8 : 16;

// What a block's warps hand over at a row's end, in turns: the last warp
// works on one row's while the others fill in the next one's.
template <typename T, int WARPS>
struct alignas(16) Handover {
    Part part[WARPS];
    float best[WARPS][32];
    T most[kSlots<T, WARPS>][WARPS * 32];
};
// The finishing warp's own: the packs it reads again, the threads and slots
// that had them, candidates, and a cluster's exchange.
template <int WARPS>
struct alignas(16) Finish {
    static constexpr int kRead = 4, kPlaces = 128;
    uint4 again[kRead][32];
    uint64_t candidate[kCandidates + 32 * 8];
    uint64_t key[32];
    Part part;
    int thread[WARPS * 32], place[kPlaces + 32];
    int waiting;
};

template <typename T, int TPR, int UNROLL>
struct Geometry {
    static constexpr int kWarps = TPR / 32;  // of a row
    static constexpr bool kAlone = kWarps == 1;
    static constexpr int kMain = kAlone ? 128 : TPR, kBlock = kAlone ? kMain : kMain + 32, kGroups = kMain / TPR;
    static constexpr int U = UNROLL, kStages = !kAlone ? 3 : U == 2 ? 6 : 4, kHands = kAlone ? 1 : 2;
    static constexpr size_t kRing = size_t(kStages) * U * kMain * 16;
    static constexpr size_t kHand = sizeof(Handover<T, kWarps>), kFinish = sizeof(Finish<kWarps>);
    static_assert(kHand % 16 == 0 && kFinish % 16 == 0, "");
    // a row's ring comes first, its handovers next
    static constexpr size_t bytes(bool top) {
        return kRing + (top ? kGroups * (kHands * kHand + kFinish) : kGroups * kHands * (kWarps + 1) * sizeof(Part));
    }
};

// The n_top largest logits of a row (or a share) from the largest one of every
// thread and slot, by one warp; lane i gets the i-th key, 0 past the finite logits.
//
// The n_top-th largest of the threads' maxima is a bound that no alternative
// lies below, and (ties aside) n_top threads and hardly more slots have a
// logit that reaches it. (Of several warps' maxima the two largest of every
// lane are taken for all: a bound hardly lower, for a part of the sorting.) Their
// packs alone are read again; what reaches the bound is collected, and sorted in
// runs of 32. One warp's instructions are what this costs: every step leaves the
// next one little to look at.
template <typename T, int TPR, int U, int WARPS, typename S>
__device__ __forceinline__ uint64_t alternatives(const S& mine, const float (&most)[WARPS],
                                                 const T (*slots)[WARPS * 32], int n_top, int lane,
                                                 Finish<WARPS>& own) {
    constexpr int N = 16 / sizeof(T), kRead = Finish<WARPS>::kRead, kPlaces = Finish<WARPS>::kPlaces;
    constexpr int kOf = kSlots<T, WARPS>;
    using P = Pack<T, N>;
    // a bound from the two largest of every lane's threads: n_top of these reach it
    float first[1] = {most[0]}, second[1] = {-INFINITY};
#pragma unroll
    for (int w = 1; w < WARPS; ++w) {
        second[0] = fmaxf(second[0], fminf(first[0], most[w]));
        first[0] = fmaxf(first[0], most[w]);
    }
    sort_lists(first, lane);
    if constexpr (WARPS > 1) {
        sort_lists(second, lane);
        first[0] = merge_lists(first[0], __shfl_sync(kAll, second[0], 31 - lane), lane);
    }
    const float bound = fmaxf(__shfl_sync(kAll, first[0], n_top - 1), -FLT_MAX);
    int threads = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        const unsigned reach = __ballot_sync(kAll, most[w] >= bound);
        if (most[w] >= bound) own.thread[threads + __popc(reach & ((1u << lane) - 1))] = w * 32 + lane;
        threads += __popc(reach);
    }
    if (lane == 0) own.waiting = 0;
    __syncwarp();
    uint64_t found = 0, least = 0;  // the list so far, its n_top-th key
    bool some = false;
    auto take = [&](int count) {
        for (int c = 0; c < count; c += 32) {
            uint64_t next[1] = {c + lane < count ? own.candidate[c + lane] : 0};
            sort_lists(next, lane);
            found = some ? merge_lists(found, __shfl_sync(kAll, next[0], 31 - lane), lane) : next[0];
            some = true;
        }
        least = __shfl_sync(kAll, found, n_top - 1);
        __syncwarp();
        if (lane == 0) own.waiting = 0;
        __syncwarp();
    };
    const int per = (mine.stages + kOf - 1) / kOf, packs = per * U;  // stages and packs of a slot
    const int more = 32u / packs, rest = 32 - more * packs, lane_which = unsigned(lane) / packs;
    // the packs of `places` slots: item i is pack i % packs of the (i / packs)-th
    auto read = [&](int places) {
        int which = lane_which, at = lane - lane_which * packs;
        for (int first = 0; first < places * packs; first += 32 * kRead) {
            int pack[kRead];
#pragma unroll
            for (int r = 0; r < kRead; ++r) {
                pack[r] = mine.end;
                if (first + 32 * r >= places * packs) continue;
                if (which < places) {
                    const int place = own.place[which];
                    pack[r] = mine.begin + ((place >> 16) * packs + at) * TPR + (place & 0xffff);
                }
                if (pack[r] < mine.end && mine.packs.whole(pack[r]))
                    copy_async<16>(&own.again[r][lane], mine.packs.base + int64_t(pack[r]) * N);
                which += more, at += rest;
                if (at >= packs) at -= packs, ++which;
            }
            copy_commit();
            copy_wait<0>();
#pragma unroll
            for (int r = 0; r < kRead; ++r) {
                if (first + 32 * r >= places * packs) break;
                bool any = false;
                if (pack[r] < mine.end) {
                    const P q[1] = {mine.packs.whole(pack[r]) ? *reinterpret_cast<const P*>(&own.again[r][lane])
                                                              : mine.packs.edge(pack[r], kNone<T>)};
                    any = largest(q) >= bound;
                    if (any) {
                        for (int i = 0; i < N; ++i) {
                            const float v = to_f32(q[0].v[i]);
                            if (!(v >= bound)) continue;
                            const uint64_t k =
                                key_of(v, static_cast<uint32_t>(int64_t(pack[r]) * N + i - mine.packs.skew));
                            if (k > least) own.candidate[atomicAdd(&own.waiting, 1)] = k;
                        }
                    }
                }
                if (__any_sync(kAll, any)) {
                    __syncwarp();
                    const int waiting = own.waiting;
                    __syncwarp();
                    if (waiting >= kCandidates) take(waiting);
                }
            }
        }
        __syncwarp();
    };
    int places = 0;
    const int used = (mine.stages + per - 1) / per;
    for (int i = 0; i < used * threads; i += 32) {
        // item i + lane: thread by thread, slot by slot
        const int item = i + lane, slot = unsigned(item) / threads;
        const int who = own.thread[item - slot * threads];
        const float most_here = to_f32(slots[min(slot, kOf - 1)][who]);
        bool reaches = slot < used && most_here >= bound;
        if (least != 0) {  // many equal logits: columns behind the ones found already are not read
            const int64_t column = (mine.begin + int64_t(slot) * packs * TPR + who) * N - mine.packs.skew;
            reaches = reaches && key_of(most_here, static_cast<uint32_t>(column < 0 ? 0 : column)) > least;
        }
        const unsigned lanes = __ballot_sync(kAll, reaches);
        if (reaches) own.place[places + __popc(lanes & ((1u << lane) - 1))] = slot << 16 | who;
        places += __popc(lanes);
        if (places >= kPlaces) {
            __syncwarp();
            read(places);
            places = 0;
        }
    }
    __syncwarp();
    read(places);
    take(own.waiting);
    return found;
}

// TPR threads per row: a warp (four rows to a block), or a block's, or with
// CLUSTER those of a cluster's blocks. Every thread keeps the running maximum and
// sums of its packs and a warp joins its lanes'.
//
// Packs come in by asynchronous copies into a ring that each thread has to
// itself, so no barrier guards it, kStages - 1 stages ahead and on into the next
// rows: HBM stays busy while a row's parts are joined (8192 x 128256 bf16, loads
// straight into registers: 428 us). Where a block's warps share a row one more
// joins their parts, finds the alternatives and writes the outputs while they
// are at the next row; one barrier per row hands over (without that warp, the
// alternatives found by all: 535 us where this takes 359).
//
// Without alternatives near what HBM gives (80% of its peak in the counters): 8192 x
// 128256 bf16 293 us (105% of the rate of a copy, half of whose bytes are writes),
// with entropy 315 (98%); 16384 x 32000 158 (98%); 8192 x 32000 fp32 with entropy and
// 5 alternatives 157 (98%). With alternatives in 16 bits by instruction issue beside
// HBM: 8192 x 128256 with entropy and 20 of them 359 us (86%), 16384 x 32000 with 5
// 212 (73%). fp16 takes longer (297, 337, 408 and 239 us for these), most where its
// forms with entropy spill up to 64 bytes at the registers of five blocks per SM.
// Few rows: 3 x 128256 with 8 alternatives 9.0 us, 1 x 128256 without 4.6; 512 x 512
// 2.8 us. All logits equal, with 20 alternatives: 8192 x 128256 657 us, 16384 x 32000
// 637; rising ones 373 and 302.
template <typename T, int TPR, int U, bool ENTROPY, bool TOP, bool CLUSTER>
__global__ void __launch_bounds__(Geometry<T, TPR, U>::kBlock, TPR == 32 ? 6 : TPR == 128 ? 5 : 3)
    k_logprobs(const __grid_constant__ ForwardArgs<T> a) {
    using Geo = Geometry<T, TPR, U>;
    constexpr int N = 16 / sizeof(T), kWarps = Geo::kWarps, kAhead = Geo::kStages - 1;
    constexpr bool kAlone = Geo::kAlone;
    using P = Pack<T, N>;
    using Mine = Share<T, TPR, U>;
    extern __shared__ __align__(16) unsigned char smem[];
    const int group = kAlone ? threadIdx.x / 32 : 0, lane = threadIdx.x % 32;
    // without alternatives only parts are handed over, and a cluster exchanges one
    using Hand = Handover<T, kWarps>;
    Hand* const hand = reinterpret_cast<Hand*>(smem + Geo::kRing) + (TOP ? group * Geo::kHands : 0);
    auto parts = [&](int set) {
        return TOP ? hand[set].part : reinterpret_cast<Part*>(smem + Geo::kRing) + set * kWarps;
    };
    Finish<kWarps>& own =
        reinterpret_cast<Finish<kWarps>*>(smem + Geo::kRing + Geo::kHand * Geo::kHands * Geo::kGroups)[group];
    const int rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
    const int ranks = CLUSTER ? static_cast<int>(cluster_size()) : 1;
    const int64_t step = int64_t(gridDim.x) / ranks * Geo::kGroups;
    auto token_of = [&](int64_t row) { return a.tokens && row < a.rows ? token_at(a.tokens, a.token_type, row) : 0; };
    auto share = [&](int64_t row) {
        return Mine(a.logits + row * a.stride, a.vocab, rank, ranks, a.logits,
                    a.logits + (a.rows - 1) * a.stride + a.vocab);
    };
    int64_t row = (CLUSTER ? blockIdx.x / ranks : blockIdx.x) * int64_t(Geo::kGroups) + group;
    int64_t token = token_of(row);

    auto finish = [&](const Mine& mine, float z, Part part, const float (&most)[kWarps], int set) {
        uint64_t found = 0;
        if constexpr (TOP) found = alternatives<T, TPR, U, kWarps>(mine, most, hand[set].most, a.n_top, lane, own);
        if constexpr (CLUSTER) {
            Part* const shared = TOP ? &own.part : parts(Geo::kHands);
            if (lane == 0) *shared = part;
            if (TOP) own.key[lane] = found;
            cluster_barrier();
            if (rank == 0) {
                part = Part::nothing();
                if (lane < ranks) {
                    part.m = load_cluster(&shared->m, lane);
                    part.s = load_cluster(&shared->s, lane);
                    part.a = load_cluster(&shared->a, lane);
                }
                join(part);
                if constexpr (TOP) {
                    uint64_t of[8];
#pragma unroll
                    for (int r = 0; r < 8; ++r) of[r] = r < ranks ? load_cluster(&own.key[lane], r) : 0;
#pragma unroll
                    for (int half = 4; half > 0; half /= 2)
#pragma unroll
                        for (int r = 0; r < half; ++r)
                            if (half < ranks)
                                of[r] = merge_lists(of[r], __shfl_sync(kAll, of[r + half], 31 - lane), lane);
                    found = of[0];
                }
            }
            cluster_barrier();
            if (rank != 0) return;
        }
        // nothing but -inf: no sum; NaN or +inf: a sum of NaN
        const bool empty = part.s == 0.f, bad = !(part.s >= 0.f);
        // the largest term is 1, up to what the powers and their correction round: no
        // probability is above 1, and no entropy below 0
        const float s = empty ? 0.f : max_nan(part.s, 1.f);
        const float m = bad ? NAN : empty ? 0.f : part.m, log_sum = logf(s);
        if (lane == 0) {
            if (a.tokens) a.logp[row] = empty && token < a.vocab ? -INFINITY : (z - m) - log_sum;
            if (a.lse) a.lse[row] = m + log_sum;
            if (a.entropy) a.entropy[row] = empty ? 0.f : max_nan(log_sum - part.a / s * kLn2, 0.f);
            if (a.row_max) a.row_max[row] = m, a.log_sum[row] = log_sum;
        }
        if (TOP && lane < a.n_top) {
            const bool have = found != 0 && !bad;
            a.top_tokens[row * a.n_top + lane] = have ? static_cast<int64_t>(column_of(found)) : -1;
            a.top_logp[row * a.n_top + lane] = bad ? NAN : have ? (logit_of(found) - m) - log_sum : -INFINITY;
        }
    };
    auto leave_out = [&]() {
        if (rank != 0) return;
        if (lane == 0) {
            a.logp[row] = 0.f;
            if (a.lse) a.lse[row] = 0.f;
            if (a.entropy) a.entropy[row] = 0.f;
            if (a.row_max) a.row_max[row] = 0.f, a.log_sum[row] = 0.f;
        }
        if (TOP && lane < a.n_top) {
            a.top_tokens[row * a.n_top + lane] = -1;
            a.top_logp[row * a.n_top + lane] = -INFINITY;
        }
    };

    if (!kAlone && threadIdx.x >= Geo::kMain) {  // the warp that finishes the others' rows
        for (int set = 0; row < a.rows; row += step) {
            const int64_t after = token_of(row + step);
            if (token < 0) {
                leave_out();
            } else {
                float z = NAN;
                if (lane == 0 && a.tokens && token < a.vocab) z = to_f32(a.logits[row * a.stride + token]);
                __syncthreads();
                Part part = lane < kWarps ? parts(set)[lane] : Part::nothing();
                join(part);
                const Mine mine = share(row);
                float most[kWarps];
                if constexpr (TOP) {
#pragma unroll
                    for (int w = 0; w < kWarps; ++w) most[w] = hand[set].best[w][lane];
                }
                finish(mine, z, part, most, set);
                set ^= 1;
            }
            token = after;
        }
        return;
    }

    const int t = threadIdx.x % TPR;
    P* const ring = reinterpret_cast<P*>(smem) + threadIdx.x;
    auto slot = [&](int stage, int u) { return ring + (stage * U + u) * Geo::kMain; };
    const T none = from_f32<T>(-INFINITY);
    // what is copied next: a stage of row `next`, which has next_stages to go
    int64_t next = row, next_token = token, next_after = token_of(row + step);
    auto skip = [&]() {  // to the first row that is not left out
        while (next < a.rows && next_token < 0) next += step, next_token = next_after, next_after = token_of(next + step);
    };
    skip();
    const T* src;                    // this thread's first pack of the stage
    int at, low, span, next_stages;  // its number; which ones are copied
    auto begin = [&]() {
        if (next >= a.rows) return;
        const Mine m = share(next);
        at = m.begin + t, src = m.packs.base + int64_t(at) * N;
        low = m.low, span = m.high - m.low, next_stages = m.stages;
    };
    begin();
    auto issue = [&](int stage) {
        if (next < a.rows) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (static_cast<unsigned>(at + u * TPR - low) < static_cast<unsigned>(span))
                    copy_async<16>(slot(stage, u), src + u * TPR * N);
            at += U * TPR, src += U * TPR * N;
            if (--next_stages == 0) {
                next += step, next_token = next_after, next_after = token_of(next + step);
                skip();
                begin();
            }
        }
        copy_commit();
    };
    for (int k = 0; k < kAhead; ++k) issue(k);
    int stage = 0, set = 0;
    for (; row < a.rows; row += step) {
        const int64_t after = token_of(row + step);
        if (token < 0) {
            if (kAlone) leave_out();
            token = after;
            continue;
        }
        const Mine mine = share(row);
        // the token's logit; a row's only warp finds it in the ring
        float z = NAN;
        const int64_t place = token + mine.packs.skew;
        const int place_pack = kAlone && a.tokens && token < a.vocab ? static_cast<int>(place / N) : -1;
        Part part = Part::nothing();
        constexpr int kOf = kSlots<T, kWarps>;
        const int per = TOP ? (mine.stages + kOf - 1) / kOf : 1;
        T* slot_to = TOP ? &hand[set].most[0][t] : nullptr;
        int in_slot = 0;
        float slot_most = -INFINITY;
        for (int k = 0; k < mine.stages; ++k) {
            copy_wait<kAhead - 1>();
            const int first = mine.begin + k * U * TPR;
            P q[U];
#pragma unroll
            for (int u = 0; u < U; ++u) q[u] = *slot(stage, u);
            // the row's edges and the share's end
            if ((k == 0 && rank == 0) || k == mine.stages - 1) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int p = first + u * TPR + t;
                    if (p >= mine.end) {
                        q[u] = filled<T, N>(kNone<T>);
                    } else if (!mine.packs.whole(p)) {
                        if (p >= mine.low && p < mine.high) {
#pragma unroll
                            for (int i = 0; i < N; ++i)
                                if (!mine.packs.inside(int64_t(p) * N + i)) q[u].v[i] = none;
                        } else {
                            q[u] = mine.packs.edge(p, kNone<T>);
                        }
                    }
                }
            }
            if (kAlone && place_pack >= first && place_pack < first + U * TPR && place_pack % TPR == t) {
                z = to_f32(place_pack >= mine.low && place_pack < mine.high
                               ? reinterpret_cast<const T*>(slot(stage, (place_pack - first) / TPR))[place % N]
                               : mine.packs.base[place]);
            }
            issue(stage == 0 ? kAhead : stage - 1);  // where the stage before this one was
            const float here = largest(q);
            add_packs<ENTROPY>(part, q, here);
            if constexpr (TOP) {
                slot_most = fmaxf(slot_most, here);
                if (++in_slot == per) {
                    *slot_to = from_f32<T>(slot_most);
                    slot_to += TPR, in_slot = 0, slot_most = -INFINITY;
                }
            }
            stage = stage == kAhead ? 0 : stage + 1;
        }
        if (TOP && in_slot > 0) *slot_to = from_f32<T>(slot_most);
        const float most = part.m;
        join(part);
        if constexpr (kAlone) {
            const float mosts[1] = {most};
            __syncwarp();  // the slots
            finish(mine, __shfl_sync(kAll, z, place_pack & 31), part, mosts, 0);
        } else {
            if (lane == 0) parts(set)[t / 32] = part;
            if (TOP) hand[set].best[t / 32][lane] = most;
            __syncthreads();
            if constexpr (CLUSTER) {
                cluster_barrier();
                cluster_barrier();
            }
        }
        token = after;
        if (!kAlone) set ^= 1;
    }
    copy_wait<0>();
}

template <typename T, int TPR, int U, bool ENTROPY, bool TOP, bool CLUSTER>
int launch(const ForwardArgs<T>& a, int ranks, cudaStream_t s) {
    using Geo = Geometry<T, TPR, U>;
    auto* kernel = k_logprobs<T, TPR, U, ENTROPY, TOP, CLUSTER>;
    static Resident resident;
    const int64_t work = (a.rows + Geo::kGroups - 1) / Geo::kGroups * ranks;
    const int grid = resident.grid(reinterpret_cast<const void*>(kernel), Geo::kBlock, Geo::bytes(TOP), work);
    if (grid == 0) return DL_ERR_CUDA;
    cudaLaunchConfig_t config = {};
    config.gridDim = dim3(grid < ranks ? ranks : grid / ranks * ranks);
    config.blockDim = dim3(Geo::kBlock);
    config.dynamicSmemBytes = Geo::bytes(TOP);
    config.stream = s;
    cudaLaunchAttribute cluster;
    cluster.id = cudaLaunchAttributeClusterDimension;
    cluster.val.clusterDim.x = ranks;
    cluster.val.clusterDim.y = cluster.val.clusterDim.z = 1;
    config.attrs = &cluster;
    config.numAttrs = CLUSTER ? 1 : 0;
    if (cudaLaunchKernelEx(&config, kernel, a) != cudaSuccess) {
        cudaGetLastError();
        return DL_ERR_CUDA;
    }
    return DL_OK;
}

template <typename T, int TPR, int U, bool CLUSTER, bool TOP = true>
int launch(const ForwardArgs<T>& a, int ranks, cudaStream_t s) {
    if constexpr (TOP) {
        if (a.n_top)
            return a.entropy ? launch<T, TPR, U, true, true, CLUSTER>(a, ranks, s)
                             : launch<T, TPR, U, false, true, CLUSTER>(a, ranks, s);
    }
    return a.entropy ? launch<T, TPR, U, true, false, CLUSTER>(a, ranks, s)
                     : launch<T, TPR, U, false, false, CLUSTER>(a, ranks, s);
}

// A warp per row while that leaves it less than 64 packs per lane and there
// are rows for every warp (65536 x 4096 bf16 102 us, 331 with a block of eight
// warps; 16384 x 32000 166, with a block of four 157). Its stages are of four packs
// per lane for rows of more than 96 packs without alternatives (32768 x 8192 84 us,
// in stages of two 93), of two for shorter rows (262144 x 512 146 us, in stages of
// four 173) and with alternatives, whose shared memory leaves fewer blocks. So
// the order of a row's sums goes by n_top too.
//
// Few rows by clusters of up to eight blocks of eight warps, while there are SMs
// for them and the shares fill a block (64 x 128256: 8.0 us, with one block each 19);
// else a block of four warps (eight: 16384 x 32000 185 us for 161 then, 8192 x 128256
// 291 for 297, with entropy and 20 alternatives 388 for 376, 600 x 128256 30 for 27).
// That one rule also takes the rows that do not fill the SMs, where eight warps
// were faster: 300 x 128256 15.3 us for 17.9, with 8 alternatives 21 for 25,
// 300 x 32000 7.1 for 7.5.
template <typename T>
int forward(const ForwardArgs<T>& a, cudaStream_t s) {
    constexpr int N = 16 / sizeof(T);
    const int64_t packs = a.vocab / N;
    if (packs <= 2048 && (packs <= 256 || a.rows >= 4096))
        return packs > 96 && !a.n_top ? launch<T, 32, 4, false, false>(a, 1, s) : launch<T, 32, 2, false>(a, 1, s);
    int ranks = 1;
    while (ranks < 8 && a.rows * ranks * 2 <= 3 * sm_count() && packs / (ranks * 2) >= 256) ranks *= 2;
    if (ranks > 1) return launch<T, 256, 4, true>(a, ranks, s);
    return launch<T, 128, 4, false>(a, 1, s);
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
