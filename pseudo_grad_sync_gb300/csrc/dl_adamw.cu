// A learner's inner optimiser step: the global gradient norm with its clip
// coefficient, and AdamW over every tensor of a list of fragments with
// states in 32 or in 8 bits.
#include <float.h>
#include <math.h>
#include <stdint.h>

#include "dl_types.cuh"

namespace dl {
namespace {

// ---------------------------------------------------------------------------
// gradient norm

constexpr int kNormBuffers = 64;  // per launch; longer lists take several
constexpr int kNormBlocks = 2048;
constexpr int kNormVecs = 8;      // 16-byte loads of a thread in flight
constexpr int kNormChunk = kThreads * kNormVecs;  // 16-byte vectors per chunk

struct NormWorkspace {  // after the header; zeroed once, left as found
    double total;       // sum over the launches of one call so far; the first sets it
    uint32_t done;      // blocks of this launch that have finished
    double partial[kNormBlocks];
};

struct NormArgs {
    const void* g[kNormBuffers];
    int64_t numel[kNormBuffers];
    int64_t chunk_end[kNormBuffers];  // running number of chunks
    int n;
    int first, last;  // whether this is the call's first, its last launch
    double max_norm;
    float* out;
    NormWorkspace* ws;
};

__device__ __forceinline__ void unpack(const uint4& q, float (&v)[4], float) {
    v[0] = __uint_as_float(q.x), v[1] = __uint_as_float(q.y);
    v[2] = __uint_as_float(q.z), v[3] = __uint_as_float(q.w);
}
__device__ __forceinline__ void unpack(const uint4& q, float (&v)[8], __nv_bfloat16) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
}

// A group's sum of squares in this range lost nothing to fp32's range: none
// of its squares overflowed, and a subnormal square is off by 2^-150 at most.
// A group of zeros (told by the words' bits) adds nothing; any other group
// (tiny or huge values, Inf, NaN) is summed again in fp64.
constexpr float kSquareLo = 0x1p-100f, kSquareHi = 0x1p126f;

// read once, not kept in L1
__device__ __forceinline__ uint4 load_once(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// One group's squares in fp64, read again: out of line, so that the groups in
// range keep their registers.
template <typename T>
__device__ __noinline__ double squares64(const uint4* body, int64_t i, int64_t vecs) {
    constexpr int W = 16 / sizeof(T);
    double s = 0.0;
    for (int u = 0; u < kNormVecs && i < vecs; ++u, i += kThreads) {
        const uint4 q = __ldg(body + i);
        if ((q.x | q.y | q.z | q.w) == 0) continue;
        float v[W];
        unpack(q, v, T());
#pragma unroll
        for (int w = 0; w < W; ++w) s = fma(static_cast<double>(v[w]), static_cast<double>(v[w]), s);
    }
    return s;
}

// Elements before the first 16-byte boundary of a buffer.
template <typename T>
__host__ __device__ inline int64_t head_of(const void* p, int64_t n) {
    const int64_t h = static_cast<int64_t>((16 - (reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) /
                      static_cast<int64_t>(sizeof(T));
    return h < n ? h : n;
}

// One pass, bound by HBM: 2 flops for 2 or 4 bytes. Chunks of 32 KB go round
// the blocks of a persistent grid, each thread with eight 16-byte loads in
// flight. Squares are added in fp32 within a thread's chunk (at most 64 of
// them: relative error 64 * 2^-24) and in fp64 beyond; adding every square in
// fp64 instead ran at a twelfth of the speed (GB300's fp64 rate). The block
// that finishes last joins the partial sums, lane by lane in a fixed order,
// and leaves the ticket at zero: one launch and no memset per 64 buffers.
// 1.1G bf16 gradients: 309 us, 7.1 TB/s (105% of the copy rate; it only
// reads), zeros among them or not. Twelve small tensors (150001 fp32): 4.9 us
// on the device.
template <typename T>
__global__ void __launch_bounds__(kThreads) k_grad_norm(const __grid_constant__ NormArgs a) {
    constexpr int W = 16 / sizeof(T);
    __shared__ double red[kWarps];
    __shared__ bool final_block;
    double sum = 0.0;
    int j = 0;
    const int64_t chunks = a.chunk_end[a.n - 1];
    for (int64_t c = blockIdx.x; c < chunks; c += gridDim.x) {
        while (c >= a.chunk_end[j]) ++j;
        const int64_t first = c - (j ? a.chunk_end[j - 1] : 0);
        const T* g = static_cast<const T*>(a.g[j]);
        const int64_t n = a.numel[j], head = head_of<T>(g, n);
        const int64_t vecs = (n - head) / W;
        const uint4* body = reinterpret_cast<const uint4*>(g + head);
        uint4 q[kNormVecs];
        const int64_t i0 = first * kNormChunk + threadIdx.x;
#pragma unroll
        for (int u = 0; u < kNormVecs; ++u)
            q[u] = i0 + u * kThreads < vecs ? load_once(body + i0 + u * kThreads) : uint4{0, 0, 0, 0};
        float part[4] = {0.f, 0.f, 0.f, 0.f};
        uint32_t any = 0;
#pragma unroll
        for (int u = 0; u < kNormVecs; ++u) {
            any |= q[u].x | q[u].y | q[u].z | q[u].w;
            float v[W];
            unpack(q[u], v, T());
#pragma unroll
            for (int w = 0; w < W; ++w) part[w & 3] = fmaf(v[w], v[w], part[w & 3]);
        }
        const float group = (part[0] + part[1]) + (part[2] + part[3]);
        if (group >= kSquareLo && group <= kSquareHi)
            sum += static_cast<double>(group);
        else if (any & (sizeof(T) == 4 ? 0x7fffffffu : 0x7fff7fffu))
            sum += squares64<T>(body, i0, vecs);
        if (first == 0) {
            const int64_t rest = n - vecs * W;  // the head's and the tail's elements
            if (threadIdx.x < rest) {
                const int64_t i = threadIdx.x < head ? threadIdx.x : threadIdx.x + vecs * W;
                const double v = to_f32(g[i]);
                sum = fma(v, v, sum);
            }
        }
    }
    for (int sh = 16; sh; sh >>= 1) sum += __shfl_xor_sync(kFull, sum, sh);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) red[warp] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double s = 0.0;
        for (int w = 0; w < kWarps; ++w) s += red[w];
        a.ws->partial[blockIdx.x] = s;
        __threadfence();
        final_block = atomicAdd(&a.ws->done, 1u) == gridDim.x - 1;
    }
    __syncthreads();
    if (!final_block) return;
    __threadfence();
    double s = 0.0;
    for (int b = threadIdx.x; b < static_cast<int>(gridDim.x); b += kThreads)
        s += __ldcg(&a.ws->partial[b]);
    for (int sh = 16; sh; sh >>= 1) s += __shfl_xor_sync(kFull, s, sh);
    if (lane == 0) red[warp] = s;
    __syncthreads();
    if (threadIdx.x == 0) {
        double t = a.first ? 0.0 : a.ws->total;  // a call that failed halfway leaves a total
        for (int w = 0; w < kWarps; ++w) t += red[w];
        a.ws->done = 0;
        a.ws->total = a.last ? 0.0 : t;
        if (a.last) {
            const double norm = sqrt(t);
            a.out[0] = static_cast<float>(norm);
            a.out[1] = !isfinite(norm) ? __int_as_float(0x7fc00000)
                       : norm > a.max_norm ? static_cast<float>(a.max_norm / norm)
                                           : 1.0f;
        }
    }
}

// ---------------------------------------------------------------------------
// AdamW

constexpr int kAdamJobs = 32;  // per launch; longer lists take several
constexpr int kBlock = DL_ADAMW_BLOCK;

struct AdamJob {
    float* theta;
    const void* grad;
    void* m;
    void* v;
    float* m_scale;
    float* v_scale;
    __nv_bfloat16* copy;
    const float* decay;
    const int64_t* off;
    int64_t n;
    int64_t slot0;     // slots of all jobs before this one
    int64_t work_end;  // running number of tiles (32-bit states) or slots (8-bit)
    int T;
};

struct AdamArgs {
    AdamJob job[kAdamJobs];
    int n;
    int64_t run;  // 8-bit states: consecutive slots of a warp
    float lr_wd, step_size, beta1, om_beta1, beta2, om_beta2, inv_root_bc2, eps;
    float one;  // 1
    uint64_t key;
    const float* clip;
};

// The approximate quotients below take a denominator beyond 2^126 for infinite
// (the update would be lost). A finite root is below 2^64 and its scale below
// 2^27, so eps alone could reach that far.
constexpr double kMostEps = 0x1p125;

// theta' from the new moments; root = sqrt(v')
__device__ __forceinline__ float step_theta(const AdamArgs& a, float theta, float m, float root,
                                            float keep) {
    const float denom = fmaf(root, a.inv_root_bc2, a.eps);
    return fmaf(-a.step_size, __fdividef(m, denom), theta * keep);
}

__device__ __forceinline__ float clip_coef(const AdamArgs& a) { return a.clip ? __ldg(a.clip + 1) : 1.0f; }

__device__ __forceinline__ float keep_of(const AdamArgs& a, const AdamJob& J, int t) {
    return J.decay ? 1.0f - a.lr_wd * __ldg(J.decay + t) : 1.0f - a.lr_wd;
}

// Four elements of a type as one aligned load or store.
__device__ __forceinline__ void load4(const float* p, float (&v)[4]) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
}
__device__ __forceinline__ void load4(const __nv_bfloat16* p, float (&v)[4]) {
    const uint2 q = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xffff0000u);
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
    __nv_bfloat162 q[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
    *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(q);
}

__device__ __forceinline__ float rcp_approx(float v) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float sqrt_approx(float v) {
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

constexpr int kGroups32 = 2;                         // groups of four elements per thread
constexpr int kTile32 = kThreads * 4 * kGroups32;

// States in 32 bits: elementwise, bound by HBM (24 bytes of state and
// parameters plus the gradient and the copy for some 20 flops). A block takes
// one tile of 2048 elements, all its loads first; blocks are scheduled by the
// hardware, which keeps the SMs level (a persistent grid with equal shares
// left up to a fifth of the SMs idle at the end). Only a tile that meets
// several tensors looks up each group's decay. Square root and quotient are
// the approximate instructions (2 ulp; nothing is stored of them but theta,
// whose update they scale).
// 1.1B set (24 fragments, bf16 gradients and copy): 4333 us, 7.1 TB/s (105%
// of the copy rate); 2000 ragged tensors (48M elements, fp32): 205 us, 6.6 TB/s.
// Loads of single elements instead of fours: 5648 and 370 us.

template <typename G>
__global__ void __launch_bounds__(kThreads) k_adamw(const __grid_constant__ AdamArgs a) {
    const float coef = clip_coef(a);
    if (!isfinite(coef)) return;
    int j = 0;
    while (static_cast<int64_t>(blockIdx.x) >= a.job[j].work_end) ++j;
    const AdamJob& J = a.job[j];
    const int64_t base = (blockIdx.x - (j ? a.job[j - 1].work_end : 0)) * int64_t(kTile32);
    const int n = static_cast<int>(min(J.n - base, int64_t(kTile32)));  // of this tile
    const G* g = static_cast<const G*>(J.grad) + base;
    float* m = static_cast<float*>(J.m) + base;
    float* v = static_cast<float*>(J.v) + base;
    float* theta = J.theta + base;
    __nv_bfloat16* copy = J.copy ? J.copy + base : nullptr;
    float tv[kGroups32][4], gv[kGroups32][4], mv[kGroups32][4], vv[kGroups32][4];
#pragma unroll
    for (int u = 0; u < kGroups32; ++u) {
        const int i = (u * kThreads + static_cast<int>(threadIdx.x)) * 4;
        if (i + 4 <= n) {
            load4(theta + i, tv[u]);
            load4(g + i, gv[u]);
            load4(m + i, mv[u]);
            load4(v + i, vv[u]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                tv[u][e] = gv[u][e] = mv[u][e] = vv[u][e] = 0.f;
                if (i + e < n) {
                    tv[u][e] = theta[i + e], gv[u][e] = to_f32(g[i + e]);
                    mv[u][e] = m[i + e], vv[u][e] = v[i + e];
                }
            }
        }
    }
    // the tile's tensor; a tile of several looks each group's up
    int t = 0;
    bool one = true;
    if (J.decay) {
        t = tensor_containing(J.off, J.T, base);
        one = __ldg(J.off + t + 1) >= base + n;
    }
    const float keep = keep_of(a, J, t);
#pragma unroll
    for (int u = 0; u < kGroups32; ++u) {
        const int i = (u * kThreads + static_cast<int>(threadIdx.x)) * 4;
        if (i >= n) continue;
        float kv[4] = {keep, keep, keep, keep};
        if (!one) {
            int te = tensor_from(J.off, t, J.T, base + i);
            int64_t end = __ldg(J.off + te + 1);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                while (base + i + e >= end && te < J.T - 1) end = __ldg(J.off + ++te + 1);
                kv[e] = keep_of(a, J, te);
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float gi = gv[u][e] * coef;
            mv[u][e] = fmaf(a.beta1, mv[u][e], a.om_beta1 * gi);
            vv[u][e] = fmaf(a.beta2, vv[u][e], a.om_beta2 * (gi * gi));
            tv[u][e] = step_theta(a, tv[u][e], mv[u][e], sqrt_approx(vv[u][e]), kv[e]);
        }
        if (i + 4 <= n) {
            store4(theta + i, tv[u]);
            store4(m + i, mv[u]);
            store4(v + i, vv[u]);
            if (copy) store4(copy + i, tv[u]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (i + e < n) {
                    theta[i + e] = tv[u][e], m[i + e] = mv[u][e], v[i + e] = vv[u][e];
                    if (copy) copy[i + e] = __float2bfloat16_rn(tv[u][e]);
                }
        }
    }
}

__host__ __device__ inline uint64_t mix64(uint64_t z) {
    z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
    z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
    return z ^ (z >> 31);
}
constexpr uint64_t kGolden = 0x9E3779B97F4A7C15ull;

// Smallest exponent field of a block's largest value: k = -53
constexpr uint32_t kMinExp = 127 - 53;

// 2^(k-7) of a block whose largest magnitude has these bits
__device__ __forceinline__ float block_scale(uint32_t top) {
    const uint32_t e = max(top >> 23, kMinExp);
    return e == 255 ? __int_as_float(0x7fc00000) : __uint_as_float((e - 7) << 23);
}
// its reciprocal (a power of two; any finite value for a NaN scale)
__device__ __forceinline__ float block_inverse(uint32_t top) {
    return __uint_as_float((261 - max(top >> 23, kMinExp)) << 23);
}

// four e4m3 codes, the first in the low byte, to fp32
__device__ __forceinline__ void decode4(uint32_t c, float (&x)[4]) {
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
    const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&lo));
    const float2 q = __half22float2(*reinterpret_cast<const __half2*>(&hi));
    x[0] = p.x, x[1] = p.y, x[2] = q.x, x[3] = q.y;
}

// Four values to codes with stochastic rounding by the hardware conversion:
// of the 32 random bits, values 0 and 2 use the low and the high half, 1 and
// 3 the same halves in reverse bit order; the first operand is the top byte.
__device__ __forceinline__ uint32_t encode4(const float (&x)[4], uint32_t bits) {
    uint32_t c;
    asm("cvt.rs.satfinite.e4m3x4.f32 %0, {%1, %2, %3, %4}, %5;"
        : "=r"(c)
        : "f"(x[3]), "f"(x[2]), "f"(x[1]), "f"(x[0]), "r"(bits));
    return c;
}

// first tensor t with off[t+1] / 128 + t + 1 > slot
__device__ __forceinline__ int tensor_of_slot(const int64_t* off, int T, int64_t slot) {
    int lo = 0, hi = T - 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(off + mid + 1) / kBlock + mid + 1 > slot)
            hi = mid;
        else
            lo = mid + 1;
    }
    return lo;
}

// The tensor of a warp's current slot, walking forward.
struct SlotCursor {
    int t;
    int64_t o0, o1, first, next;  // elements [o0, o1), slots [first, next)
    __device__ __forceinline__ void load(const int64_t* off) {
        o0 = __ldg(off + t), o1 = __ldg(off + t + 1);
        first = o0 / kBlock + t, next = o1 / kBlock + t + 1;
    }
    __device__ __forceinline__ void seek(const int64_t* off, int64_t slot) {
        while (slot >= next) ++t, load(off);
    }
};

__device__ __forceinline__ float max_nan(float x, float y, float z) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(x), "f"(y), "f"(z));
    return r;
}
__device__ __forceinline__ float rsqrt_approx(float v) {
    float r;
    asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}
// One lane's share of a block: four elements (those past a tensor's end are
// zeros and are not stored).
struct Quad {
    float2 th[2], gr[2];
    uint32_t cm, cs;
    float msc, ssc;
};

// Moments from here on have the rounded square root from root2 (compared with
// the exact function for every float from here to FLT_MAX: no difference).
constexpr float kRootLo = 0x1p-100f;

// sqrt(v): the estimate g = v y with y = rsqrt(v), corrected once by its
// residual v - g^2, which the fused multiply-add gives (Markstein 1990).
__device__ __forceinline__ float2 root2(float2 v) {
    const float2 y = make_float2(rsqrt_approx(v.x), rsqrt_approx(v.y));
    const float2 g = mul2(v, y);
    const float2 less = fma2(g, g, mul2(v, both(-1.f)));
    return fma2(less, mul2(y, both(-0.5f)), g);
}

// The step of one quad: theta and the codes in place; all 32 lanes of the
// block's warp call it. Returns the bits of the block's largest moments.
__device__ __forceinline__ void step_quad(const AdamArgs& a, float coef, float keep, uint64_t z,
                                          Quad& q, uint32_t& mtop, uint32_t& stop) {
    float c[4], d[4];
    decode4(q.cm, c);
    decode4(q.cs, d);
    // m's scale, a power of two, is folded into beta1: the same bits as value =
    // code * scale first. s takes its own product: folded into a small beta2 the
    // smallest scale's square would leave fp32's normal range, and a square that
    // is Inf could come out finite (measured with the fold: 0.5% faster).
    const float2 b1 = both(a.beta1 * q.msc), b2 = both(a.beta2), ssc = both(q.ssc);
    // The definition rounds the products before the sum. A packed product and
    // a packed sum come out fused (CUDA 13.0, their .rn notwithstanding: exact
    // cancellations then leave a residue), so the sums are x * one + y with a
    // one that the compiler does not know.
    const float2 one = both(a.one);
    float2 m[2], v[2], r[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float2 cd = make_float2(c[2 * h], c[2 * h + 1]);
        const float2 s = mul2(make_float2(d[2 * h], d[2 * h + 1]), ssc);
        const float2 g = mul2(q.gr[h], both(coef));
        m[h] = fma2(mul2(cd, b1), one, mul2(g, both(a.om_beta1)));
        v[h] = fma2(mul2(mul2(s, s), b2), one, mul2(mul2(g, g), both(a.om_beta2)));
        r[h] = root2(v[h]);
    }
    // Zeros and tiny values take the exact function, as does Inf, whose
    // corrected estimate is NaN (NaN stays NaN).
    const bool plain = fminf(fminf(v[0].x, v[0].y), fminf(v[1].x, v[1].y)) >= kRootLo &&
                       max_nan(max_nan(r[0].x, r[0].y, r[1].x), r[1].y, 0.f) < __int_as_float(0x7f800000);
    if (!plain) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            r[h] = make_float2(__fsqrt_rn(v[h].x), __fsqrt_rn(v[h].y));
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float2 denom = fma2(r[h], both(a.inv_root_bc2), both(a.eps));
        const float2 up = mul2(m[h], make_float2(rcp_approx(denom.x), rcp_approx(denom.y)));
        q.th[h] = fma2(up, both(-a.step_size), mul2(q.th[h], both(keep)));
    }
    const float m3 = max_nan(fabsf(m[0].x), fabsf(m[0].y), fabsf(m[1].x));
    const float s3 = max_nan(r[0].x, r[0].y, r[1].x);
    const float mt = max_nan(m3, fabsf(m[1].y), 0.f), st = max_nan(s3, r[1].y, 0.f);
    mtop = __reduce_max_sync(kFull, __float_as_uint(mt));
    stop = __reduce_max_sync(kFull, __float_as_uint(st) & 0x7fffffffu);
    const float2 minv = both(block_inverse(mtop)), sinv = both(block_inverse(stop));
    float mx[4], sx[4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const float2 x = mul2(m[h], minv), y = mul2(r[h], sinv);
        mx[2 * h] = x.x, mx[2 * h + 1] = x.y;
        sx[2 * h] = y.x, sx[2 * h + 1] = y.y;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {  // a positive root keeps at least the smallest code
        const float x = sx[e];
        sx[e] = fmaxf(x, 0x1p-9f);
        if (!plain && !(x > 0.f)) sx[e] = x;
    }
    q.cm = encode4(mx, static_cast<uint32_t>(z));
    q.cs = encode4(sx, static_cast<uint32_t>(z >> 32));
}

// ---------------------------------------------------------------------------
// A warp's run of whole blocks. Each warp has a ring of stages in shared
// memory that asynchronous copies fill some blocks ahead; a stage holds the
// aligned groups of four elements ("quads") that a block touches: 32, or 33
// when the block starts A = 1, 2 or 3 elements into its first quad.
constexpr int kStages = 5;
constexpr int64_t kMostRun = 32;  // slots of a warp: 16 KB of theta (34 instead: 4% slower)

template <typename G>
struct __align__(16) Stage {
    float4 th[33];
    Pack<G, 4> gr[33];
    uint32_t cm[33], cs[33];
    float scale[2];
};

// the four elements from A on of two consecutive quads
template <int A>
__device__ __forceinline__ void shifted(const float4* q, float2 (&v)[2]) {
    const float4 x = q[0];
    if constexpr (A == 0) {
        v[0] = make_float2(x.x, x.y), v[1] = make_float2(x.z, x.w);
    } else {
        const float4 y = q[1];
        const float w[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
        v[0] = make_float2(w[A], w[A + 1]), v[1] = make_float2(w[A + 2], w[A + 3]);
    }
}
template <int A>
__device__ __forceinline__ void shifted(const Pack<float, 4>* q, float2 (&v)[2]) {
    shifted<A>(reinterpret_cast<const float4*>(q), v);
}
template <int A>
__device__ __forceinline__ void shifted(const Pack<__nv_bfloat16, 4>* q, float2 (&v)[2]) {
    const uint2 x = *reinterpret_cast<const uint2*>(q);
    uint32_t lo = x.x, hi = x.y;
    if constexpr (A != 0) {
        const uint2 y = *reinterpret_cast<const uint2*>(q + 1);
        const uint32_t w[4] = {x.x, x.y, y.x, y.y};
        lo = __funnelshift_r(w[A / 2], w[A / 2 + 1], 16 * (A & 1));
        hi = __funnelshift_r(w[A / 2 + 1], w[(A + 1) / 2 + 1], 16 * (A & 1));
    }
    v[0] = make_float2(__uint_as_float(lo << 16), __uint_as_float(lo & 0xffff0000u));
    v[1] = make_float2(__uint_as_float(hi << 16), __uint_as_float(hi & 0xffff0000u));
}

// `count` whole blocks from element `begin` (begin % 4 == A), slot `slot` on.
// For A > 0 the A elements before `begin` are of a block that this warp did.
template <typename G, int A>
__device__ __forceinline__ void run_blocks(const AdamArgs& a, const AdamJob& J, float coef, float keep,
                                           int64_t begin, int64_t slot, int count, int lane,
                                           Stage<G>* ring) {
    const int64_t q0 = begin - A + 4 * lane;  // this lane's quad of the first block
    float* const th = J.theta + q0;
    const G* const g = static_cast<const G*>(J.grad) + q0;
    uint8_t* const m8 = static_cast<uint8_t*>(J.m) + q0;
    uint8_t* const s8 = static_cast<uint8_t*>(J.v) + q0;
    __nv_bfloat16* const copy = J.copy ? J.copy + q0 : nullptr;
    float* const sc = (lane == 0 ? J.m_scale : J.v_scale) + slot;  // of lanes 0 and 1
    auto issue = [&](int i, Stage<G>& st) {
        const int o = i * kBlock;
        copy_async<16>(&st.th[lane], th + o);
        copy_async<4 * sizeof(G)>(&st.gr[lane], g + o);
        copy_async<4>(&st.cm[lane], m8 + o);
        copy_async<4>(&st.cs[lane], s8 + o);
        if (lane < 2) copy_async<4>(&st.scale[lane], sc + i);
        if (A > 0 && lane == 0) {  // the block's last A elements
            copy_async<16>(&st.th[32], th + o + kBlock, 4 * A);
            copy_async<4 * sizeof(G)>(&st.gr[32], g + o + kBlock, sizeof(G) * A);
            copy_async<4>(&st.cm[32], m8 + o + kBlock, A);
            copy_async<4>(&st.cs[32], s8 + o + kBlock, A);
        }
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
        if (i < count) issue(i, ring[i]);
        copy_commit();
    }
    uint64_t counter = a.key + ((J.slot0 + slot) * (kBlock / 4) + lane) * kGolden;
    // What the block before left of this block's first quad (lane 0 only): the
    // warp wrote it, and lane 0 writes it again with the rest of the quad.
    float left[A + 1];
    uint32_t left_m = 0, left_s = 0;
    if constexpr (A > 0) {
        __syncwarp();
        if (lane == 0) {
#pragma unroll
            for (int k = 0; k < A; ++k) {
                left[k] = th[k];
                left_m |= uint32_t(m8[k]) << (8 * (4 - A + k));
                left_s |= uint32_t(s8[k]) << (8 * (4 - A + k));
            }
        }
    }
    Stage<G>* st = ring;                     // the block's stage
    Stage<G>* freed = ring + (kStages - 1);  // the one of the block before
#pragma unroll (A == 0 ? 2 : 1)
    for (int i = 0; i < count; ++i) {
        copy_wait<kStages - 2>();
        __syncwarp();  // the stage has every lane's copies, and `freed` every lane's reads
        if (i + kStages - 1 < count) issue(i + kStages - 1, *freed);
        copy_commit();
        Quad q;
        shifted<A>(&st->th[lane], q.th);
        shifted<A>(&st->gr[lane], q.gr);
        q.cm = A ? __funnelshift_r(st->cm[lane], st->cm[lane + 1], 8 * A) : st->cm[lane];
        q.cs = A ? __funnelshift_r(st->cs[lane], st->cs[lane + 1], 8 * A) : st->cs[lane];
        q.msc = st->scale[0], q.ssc = st->scale[1];
        freed = st;
        st = st == ring + (kStages - 1) ? ring : st + 1;
        uint32_t mtop, stop;
        step_quad(a, coef, keep, mix64(counter), q, mtop, stop);
        counter += (kBlock / 4) * kGolden;
        float out[4] = {q.th[0].x, q.th[0].y, q.th[1].x, q.th[1].y};
        const int o = i * kBlock;
        if constexpr (A > 0) {
            // quads as they lie in memory: the lane before gives the first A elements
            const int from = (lane + 31) & 31;
            float own[4], got[A];
#pragma unroll
            for (int k = 0; k < 4; ++k) own[k] = out[k];
#pragma unroll
            for (int k = 0; k < A; ++k) got[k] = __shfl_sync(kFull, own[4 - A + k], from);
            const uint32_t pm = __shfl_sync(kFull, q.cm, from), ps = __shfl_sync(kFull, q.cs, from);
#pragma unroll
            for (int k = 0; k < 4; ++k) out[k] = k < A ? (lane ? got[k] : left[k]) : own[k - A];
            q.cm = __funnelshift_l(lane ? pm : left_m, q.cm, 8 * A);
            q.cs = __funnelshift_l(lane ? ps : left_s, q.cs, 8 * A);
#pragma unroll
            for (int k = 0; k < A; ++k) left[k] = got[k];
            left_m = pm, left_s = ps;
        }
        store4(th + o, out);
        *reinterpret_cast<uint32_t*>(m8 + o) = q.cm;
        *reinterpret_cast<uint32_t*>(s8 + o) = q.cs;
        if (copy) store4(copy + o, out);
        if (lane < 2) sc[i] = block_scale(lane ? stop : mtop);
    }
    if (A > 0 && lane == 0) {
        const int o = count * kBlock;
#pragma unroll
        for (int k = 0; k < A; ++k) {
            th[o + k] = left[k];
            m8[o + k] = static_cast<uint8_t>(left_m >> (8 * (4 - A + k)));
            s8[o + k] = static_cast<uint8_t>(left_s >> (8 * (4 - A + k)));
            if (copy) copy[o + k] = __float2bfloat16_rn(left[k]);
        }
    }
    copy_wait<0>();
    __syncwarp();  // before the ring is filled again
}

// One block at any element, of any length up to 128.
template <typename G>
__device__ __forceinline__ void any_block(const AdamArgs& a, const AdamJob& J, float coef, float keep,
                                          int64_t begin, int64_t end, int64_t slot, int lane) {
    const int64_t i0 = begin + 4 * lane;
    const int cnt = static_cast<int>(max(int64_t(0), min(int64_t(4), end - i0)));
    float* th = J.theta + i0;
    const G* g = static_cast<const G*>(J.grad) + i0;
    uint8_t* m8 = static_cast<uint8_t*>(J.m) + i0;
    uint8_t* s8 = static_cast<uint8_t*>(J.v) + i0;
    Quad q;
    q.msc = J.m_scale[slot], q.ssc = J.v_scale[slot];
    float t4[4], g4[4];
    q.cm = q.cs = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        t4[e] = g4[e] = 0.f;
        if (e < cnt) {
            t4[e] = th[e];
            g4[e] = to_f32(g[e]);
            q.cm |= uint32_t(m8[e]) << (8 * e);
            q.cs |= uint32_t(s8[e]) << (8 * e);
        }
    }
    q.th[0] = make_float2(t4[0], t4[1]), q.th[1] = make_float2(t4[2], t4[3]);
    q.gr[0] = make_float2(g4[0], g4[1]), q.gr[1] = make_float2(g4[2], g4[3]);
    uint32_t mtop, stop;
    step_quad(a, coef, keep, mix64(a.key + ((J.slot0 + slot) * (kBlock / 4) + lane) * kGolden), q, mtop,
              stop);
    const float out[4] = {q.th[0].x, q.th[0].y, q.th[1].x, q.th[1].y};
#pragma unroll
    for (int e = 0; e < 4; ++e)
        if (e < cnt) {
            th[e] = out[e];
            m8[e] = static_cast<uint8_t>(q.cm >> (8 * e));
            s8[e] = static_cast<uint8_t>(q.cs >> (8 * e));
            if (J.copy) J.copy[i0 + e] = __float2bfloat16_rn(out[e]);
        }
    if (lane == 0) {
        J.m_scale[slot] = block_scale(mtop);
        J.v_scale[slot] = block_scale(stop);
    }
}

// States in 8 bits. A warp takes runs of blocks, a lane four elements of each.
// Traffic is 12 bytes per element plus the gradient and the copy, so the
// arithmetic counts: 265 instructions per block of 128 elements against about
// 350 issue slots that HBM leaves (issue active 63%). Hence the packed fp32 pairs, the hardware's
// stochastic conversion (one instruction for four codes), power-of-two scales
// (no division), one hash per four elements, and a rounded root in six
// instructions. Copies run kStages - 1 blocks ahead in the
// warp's ring (loads into registers, two blocks at a time: 1441 us). Blocks
// of a tensor that starts off a multiple of four elements go through the same
// ring as shifted quads (element by element: 233 us for the ragged set).
// Runs of 32 blocks, scheduled by the hardware; equal shares for a persistent
// grid took 1211 us, runs of 16 about 1600. Three blocks of threads per SM (80
// registers) with five stages against four (64) with four: the same time
// there, but the 1.1B set with fp32 gradients 3221 against 3293 and the ragged
// set 170 against 177. The loop of unshifted blocks is unrolled twice; the
// shifted ones' is not (ragged set 194 us when it is).
// 415M-element fragment (bf16 gradients and copy): 1122 us, 6.0 TB/s (88% of
// the copy rate); 200M elements that are mostly zero, whose roots take the
// exact function: 537 against 476 us dense.
// 2000 ragged tensors (48M elements, fp32 gradients): 171 us, 4.5 TB/s (66%).
// Neither issue (63%) nor HBM (56%) is full there. The same set with its sizes
// rounded to fours takes 152 us, to whole blocks 143, one tensor of that size
// 136 (83%), and four times the elements run at 78%: what it pays is the
// shifts and the first block of each run, which is loaded element by element
// (15 us), blocks cut short and changes of tensor (17), and a call of 3.2 waves
// whose warps fill and drain their rings once each (the rest).
template <typename G>
__global__ void __launch_bounds__(kThreads, 3) k_adamw8(const __grid_constant__ AdamArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    const float coef = clip_coef(a);
    if (!isfinite(coef)) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    Stage<G>* ring = reinterpret_cast<Stage<G>*>(smem) + warp * kStages;
    int64_t at = (int64_t(blockIdx.x) * kWarps + warp) * a.run;  // slot over the launch's jobs
    const int64_t last = min(at + a.run, a.job[a.n - 1].work_end);
    for (int j = 0; at < last; ++j) {
        const AdamJob& J = a.job[j];
        if (at >= J.work_end) continue;
        const int64_t base = j ? a.job[j - 1].work_end : 0;
        int64_t s = at - base;
        const int64_t end = min(last, J.work_end) - base;
        at = end + base;
        SlotCursor c;
        c.t = tensor_of_slot(J.off, J.T, s);
        c.load(J.off);
        bool own = false;  // whether the block before s was this warp's, of the same tensor
        while (s < end) {
            if (s >= c.next) c.seek(J.off, s), own = false;
            const int64_t begin = c.o0 + (s - c.first) * kBlock;
            if (begin >= c.o1) {  // a slot without a block
                ++s;
                continue;
            }
            const float keep = keep_of(a, J, c.t);
            const int count = static_cast<int>(min(min(end - s, (c.o1 - begin) / kBlock), int64_t(1) << 20));
            const int shift = static_cast<int>(begin & 3);
            if (count > 0 && (shift == 0 || own)) {
                switch (shift) {
                    case 0: run_blocks<G, 0>(a, J, coef, keep, begin, s, count, lane, ring); break;
                    case 1: run_blocks<G, 1>(a, J, coef, keep, begin, s, count, lane, ring); break;
                    case 2: run_blocks<G, 2>(a, J, coef, keep, begin, s, count, lane, ring); break;
                    default: run_blocks<G, 3>(a, J, coef, keep, begin, s, count, lane, ring); break;
                }
                s += count;
            } else {
                any_block<G>(a, J, coef, keep, begin, c.o1, s, lane);
                ++s;
            }
            own = true;
        }
    }
}

}  // namespace
}  // namespace dl

using namespace dl;

extern "C" size_t dl_grad_norm_workspace_bytes(void) {
    return align256(kWsHeader + sizeof(NormWorkspace));
}

extern "C" int dl_grad_norm(const void* const* grads, const int64_t* numel, int32_t n_grads,
                            int32_t grad_type, double max_norm, float* d_out, void* d_workspace,
                            size_t workspace_bytes, void* stream) {
    if (n_grads < 0 || (n_grads > 0 && (!grads || !numel)) || !d_out || !(max_norm > 0.0) ||
        (grad_type != DL_F32 && grad_type != DL_BF16))
        return DL_ERR_ARG;
    for (int32_t i = 0; i < n_grads; ++i) {
        if (numel[i] < 0 || (numel[i] > 0 && !grads[i])) return DL_ERR_ARG;
        if (numel[i] > 0 && !aligned_to(grads[i], type_size(grad_type))) return DL_ERR_ALIGN;
    }
    if (!aligned_to(d_out, 4)) return DL_ERR_ALIGN;
    if (!d_workspace || workspace_bytes < dl_grad_norm_workspace_bytes()) return DL_ERR_WORKSPACE;
    if (!aligned_to(d_workspace, 256)) return DL_ERR_ALIGN;
    const void* kernel = grad_type == DL_F32 ? reinterpret_cast<const void*>(k_grad_norm<float>)
                                             : reinterpret_cast<const void*>(k_grad_norm<__nv_bfloat16>);
    NormArgs a;
    a.max_norm = max_norm;
    a.out = d_out;
    a.ws = reinterpret_cast<NormWorkspace*>(static_cast<char*>(d_workspace) + kWsHeader);
    int32_t i = 0;
    int first = 1;
    do {
        a.n = 0;
        int64_t chunks = 0;
        for (; i < n_grads && a.n < kNormBuffers; ++i) {
            if (numel[i] == 0) continue;
            const int64_t head = grad_type == DL_F32 ? head_of<float>(grads[i], numel[i])
                                                     : head_of<__nv_bfloat16>(grads[i], numel[i]);
            const int64_t vecs = (numel[i] - head) * static_cast<int64_t>(type_size(grad_type)) / 16;
            chunks += vecs ? (vecs + kNormChunk - 1) / kNormChunk : 1;
            a.g[a.n] = grads[i];
            a.numel[a.n] = numel[i];
            a.chunk_end[a.n++] = chunks;
        }
        a.first = first;
        a.last = i == n_grads;
        first = 0;
        if (a.n == 0) {  // nothing left to read: one block writes the result
            a.g[0] = nullptr;
            a.numel[0] = 0;
            a.chunk_end[0] = 0;
            a.n = 1;
        }
        static Resident resident[2];
        int grid = resident[grad_type].grid(kernel, kThreads, 0, chunks ? chunks : 1);
        if (grid == 0) return DL_ERR_CUDA;
        if (grid > kNormBlocks) grid = kNormBlocks;
        // Half the blocks read as fast until a call is long, and their end
        // (ticket, join of the partial sums) is shorter: 80 MB 22.0 -> 19.4 us,
        // 320 MB 54.5 -> 52.7, but 2.2 GB 310 -> 318.
        const int few = 4 * sm_count();
        if (grid > few && chunks < int64_t(few) * 32) grid = few;
        void* args[] = {&a};
        if (cudaLaunchKernel(kernel, dim3(grid), dim3(kThreads), args, 0,
                             static_cast<cudaStream_t>(stream)) != cudaSuccess) {
            cudaGetLastError();  // reported here, not by a later call
            return DL_ERR_CUDA;
        }
    } while (i < n_grads);
    return DL_OK;
}

extern "C" int64_t dl_adamw_scale_slots(const dl_fragment* frag) {
    HostFrag f;
    const int st = check_fragment(frag, &f);
    return st != DL_OK ? st : f.n / kBlock + f.T;
}

extern "C" int dl_adamw_step(const dl_adamw_job* jobs, int32_t n_jobs, int32_t grad_type,
                             int32_t state_type, const dl_adamw_config* cfg, const float* d_clip,
                             void* stream) {
    if (n_jobs < 0 || (n_jobs > 0 && !jobs) || !cfg || (grad_type != DL_F32 && grad_type != DL_BF16) ||
        (state_type != DL_F32 && state_type != DL_E4M3))
        return DL_ERR_ARG;
    if (!(cfg->lr >= 0.0 && cfg->lr <= FLT_MAX) || !(cfg->beta1 >= 0.0 && cfg->beta1 < 1.0) ||
        !(cfg->beta2 >= 0.0 && cfg->beta2 < 1.0) || !(cfg->eps >= FLT_MIN && cfg->eps <= kMostEps) ||
        !(cfg->weight_decay >= 0.0 && cfg->weight_decay <= FLT_MAX) || cfg->step < 1)
        return DL_ERR_ARG;
    if (!aligned_to(d_clip, 4)) return DL_ERR_ALIGN;
    const bool by8 = state_type == DL_E4M3;
    for (int32_t i = 0; i < n_jobs; ++i) {
        const dl_adamw_job& q = jobs[i];
        HostFrag f;
        const int st = check_fragment(q.frag, &f);
        if (st != DL_OK) return st;
        if (f.n == 0) continue;
        if (!q.theta || !q.grad || !q.m || !q.v || (by8 && (!q.m_scale || !q.v_scale)))
            return DL_ERR_ARG;
        for (const void* p : {static_cast<const void*>(q.theta), q.grad, static_cast<const void*>(q.m),
                              static_cast<const void*>(q.v), static_cast<const void*>(q.theta_bf16)})
            if (!aligned16(p)) return DL_ERR_ALIGN;
        if (!aligned_to(q.m_scale, 4) || !aligned_to(q.v_scale, 4) || !aligned_to(q.d_decay, 4))
            return DL_ERR_ALIGN;
    }
    AdamArgs a;
    const double t = static_cast<double>(cfg->step);
    const double bc1 = 1.0 - pow(cfg->beta1, t), bc2 = 1.0 - pow(cfg->beta2, t);
    if (cfg->lr * cfg->weight_decay > FLT_MAX || cfg->lr / bc1 > FLT_MAX) return DL_ERR_ARG;
    a.lr_wd = static_cast<float>(cfg->lr * cfg->weight_decay);
    a.step_size = static_cast<float>(cfg->lr / bc1);
    a.beta1 = static_cast<float>(cfg->beta1);
    a.om_beta1 = static_cast<float>(1.0 - cfg->beta1);
    a.beta2 = static_cast<float>(cfg->beta2);
    a.om_beta2 = static_cast<float>(1.0 - cfg->beta2);
    a.inv_root_bc2 = static_cast<float>(1.0 / sqrt(bc2));
    a.eps = static_cast<float>(cfg->eps);
    a.one = 1.0f;
    a.key = mix64(cfg->seed + static_cast<uint64_t>(cfg->step) * kGolden);
    a.clip = d_clip;
    int64_t slot0 = 0;
    int32_t i = 0;
    while (i < n_jobs) {
        a.n = 0;
        int64_t work = 0;
        for (; i < n_jobs && a.n < kAdamJobs; ++i) {
            const dl_adamw_job& q = jobs[i];
            HostFrag f;
            check_fragment(q.frag, &f);
            const int64_t slots = f.n / kBlock + f.T;
            if (f.n > 0) {
                work += by8 ? slots : (f.n + kTile32 - 1) / kTile32;
                a.job[a.n++] = AdamJob{q.theta, q.grad, q.m, q.v, q.m_scale, q.v_scale,
                                       static_cast<__nv_bfloat16*>(q.theta_bf16), q.d_decay,
                                       f.d_offsets, f.n, slot0, work, f.T};
            }
            slot0 += slots;
        }
        if (a.n == 0) continue;
        const void* kernel =
            by8 ? (grad_type == DL_F32 ? reinterpret_cast<const void*>(k_adamw8<float>)
                                       : reinterpret_cast<const void*>(k_adamw8<__nv_bfloat16>))
                : (grad_type == DL_F32 ? reinterpret_cast<const void*>(k_adamw<float>)
                                       : reinterpret_cast<const void*>(k_adamw<__nv_bfloat16>));
        size_t smem = 0;
        int64_t grid = work;
        if (by8) {  // as many warps as the GPU holds, each with one run of slots
            smem = kWarps * kStages * (grad_type == DL_F32 ? sizeof(Stage<float>) : sizeof(Stage<__nv_bfloat16>));
            static Resident resident[2];
            grid = resident[grad_type].grid(kernel, kThreads, smem, (work + kWarps - 1) / kWarps);
            if (grid == 0) return DL_ERR_CUDA;
            a.run = (work + grid * kWarps - 1) / (grid * kWarps);
            if (a.run > kMostRun) {
                a.run = kMostRun;
                grid = (work + kWarps * a.run - 1) / (kWarps * a.run);
            }
        }
        if (grid > INT32_MAX) return DL_ERR_ARG;
        void* args[] = {&a};
        if (cudaLaunchKernel(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), args, smem,
                             static_cast<cudaStream_t>(stream)) != cudaSuccess) {
            cudaGetLastError();
            return DL_ERR_CUDA;
        }
    }
    return DL_OK;
}
