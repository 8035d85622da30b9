// How rotary positions share out a head's elements and a token's heads, up to
// the largest sizes that fit 31 bits. Plain C++ so that the host can step it there.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define DL_FORM_FN __host__ __device__ __forceinline__
#else
#define DL_FORM_FN inline
#endif

namespace dl {

// A unit of a head: what one thread turns or copies at once. Packs of
// neighbouring pairs lie at multiples of N from the head's start, the last
// turned one perhaps with elements behind the rotated part; units of two packs
// hold nothing but pairs, or nothing but elements behind them.
template <int N, bool INTERLEAVED>
struct Form {
    static constexpr bool kTwo = !INTERLEAVED || N == 1;  // two packs, else one
    static constexpr int kSize = kTwo ? 2 * N : N, kPairs = kSize / 2;
    static constexpr int kStep = INTERLEAVED ? kSize : N;  // from a turned unit's first pack to the next one's
    DL_FORM_FN static int turned(int pairs) { return (pairs + kPairs - 1) / kPairs; }
    // elements of a head behind the rotated part's units
    DL_FORM_FN static int rest(int head_dim, int pairs) { return head_dim - turned(pairs) * kSize; }
    DL_FORM_FN static int units(int head_dim, int pairs) {
        return turned(pairs) + (rest(head_dim, pairs) / N * N + kSize - 1) / kSize;
    }
    // whether packs of N suit these sizes
    static bool fits(int head_dim, int pairs) {
        return kTwo ? pairs % N == 0 || N == 1 : rest(head_dim, pairs) >= 0;
    }
    // the first element of unit u of a head with `turned` units of pairs
    DL_FORM_FN static int first(int u, int turned) {
        return u < turned ? u * kStep : turned * kSize + (u - turned) * kSize;
    }
    // whether the unit at element `low` has a second pack: a turned one does, one
    // behind the pairs where the head has room for it
    DL_FORM_FN static bool two(bool turns, int low, int head_dim) {
        return kTwo && (turns || low <= head_dim - 2 * N);
    }
};

// The heads of one thread: from its own on every lanes-th, ROWS of them at a
// time. Unsigned, so that the step past the last of up to 2^31 - 1 heads (of
// ROWS * lanes, some thousands) stays in range.
template <int ROWS>
struct HeadWalk {
    uint32_t at, lanes, heads;
    DL_FORM_FN HeadWalk(int head, int lanes_, int heads_)
        : at(static_cast<uint32_t>(head)), lanes(static_cast<uint32_t>(lanes_)), heads(static_cast<uint32_t>(heads_)) {}
    DL_FORM_FN bool more() const { return at < heads; }
    DL_FORM_FN uint32_t row(int r) const { return at + static_cast<uint32_t>(r) * lanes; }
    DL_FORM_FN bool has(int r) const { return row(r) < heads; }
    DL_FORM_FN void next() { at += ROWS * lanes; }
};

}  // namespace dl
