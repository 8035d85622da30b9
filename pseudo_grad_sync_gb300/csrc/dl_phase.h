// Which stage of a ring of copies holds which round, and what is still in
// flight once a bounded wait has run out. Plain C++ so that the host can step
// it against a model of the barriers.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define DL_PHASE_FN __host__ __device__ __forceinline__
#else
#define DL_PHASE_FN inline
#endif

namespace dl {

// Round r lies in stage r % STAGES, whose barrier completes phase r / STAGES
// with it. When round r is waited for, rounds r .. r + STAGES - 2 have been
// issued, as far as there are any.
template <int STAGES>
struct RingPhase {
    int stage = 0;        // of the round to wait for
    uint32_t parity = 0;  // of its phase

    // the stage of the round before, free for the round STAGES - 1 ahead
    DL_PHASE_FN int before() const { return stage == 0 ? STAGES - 1 : stage - 1; }
    DL_PHASE_FN void advance() {
        parity ^= stage == STAGES - 1;
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    // Rounds in flight at this round's wait, with `left` rounds to go (this one
    // included), and the stage and the parity of the i-th of them.
    DL_PHASE_FN static int in_flight(int64_t left) { return left < STAGES - 1 ? static_cast<int>(left) : STAGES - 1; }
    DL_PHASE_FN int stage_of(int i) const { return stage + i >= STAGES ? stage + i - STAGES : stage + i; }
    DL_PHASE_FN uint32_t parity_of(int i) const { return parity ^ (stage + i >= STAGES); }
};

}  // namespace dl
