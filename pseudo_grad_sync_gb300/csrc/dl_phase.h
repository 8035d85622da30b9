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
    int pending = -1;     // after a failed wait: rounds issued and not waited for

    DL_PHASE_FN bool ok() const { return pending < 0; }
    // the stage of the round before, free for the round STAGES - 1 ahead
    DL_PHASE_FN int before() const { return stage == 0 ? STAGES - 1 : stage - 1; }
    // After a failed wait the ring stays where it is: stage and parity then
    // tell which copies are in flight.
    DL_PHASE_FN void advance() {
        if (!ok()) return;
        parity ^= stage == STAGES - 1;
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    // the wait for this round ran out with `left` rounds to go, this one included
    DL_PHASE_FN void fail(int64_t left) { pending = left < STAGES - 1 ? static_cast<int>(left) : STAGES - 1; }
    // the i-th round in flight, i < pending
    DL_PHASE_FN int stage_of(int i) const { return stage + i >= STAGES ? stage + i - STAGES : stage + i; }
    DL_PHASE_FN uint32_t parity_of(int i) const { return parity ^ (stage + i >= STAGES); }
};

}  // namespace dl
