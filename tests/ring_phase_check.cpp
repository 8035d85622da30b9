// Steps dl::RingPhase (csrc/dl_phase.h) against a model of the barriers of a
// ring of copies: for every number of rounds and every round whose wait runs
// out, the waits that follow meet exactly the copies in flight.
#include <cstdio>

#include "dl_phase.h"

namespace {

template <int S>
struct Model {
    int issued[S] = {}, landed[S] = {};  // copies, i.e. phases begun and completed
    // mbarrier.try_wait.parity: true when the phase of this parity is the one
    // completed last; a wait for the phase in progress lets its copy land
    bool passes_at_once(int s, unsigned parity) const { return (landed[s] & 1u) != parity; }
};

template <int S>
int run(int rounds, int failing) {
    Model<S> m;
    dl::RingPhase<S> phase;
    bool ok = true;
    auto issue = [&](int stage, int round) {
        if (round < rounds && ok) ++m.issued[stage];
    };
    for (int i = 0; i < S - 1; ++i) issue(i, i);
    for (int r = 0; r < rounds; ++r) {
        if (ok) {
            if (phase.stage != r % S || phase.parity != unsigned(r / S & 1)) return 1;
            if (m.passes_at_once(phase.stage, phase.parity)) return 2;
            ok = r != failing;
            if (ok)
                m.landed[phase.stage] = m.issued[phase.stage];
            else
                for (int i = 0; i < phase.in_flight(rounds - r); ++i) {
                    const int s = phase.stage_of(i);
                    if (m.passes_at_once(s, phase.parity_of(i))) return 3;  // would not wait for its copy
                    if (m.issued[s] != m.landed[s] + 1) return 4;           // waits for a copy nobody issued
                    m.landed[s] = m.issued[s];
                }
        }
        issue(phase.before(), r + S - 1);
        phase.advance();
    }
    for (int s = 0; s < S; ++s)
        if (m.issued[s] != m.landed[s]) return 5;  // the block would end with a copy in flight
    return 0;
}

template <int S>
int all() {
    for (int rounds = 1; rounds <= 5 * S + 2; ++rounds)
        for (int failing = 0; failing <= rounds; ++failing)  // == rounds: none fails
            if (const int why = run<S>(rounds, failing)) {
                std::printf("%d stages, %d rounds, round %d fails: %d\n", S, rounds, failing, why);
                return 1;
            }
    return 0;
}

}  // namespace

int main() {
    if (all<2>() || all<3>() || all<4>() || all<5>()) return 1;
    std::puts("ok");
    return 0;
}
